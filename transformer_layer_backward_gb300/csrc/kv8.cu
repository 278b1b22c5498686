// The 8-bit K/V cache: rows quantised as they are written, and read back as floats.
#include "kv8.cuh"

namespace tlb {

namespace {

// A warp quantises the key and the value of one (row, head): four values a lane, HALVES times 128
// values of a head.  Bound by memory (5 or 3 bytes a value) from a few hundred rows on, below that by the launch:
// 2048 rows of 8 heads of 128 float32 5.0 us (4.2 TB/s), 8 rows 1.7 us.
template <typename T, int HALVES, bool VEC>
__global__ void __launch_bounds__(128) kv8_write_kernel(tlb_kv8 c, const T *__restrict__ k, int64_t k_row, int64_t k_head,
                                                        const T *__restrict__ v, int64_t v_row, int64_t v_head,
                                                        const int64_t *__restrict__ slots, int64_t items) {
    const int64_t item = int64_t(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5);
    if (item >= items) return;
    const int lane = threadIdx.x & 31, nkv = c.n_kv_heads, hd = c.head_dim;
    const int64_t row = item / nkv;
    const int h = int(item - row * nkv);
    const T *src[2] = {k + row * k_row + h * k_head, v + row * v_row + h * v_head};
    const int64_t slot = __ldg(slots + row);
    float x[2][HALVES][4];
#pragma unroll
    for (int w = 0; w < 2; ++w)
#pragma unroll
        for (int u = 0; u < HALVES; ++u) {
            const int d = u * 128 + lane * 4;               // head_dim % 16 == 0: four are there or none
            if (d >= hd) {
                x[w][u][0] = x[w][u][1] = x[w][u][2] = x[w][u][3] = 0.f;
            } else if (VEC) {
                const float4 f = load_float4(src[w] + d);
                x[w][u][0] = f.x; x[w][u][1] = f.y; x[w][u][2] = f.z; x[w][u][3] = f.w;
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e) x[w][u][e] = load_float(src[w] + d + e);
            }
        }
    if (slot < 0 || slot >= c.n_slots) return;
#pragma unroll
    for (int w = 0; w < 2; ++w) {
        uint32_t top = 0;
#pragma unroll
        for (int u = 0; u < HALVES; ++u)
#pragma unroll
            for (int e = 0; e < 4; ++e) top = max(top, magnitude(x[w][u][e]));
        top = __reduce_max_sync(0xffffffffu, top);
        float inv;
        const float s = block_scale(top, inv);
        uint8_t *dst = (w == 0 ? c.k : c.v) + (slot * nkv + h) * hd;
#pragma unroll
        for (int u = 0; u < HALVES; ++u) {
            const int d = u * 128 + lane * 4;
            if (d < hd)
                *reinterpret_cast<uint32_t *>(dst + d) =
                    to_e4m3x4(x[w][u][0] * inv, x[w][u][1] * inv, x[w][u][2] * inv, x[w][u][3] * inv);
        }
        if (lane == 0) (w == 0 ? c.k_scale : c.v_scale)[int64_t(h) * c.n_slots + slot] = s;
    }
}

// A warp reads the key and the value of one (row, head) back.  8192 rows of 8 heads of 128 to float32: 14.6 us, 5.8 TB/s,
// four fifths of it written.
template <typename T, int HALVES, bool VEC>
__global__ void __launch_bounds__(128) kv8_read_kernel(tlb_kv8 c, const int64_t *__restrict__ slots, int64_t items,
                                                       T *__restrict__ k, T *__restrict__ v, int64_t stride_row,
                                                       int64_t stride_head) {
    const int64_t item = int64_t(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5);
    if (item >= items) return;
    const int lane = threadIdx.x & 31, nkv = c.n_kv_heads, hd = c.head_dim;
    const int64_t row = item / nkv;
    const int h = int(item - row * nkv);
    const int64_t slot = __ldg(slots + row);
    const bool there = slot >= 0 && slot < c.n_slots;
    uint32_t y[2][HALVES];
    float s[2];
#pragma unroll
    for (int w = 0; w < 2; ++w) {
        s[w] = there ? __ldg((w == 0 ? c.k_scale : c.v_scale) + int64_t(h) * c.n_slots + slot) : 0.f;
#pragma unroll
        for (int u = 0; u < HALVES; ++u) {
            const int d = u * 128 + lane * 4;
            y[w][u] = there && d < hd
                          ? __ldg(reinterpret_cast<const uint32_t *>((w == 0 ? c.k : c.v) + (slot * nkv + h) * hd + d))
                          : 0u;
        }
    }
#pragma unroll
    for (int w = 0; w < 2; ++w)
#pragma unroll
        for (int u = 0; u < HALVES; ++u) {
            const int d = u * 128 + lane * 4;
            if (d >= hd) continue;
            const float2 a = e4m3x2_to_float2(y[w][u] & 0xFFFFu), b = e4m3x2_to_float2(y[w][u] >> 16);
            T *dst = (w == 0 ? k : v) + row * stride_row + h * stride_head + d;
            const float4 f = make_float4(a.x * s[w], a.y * s[w], b.x * s[w], b.y * s[w]);
            if (VEC) {
                store_float4(dst, f);
            } else {
                store_float(dst, f.x);
                store_float(dst + 1, f.y);
                store_float(dst + 2, f.z);
                store_float(dst + 3, f.w);
            }
        }
}

// Whether four elements of T at p, and at multiples of these strides from it, may be moved at once.
template <typename T> bool by_four(const void *p, int64_t a, int64_t b) {
    return reinterpret_cast<uintptr_t>(p) % (4 * sizeof(T)) == 0 && a % 4 == 0 && b % 4 == 0;
}

template <typename T>
int write_launch(const tlb_kv8 &c, const T *k, int64_t kr, int64_t kh, const T *v, int64_t vr, int64_t vh,
                 const int64_t *slots, int64_t rows, cudaStream_t st) {
    const int64_t items = rows * c.n_kv_heads;
    const unsigned grid = unsigned(ceil_div(items, 4));
    const bool vec = by_four<T>(k, kr, kh) && by_four<T>(v, vr, vh), two = c.head_dim > 128;
    auto kernel = two ? (vec ? kv8_write_kernel<T, 2, true> : kv8_write_kernel<T, 2, false>)
                      : (vec ? kv8_write_kernel<T, 1, true> : kv8_write_kernel<T, 1, false>);
    kernel<<<grid, 128, 0, st>>>(c, k, kr, kh, v, vr, vh, slots, items);
    return check_launch("kv8_write");
}

template <typename T>
int read_launch(const tlb_kv8 &c, const int64_t *slots, int64_t rows, T *k, T *v, int64_t sr, int64_t sh, cudaStream_t st) {
    const int64_t items = rows * c.n_kv_heads;
    const unsigned grid = unsigned(ceil_div(items, 4));
    const bool vec = by_four<T>(k, sr, sh) && by_four<T>(v, sr, sh), two = c.head_dim > 128;
    auto kernel = two ? (vec ? kv8_read_kernel<T, 2, true> : kv8_read_kernel<T, 2, false>)
                      : (vec ? kv8_read_kernel<T, 1, true> : kv8_read_kernel<T, 1, false>);
    kernel<<<grid, 128, 0, st>>>(c, slots, items, k, v, sr, sh);
    return check_launch("kv8_read");
}

}  // namespace

int kv8_check(const tlb_kv8 *c, const char *what) {
    TLB_REQUIRE(c != nullptr, TLB_EINVAL, "%s: null cache", what);
    TLB_REQUIRE(c->n_slots >= 0 && c->n_kv_heads >= 1 && c->head_dim >= 1, TLB_EINVAL, "%s: a size of the cache is not positive", what);
    TLB_REQUIRE(c->head_dim % 16 == 0 && c->head_dim <= 256, TLB_EUNSUPPORTED,
                "%s: head_dim %d is not a multiple of 16 up to 256", what, c->head_dim);
    TLB_REQUIRE(c->n_slots <= (int64_t(1) << 40) && c->n_kv_heads <= 65535, TLB_EUNSUPPORTED, "%s: the cache is too large", what);
    if (c->n_slots == 0) return TLB_OK;
    TLB_REQUIRE(c->k && c->v && c->k_scale && c->v_scale, TLB_EINVAL, "%s: null pointer in the cache", what);
    TLB_REQUIRE(aligned16(c->k) && aligned16(c->v), TLB_EINVAL, "%s: the cache's k and v must be 16-byte aligned", what);
    TLB_REQUIRE(aligned_to(c->k_scale, 4) && aligned_to(c->v_scale, 4), TLB_EINVAL, "%s: the cache's scales must be aligned", what);
    return TLB_OK;
}

}  // namespace tlb

using namespace tlb;

extern "C" {

int tlb_kv8_write(const tlb_kv8 *cache, int32_t type, const void *k, int64_t k_stride_row, int64_t k_stride_head,
                  const void *v, int64_t v_stride_row, int64_t v_stride_head, const int64_t *slots, int64_t rows,
                  void *stream) {
    clear_error();
    TLB_TRY(kv8_check(cache, "kv8_write"));
    TLB_REQUIRE(type == TLB_W_F32 || type == TLB_W_BF16, TLB_EINVAL, "kv8_write: type %d is neither f32 nor bf16", type);
    TLB_REQUIRE(rows >= 0, TLB_EINVAL, "kv8_write: negative size");
    TLB_REQUIRE(rows <= (int64_t(1) << 32) / cache->n_kv_heads, TLB_EUNSUPPORTED, "kv8_write: more than 2^32 rows of heads");
    if (rows == 0 || cache->n_slots == 0) return TLB_OK;
    TLB_REQUIRE(k && v && slots, TLB_EINVAL, "kv8_write: null pointer");
    const size_t wide = type == TLB_W_F32 ? 4 : 2;
    TLB_REQUIRE(aligned_to(k, wide) && aligned_to(v, wide) && aligned_to(slots, 8), TLB_EINVAL,
                "kv8_write: k, v and slots must be aligned to their elements");
    if (type == TLB_W_F32)
        return write_launch(*cache, static_cast<const float *>(k), k_stride_row, k_stride_head, static_cast<const float *>(v),
                            v_stride_row, v_stride_head, slots, rows, as_stream(stream));
    return write_launch(*cache, static_cast<const __nv_bfloat16 *>(k), k_stride_row, k_stride_head,
                        static_cast<const __nv_bfloat16 *>(v), v_stride_row, v_stride_head, slots, rows, as_stream(stream));
}

int tlb_kv8_read(const tlb_kv8 *cache, const int64_t *slots, int64_t rows, int32_t type, void *k, void *v,
                 int64_t stride_row, int64_t stride_head, void *stream) {
    clear_error();
    TLB_TRY(kv8_check(cache, "kv8_read"));
    TLB_REQUIRE(type == TLB_W_F32 || type == TLB_W_BF16, TLB_EINVAL, "kv8_read: type %d is neither f32 nor bf16", type);
    TLB_REQUIRE(rows >= 0, TLB_EINVAL, "kv8_read: negative size");
    TLB_REQUIRE(rows <= (int64_t(1) << 32) / cache->n_kv_heads, TLB_EUNSUPPORTED, "kv8_read: more than 2^32 rows of heads");
    if (rows == 0) return TLB_OK;
    TLB_REQUIRE(k && v && slots, TLB_EINVAL, "kv8_read: null pointer");
    const size_t wide = type == TLB_W_F32 ? 4 : 2;
    TLB_REQUIRE(aligned_to(k, wide) && aligned_to(v, wide) && aligned_to(slots, 8), TLB_EINVAL,
                "kv8_read: k, v and slots must be aligned to their elements");
    if (type == TLB_W_F32)
        return read_launch(*cache, slots, rows, static_cast<float *>(k), static_cast<float *>(v), stride_row, stride_head,
                           as_stream(stream));
    return read_launch(*cache, slots, rows, static_cast<__nv_bfloat16 *>(k), static_cast<__nv_bfloat16 *>(v), stride_row,
                       stride_head, as_stream(stream));
}

}  // extern "C"
