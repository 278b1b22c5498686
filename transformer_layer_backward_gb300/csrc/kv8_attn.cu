// Attention of single tokens over the 8-bit K/V cache, and its gradient.
#include <cmath>

#include "kv8.cuh"

namespace tlb {

namespace {

constexpr int kWarps = 4;
constexpr int kDims = 8;                 // 32 lanes x 8 dimensions: head_dim <= 256

__device__ __forceinline__ void load_row(const uint8_t *rows, int64_t at, int hd, int lane, float (&x)[kDims]) {
#pragma unroll
    for (int i = 0; i < kDims; ++i) x[i] = lane + 32 * i < hd ? e4m3x2_to_float2(rows[at + lane + 32 * i]).x : 0.f;
}

__device__ __forceinline__ float dot(const float (&a)[kDims], const float (&b)[kDims]) {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < kDims; ++i) s = fmaf(a[i], b[i], s);
    return warp_sum(s);
}

// One CTA a query head, its warps taking turns at the keys.
template <typename T>
__global__ void __launch_bounds__(kWarps * 32) kv8_attn_forward_simple(tlb_kv8 c, Kv8Pages pg, int n_heads, float scale,
                                                                       const T *__restrict__ q, T *__restrict__ ctx,
                                                                       float *__restrict__ lse) {
    __shared__ float sm[kWarps], sl[kWarps], so[kWarps][256];
    const int64_t b = blockIdx.x / n_heads;
    const int h = int(blockIdx.x - b * n_heads), kvh = h / (n_heads / c.n_kv_heads), hd = c.head_dim;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, len = kv8_length(pg, b);
    float x[kDims], o[kDims] = {}, m = -INFINITY, l = 0.f;
#pragma unroll
    for (int i = 0; i < kDims; ++i) x[i] = lane + 32 * i < hd ? load_float(q + int64_t(blockIdx.x) * hd + lane + 32 * i) * scale : 0.f;
    for (int j = warp; j < len; j += kWarps) {
        const int64_t slot = kv8_slot(pg, c.n_slots, b, j);
        if (slot < 0) continue;
        float k[kDims], v[kDims];
        load_row(c.k, (slot * c.n_kv_heads + kvh) * hd, hd, lane, k);
        load_row(c.v, (slot * c.n_kv_heads + kvh) * hd, hd, lane, v);
        const float s = dot(x, k) * c.k_scale[int64_t(kvh) * c.n_slots + slot], sv = c.v_scale[int64_t(kvh) * c.n_slots + slot];
        const float mn = fmaxf(m, s), old = m == -INFINITY ? 0.f : expf(m - mn), p = expf(s - mn);
        l = l * old + p;
#pragma unroll
        for (int i = 0; i < kDims; ++i) o[i] = o[i] * old + p * sv * v[i];
        m = mn;
    }
    if (lane == 0) { sm[warp] = m; sl[warp] = l; }
#pragma unroll
    for (int i = 0; i < kDims; ++i) so[warp][lane + 32 * i] = o[i];
    __syncthreads();
    float top = -INFINITY, total = 0.f;
    for (int w = 0; w < kWarps; ++w) top = fmaxf(top, sm[w]);
    for (int w = 0; w < kWarps; ++w) total += sl[w] > 0.f || sl[w] != sl[w] ? sl[w] * expf(sm[w] - top) : 0.f;
    for (int d = threadIdx.x; d < hd; d += blockDim.x) {
        float y = 0.f;
        for (int w = 0; w < kWarps; ++w) y += sl[w] > 0.f || sl[w] != sl[w] ? so[w][d] * expf(sm[w] - top) : 0.f;
        store_float(ctx + int64_t(blockIdx.x) * hd + d, total == 0.f ? 0.f : y / total);
    }
    if (threadIdx.x == 0) lse[blockIdx.x] = total == 0.f ? -INFINITY : top + logf(total);
}

// d_q = scale (sum p dp k - (sum p dp) (sum p k)); leaves D = sum p dp for the newest key's gradients.
template <typename T>
__global__ void __launch_bounds__(kWarps * 32) kv8_attn_backward_simple(tlb_kv8 c, Kv8Pages pg, int n_heads, float scale,
                                                                        const T *__restrict__ q, const float *__restrict__ lse,
                                                                        const T *__restrict__ d_ctx, T *__restrict__ d_q,
                                                                        float *__restrict__ D) {
    __shared__ float sd[kWarps], su[kWarps][256], sw[kWarps][256];
    const int64_t b = blockIdx.x / n_heads;
    const int h = int(blockIdx.x - b * n_heads), kvh = h / (n_heads / c.n_kv_heads), hd = c.head_dim;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, len = kv8_length(pg, b);
    const float norm = lse[blockIdx.x];
    float x[kDims], g[kDims], u[kDims] = {}, w[kDims] = {}, sum = 0.f;
#pragma unroll
    for (int i = 0; i < kDims; ++i) {
        x[i] = lane + 32 * i < hd ? load_float(q + int64_t(blockIdx.x) * hd + lane + 32 * i) * scale : 0.f;
        g[i] = lane + 32 * i < hd ? load_float(d_ctx + int64_t(blockIdx.x) * hd + lane + 32 * i) : 0.f;
    }
    for (int j = warp; j < len; j += kWarps) {
        const int64_t slot = kv8_slot(pg, c.n_slots, b, j);
        if (slot < 0) continue;
        float k[kDims], v[kDims];
        load_row(c.k, (slot * c.n_kv_heads + kvh) * hd, hd, lane, k);
        load_row(c.v, (slot * c.n_kv_heads + kvh) * hd, hd, lane, v);
        const float sk = c.k_scale[int64_t(kvh) * c.n_slots + slot], sv = c.v_scale[int64_t(kvh) * c.n_slots + slot];
        const float p = expf(dot(x, k) * sk - norm), dp = dot(g, v) * sv;
        sum += p * dp;
#pragma unroll
        for (int i = 0; i < kDims; ++i) {
            u[i] = fmaf(p * dp * sk, k[i], u[i]);
            w[i] = fmaf(p * sk, k[i], w[i]);
        }
    }
    if (lane == 0) sd[warp] = sum;
#pragma unroll
    for (int i = 0; i < kDims; ++i) {
        su[warp][lane + 32 * i] = u[i];
        sw[warp][lane + 32 * i] = w[i];
    }
    __syncthreads();
    sum = 0.f;
    for (int i = 0; i < kWarps; ++i) sum += sd[i];
    for (int d = threadIdx.x; d < hd; d += blockDim.x) {
        float a = 0.f, e = 0.f;
        for (int i = 0; i < kWarps; ++i) { a += su[i][d]; e += sw[i][d]; }
        store_float(d_q + int64_t(blockIdx.x) * hd + d, scale * (a - sum * e));
    }
    if (threadIdx.x == 0) D[blockIdx.x] = sum;
}

// Gradients of the newest key and value: a warp for each (sequence, KV head).
template <typename T>
__global__ void __launch_bounds__(32) kv8_attn_newest_simple(tlb_kv8 c, Kv8Pages pg, int n_heads, float scale,
                                                             const T *__restrict__ q, const float *__restrict__ lse,
                                                             const T *__restrict__ d_ctx, const float *__restrict__ D,
                                                             T *__restrict__ d_k, T *__restrict__ d_v) {
    const int64_t b = blockIdx.x / c.n_kv_heads;
    const int kvh = int(blockIdx.x - b * c.n_kv_heads), hd = c.head_dim, group = n_heads / c.n_kv_heads;
    const int lane = threadIdx.x, len = kv8_length(pg, b);
    const int64_t slot = len > 0 ? kv8_slot(pg, c.n_slots, b, len - 1) : -1;
    float dk[kDims] = {}, dv[kDims] = {};
    if (slot >= 0) {
        float k[kDims], v[kDims];
        load_row(c.k, (slot * c.n_kv_heads + kvh) * hd, hd, lane, k);
        load_row(c.v, (slot * c.n_kv_heads + kvh) * hd, hd, lane, v);
        const float sk = c.k_scale[int64_t(kvh) * c.n_slots + slot], sv = c.v_scale[int64_t(kvh) * c.n_slots + slot];
        for (int e = 0; e < group; ++e) {
            const int64_t row = b * n_heads + kvh * group + e;
            float x[kDims], g[kDims];
#pragma unroll
            for (int i = 0; i < kDims; ++i) {
                x[i] = lane + 32 * i < hd ? load_float(q + row * hd + lane + 32 * i) * scale : 0.f;
                g[i] = lane + 32 * i < hd ? load_float(d_ctx + row * hd + lane + 32 * i) : 0.f;
            }
            const float p = expf(dot(x, k) * sk - lse[row]), ds = p * (dot(g, v) * sv - D[row]);
#pragma unroll
            for (int i = 0; i < kDims; ++i) {
                dk[i] = fmaf(ds, x[i], dk[i]);
                dv[i] = fmaf(p, g[i], dv[i]);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < kDims; ++i)
        if (lane + 32 * i < hd) {
            store_float(d_k + int64_t(blockIdx.x) * hd + lane + 32 * i, dk[i]);
            store_float(d_v + int64_t(blockIdx.x) * hd + lane + 32 * i, dv[i]);
        }
}

bool sizes_ok(const tlb_kv8 *c, int64_t n_seq, int32_t n_heads, int64_t max_len) {
    return c != nullptr && n_seq >= 0 && max_len >= 0 && max_len <= (int64_t(1) << 30) && n_heads >= 1 && c->n_kv_heads >= 1 &&
           n_heads % c->n_kv_heads == 0 && n_heads <= 65535 && n_seq <= (int64_t(1) << 30) / n_heads && c->head_dim >= 1 &&
           c->head_dim % 16 == 0 && c->head_dim <= 256;
}

size_t ws_bytes_of(const tlb_kv8 *c, int64_t n_seq, int32_t n_heads, int64_t max_len, bool grad) {
    if (!sizes_ok(c, n_seq, n_heads, max_len)) return 0;
    WsPlan p;
    if (grad) p.take(size_t(n_seq) * n_heads * 4);
    return p.off;
}

// Checks that both calls share; fills pg.
int check_call(const char *what, const tlb_kv8 *cache, const int32_t *pages, int64_t max_pages, int32_t page,
               const int32_t *lengths, int64_t n_seq, int64_t max_len, int32_t n_heads, float scale, int32_t type,
               const void *q, const void *ws, size_t ws_bytes, bool grad, Kv8Pages &pg) {
    TLB_TRY(kv8_check(cache, what));
    TLB_REQUIRE(type == TLB_W_F32 || type == TLB_W_BF16, TLB_EINVAL, "%s: type %d is neither f32 nor bf16", what, type);
    TLB_REQUIRE(n_seq >= 0 && max_len >= 0 && max_pages >= 0, TLB_EINVAL, "%s: negative size", what);
    TLB_REQUIRE(page >= 1, TLB_EINVAL, "%s: page must be at least 1", what);
    TLB_REQUIRE(n_heads >= 1 && n_heads % cache->n_kv_heads == 0, TLB_EINVAL, "%s: n_heads %d is not a multiple of n_kv_heads %d",
                what, n_heads, cache->n_kv_heads);
    TLB_REQUIRE(std::isfinite(scale), TLB_EINVAL, "%s: scale is not finite", what);
    TLB_REQUIRE(sizes_ok(cache, n_seq, n_heads, max_len), TLB_EUNSUPPORTED, "%s: n_seq, n_heads or max_len is too large", what);
    if (n_seq == 0) return TLB_OK;
    TLB_REQUIRE(lengths && q && (pages || max_pages == 0), TLB_EINVAL, "%s: null pointer", what);
    TLB_REQUIRE(aligned16(q), TLB_EINVAL, "%s: q must be 16-byte aligned", what);
    const size_t need = ws_bytes_of(cache, n_seq, n_heads, max_len, grad);
    TLB_REQUIRE(ws != nullptr && ws_bytes >= need, TLB_EINVAL, "%s: workspace of %zu bytes is smaller than the %zu bytes needed",
                what, ws_bytes, need);
    TLB_REQUIRE((reinterpret_cast<uintptr_t>(ws) & 255) == 0, TLB_EINVAL, "%s: workspace must be 256-byte aligned", what);
    int64_t most = max_len;
    if (max_pages < (int64_t(1) << 31)) most = most < max_pages * page ? most : max_pages * page;
    pg = Kv8Pages{pages, lengths, max_pages, page, int32_t(most)};
    return TLB_OK;
}

}  // namespace

}  // namespace tlb

using namespace tlb;

extern "C" {

size_t tlb_kv8_attn_workspace_bytes(const tlb_kv8 *cache, int64_t n_seq, int32_t n_heads, int64_t max_len, int32_t grad) {
    return ws_bytes_of(cache, n_seq, n_heads, max_len, grad != 0);
}

int tlb_kv8_attn_forward(const tlb_kv8 *cache, const int32_t *pages, int64_t max_pages, int32_t page,
                         const int32_t *lengths, int64_t n_seq, int64_t max_len, int32_t n_heads, float scale, int32_t type,
                         const void *q, void *ctx, float *lse, void *ws, size_t ws_bytes, void *stream) {
    clear_error();
    Kv8Pages pg;
    TLB_TRY(check_call("kv8_attn_forward", cache, pages, max_pages, page, lengths, n_seq, max_len, n_heads, scale, type, q, ws,
                       ws_bytes, false, pg));
    if (n_seq == 0) return TLB_OK;
    TLB_REQUIRE(ctx && lse, TLB_EINVAL, "kv8_attn_forward: null pointer");
    TLB_REQUIRE(aligned16(ctx), TLB_EINVAL, "kv8_attn_forward: ctx must be 16-byte aligned");
    cudaStream_t st = as_stream(stream);
    const unsigned grid = unsigned(n_seq * n_heads);
    if (type == TLB_W_F32)
        kv8_attn_forward_simple<<<grid, kWarps * 32, 0, st>>>(*cache, pg, n_heads, scale, static_cast<const float *>(q),
                                                              static_cast<float *>(ctx), lse);
    else
        kv8_attn_forward_simple<<<grid, kWarps * 32, 0, st>>>(*cache, pg, n_heads, scale, static_cast<const __nv_bfloat16 *>(q),
                                                              static_cast<__nv_bfloat16 *>(ctx), lse);
    return check_launch("kv8_attn_forward");
}

int tlb_kv8_attn_backward(const tlb_kv8 *cache, const int32_t *pages, int64_t max_pages, int32_t page,
                          const int32_t *lengths, int64_t n_seq, int64_t max_len, int32_t n_heads, float scale, int32_t type,
                          const void *q, const float *lse, const void *d_ctx, void *d_q, void *d_k, void *d_v, void *ws,
                          size_t ws_bytes, void *stream) {
    clear_error();
    Kv8Pages pg;
    TLB_TRY(check_call("kv8_attn_backward", cache, pages, max_pages, page, lengths, n_seq, max_len, n_heads, scale, type, q, ws,
                       ws_bytes, true, pg));
    if (n_seq == 0) return TLB_OK;
    TLB_REQUIRE(lse && d_ctx && d_q && d_k && d_v, TLB_EINVAL, "kv8_attn_backward: null pointer");
    TLB_REQUIRE(aligned16(d_ctx) && aligned16(d_q) && aligned16(d_k) && aligned16(d_v), TLB_EINVAL,
                "kv8_attn_backward: d_ctx, d_q, d_k and d_v must be 16-byte aligned");
    cudaStream_t st = as_stream(stream);
    float *D = ws_at<float>(ws, kStatusBytes);
    auto run = [&](auto t) {
        using T = decltype(t);
        kv8_attn_backward_simple<T><<<unsigned(n_seq * n_heads), kWarps * 32, 0, st>>>(
            *cache, pg, n_heads, scale, static_cast<const T *>(q), lse, static_cast<const T *>(d_ctx), static_cast<T *>(d_q), D);
        const int rc = check_launch("kv8_attn_backward");
        if (rc != TLB_OK) return rc;
        kv8_attn_newest_simple<T><<<unsigned(n_seq * cache->n_kv_heads), 32, 0, st>>>(
            *cache, pg, n_heads, scale, static_cast<const T *>(q), lse, static_cast<const T *>(d_ctx), D, static_cast<T *>(d_k),
            static_cast<T *>(d_v));
        return check_launch("kv8_attn_newest");
    };
    return type == TLB_W_F32 ? run(float()) : run(__nv_bfloat16());
}

}  // extern "C"
