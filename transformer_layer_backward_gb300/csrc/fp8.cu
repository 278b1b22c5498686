// Quantising float matrices to e4m3 in blocks of 128 columns.
#include "common.cuh"
#include "fp8.cuh"

namespace tlb {

namespace {

// Eight consecutive elements.
__device__ __forceinline__ void load_float8(const float *p, float (&v)[8]) {
    const float4 a = load_float4(p), b = load_float4(p + 4);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}
__device__ __forceinline__ void load_float8(const __nv_bfloat16 *p, float (&v)[8]) {
    const uint4 a = ld_stream_u4(p);
    v[0] = bf16_lo(a.x); v[1] = bf16_hi(a.x); v[2] = bf16_lo(a.y); v[3] = bf16_hi(a.y);
    v[4] = bf16_lo(a.z); v[5] = bf16_hi(a.z); v[6] = bf16_lo(a.w); v[7] = bf16_hi(a.w);
}

// Blocks of 1 x 128: a warp takes kRowBlocks blocks at a time, whose loads are all issued before the
// first is used; a lane holds four columns of each.  Bound by memory: 5 (float32) or 3 bytes a value.
// 2048 x 9728 float32: 17.7 us, 5.7 TB/s; 2048 x 9727 (an element at a time): 23.4 us.
constexpr int kRowBlocks = 4;

template <typename T, bool VEC>
__global__ void __launch_bounds__(256) quantize_rows_kernel(const T *__restrict__ x, int64_t cols, int64_t nblk,
                                                            int64_t items, uint8_t *__restrict__ q,
                                                            float *__restrict__ scales) {
    const int lane = threadIdx.x & 31;
    const int64_t warps = int64_t(gridDim.x) * (blockDim.x >> 5);
    for (int64_t i0 = (int64_t(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5)) * kRowBlocks; i0 < items;
         i0 += warps * kRowBlocks) {
        float v[kRowBlocks][4];
        int64_t at[kRowBlocks];             // element of this lane's first column
        int left[kRowBlocks];               // columns of the block, 0 past the last
#pragma unroll
        for (int u = 0; u < kRowBlocks; ++u) {
            const int64_t i = i0 + u;
            const int64_t row = cols == nblk * kFp8Block ? 0 : i / nblk;   // whole blocks: i * 128 is the place
            const int64_t blk = i - row * nblk;
            at[u] = row * cols + blk * kFp8Block;
            left[u] = i < items ? int(min(int64_t(kFp8Block), cols == nblk * kFp8Block ? kFp8Block : cols - blk * kFp8Block)) : 0;
            if (VEC) {                      // a lane's four columns are there or not (cols % 4 == 0)
                const float4 f = lane * 4 < left[u] ? load_float4(x + at[u] + lane * 4) : make_float4(0.f, 0.f, 0.f, 0.f);
                v[u][0] = f.x; v[u][1] = f.y; v[u][2] = f.z; v[u][3] = f.w;
            } else {
#pragma unroll
                for (int k = 0; k < 4; ++k) v[u][k] = lane + 32 * k < left[u] ? load_float(x + at[u] + lane + 32 * k) : 0.f;
            }
        }
#pragma unroll
        for (int u = 0; u < kRowBlocks; ++u) {
            uint32_t top = 0;
#pragma unroll
            for (int k = 0; k < 4; ++k) top = max(top, magnitude(v[u][k]));
            top = __reduce_max_sync(0xffffffffu, top);
            float inv;
            const float s = block_scale(top, inv);
            const uint32_t y = to_e4m3x4(v[u][0] * inv, v[u][1] * inv, v[u][2] * inv, v[u][3] * inv);
            if (VEC) {
                if (lane * 4 < left[u]) *reinterpret_cast<uint32_t *>(q + at[u] + lane * 4) = y;
            } else {
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if (lane + 32 * k < left[u]) q[at[u] + lane + 32 * k] = uint8_t(y >> (8 * k));
            }
            if (lane == 0 && left[u] > 0) scales[i0 + u] = s;
        }
    }
}

// The same with 16 lanes a block and eight columns a lane, for bf16 (16 bytes loaded a lane, 8 stored): a warp takes
// kRowPairs pairs of blocks at a time.  The maximum is taken of the 16-bit magnitudes, two at a time.  4096 x 9728:
// 20.8 us, 5.8 TB/s (four columns a lane, 8-byte loads: 61 us; the maximum of floats by shuffles: 29 us).
constexpr int kRowPairs = 4;

__global__ void __launch_bounds__(256, 4) quantize_rows8_kernel(const __nv_bfloat16 *__restrict__ x, int64_t cols, int64_t nblk,
                                                                int64_t items, uint8_t *__restrict__ q,
                                                                float *__restrict__ scales) {
    const int lane = threadIdx.x & 31, part = lane & 15;
    const bool upper = lane >= 16;
    const int64_t warps = int64_t(gridDim.x) * (blockDim.x >> 5);
    for (int64_t i0 = (int64_t(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5)) * (2 * kRowPairs); i0 < items;
         i0 += warps * (2 * kRowPairs)) {
        uint4 v[kRowPairs];
        int64_t at[kRowPairs];
        bool there[kRowPairs];
#pragma unroll
        for (int u = 0; u < kRowPairs; ++u) {
            const int64_t i = i0 + 2 * u + (upper ? 1 : 0);
            const int64_t row = cols == nblk * kFp8Block ? 0 : i / nblk;
            const int64_t blk = i - row * nblk;
            at[u] = row * cols + blk * kFp8Block + part * 8;
            there[u] = i < items && (cols == nblk * kFp8Block || blk * kFp8Block + part * 8 < cols);
            v[u] = there[u] ? ld_stream_u4(x + at[u]) : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int u = 0; u < kRowPairs; ++u) {
            const uint32_t two = __vmaxu2(__vmaxu2(v[u].x & 0x7FFF7FFFu, v[u].y & 0x7FFF7FFFu),
                                          __vmaxu2(v[u].z & 0x7FFF7FFFu, v[u].w & 0x7FFF7FFFu));
            const uint32_t mine = max(two & 0xFFFFu, two >> 16) << 16;            // as float bits
            const uint32_t lo = __reduce_max_sync(0xffffffffu, upper ? 0u : mine), hi = __reduce_max_sync(0xffffffffu, upper ? mine : 0u);
            float inv;
            const float s = block_scale(upper ? hi : lo, inv);
            if (there[u]) {
                *reinterpret_cast<uint2 *>(q + at[u]) =
                    make_uint2(to_e4m3x4(bf16_lo(v[u].x) * inv, bf16_hi(v[u].x) * inv, bf16_lo(v[u].y) * inv, bf16_hi(v[u].y) * inv),
                               to_e4m3x4(bf16_lo(v[u].z) * inv, bf16_hi(v[u].z) * inv, bf16_lo(v[u].w) * inv, bf16_hi(v[u].w) * inv));
                if (part == 0) scales[i0 + 2 * u + (upper ? 1 : 0)] = s;
            }
        }
    }
}

// Blocks of 128 x 128: a CTA of 512 threads holds one in registers, 32 values a thread, 16 lanes a row (16 bytes of bf16
// loaded a lane and 8 stored).  2560 x 9728 bf16: 13.9 us, 5.4 TB/s, float32 18.5 us, 6.7 TB/s; 256 threads with 8-byte
// loads took 49 us (bf16).  2560 x 9727 bf16 (an element at a time): 42.6 us.
constexpr int kTileThreads = 512, kTileRows = kFp8Block * 16 / kTileThreads;   // rows a thread

template <typename T, bool VEC>
__global__ void __launch_bounds__(kTileThreads) quantize_tiles_kernel(const T *__restrict__ x, int64_t rows, int64_t cols,
                                                                      int nblk, uint8_t *__restrict__ q,
                                                                      float *__restrict__ scales) {
    __shared__ uint32_t tops[kTileThreads / 32];
    const int64_t r0 = int64_t(blockIdx.x / unsigned(nblk)) * kFp8Block, c0 = int64_t(blockIdx.x % unsigned(nblk)) * kFp8Block;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, row = threadIdx.x >> 4, part = threadIdx.x & 15;
    const int nc = int(min(int64_t(kFp8Block), cols - c0)), nr = int(min(int64_t(kFp8Block), rows - r0));
    const int64_t at = (r0 + row) * cols + c0;
    float v[kTileRows][8];
    uint32_t top = 0;
#pragma unroll
    for (int u = 0; u < kTileRows; ++u) {
        const T *p = x + at + u * (kTileThreads / 16) * cols;
        const bool there = row + u * (kTileThreads / 16) < nr;
        if (VEC) {
            if (there && part * 8 < nc) {
                load_float8(p + part * 8, v[u]);
            } else {
#pragma unroll
                for (int k = 0; k < 8; ++k) v[u][k] = 0.f;
            }
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k) v[u][k] = there && part + 16 * k < nc ? load_float(p + part + 16 * k) : 0.f;
        }
    }
#pragma unroll
    for (int u = 0; u < kTileRows; ++u)
#pragma unroll
        for (int k = 0; k < 8; ++k) top = max(top, magnitude(v[u][k]));
    top = __reduce_max_sync(0xffffffffu, top);
    if (lane == 0) tops[warp] = top;
    __syncthreads();
    top = __reduce_max_sync(0xffffffffu, tops[lane & 15]);
    float inv;
    const float s = block_scale(top, inv);
    if (threadIdx.x == 0) scales[blockIdx.x] = s;
#pragma unroll
    for (int u = 0; u < kTileRows; ++u) {
        if (row + u * (kTileThreads / 16) >= nr) break;
        uint8_t *p = q + at + u * (kTileThreads / 16) * cols;
        const uint32_t lo = to_e4m3x4(v[u][0] * inv, v[u][1] * inv, v[u][2] * inv, v[u][3] * inv);
        const uint32_t hi = to_e4m3x4(v[u][4] * inv, v[u][5] * inv, v[u][6] * inv, v[u][7] * inv);
        if (VEC) {
            if (part * 8 < nc) *reinterpret_cast<uint2 *>(p + part * 8) = make_uint2(lo, hi);
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (part + 16 * k < nc) p[part + 16 * k] = uint8_t((k < 4 ? lo : hi) >> (8 * (k & 3)));
        }
    }
}

template <typename T>
int quantize_launch(const T *x, int64_t rows, int64_t cols, int block_rows, uint8_t *q, float *scales, cudaStream_t st) {
    const int64_t nblk = ceil_div(cols, kFp8Block);
    // four columns a lane: every row starts where four elements may be loaded and four bytes stored
    const bool vec = cols % 4 == 0 && (reinterpret_cast<uintptr_t>(x) % (4 * sizeof(T))) == 0 &&
                     (reinterpret_cast<uintptr_t>(q) & 3) == 0;
    if (block_rows == 1) {
        const int64_t items = rows * nblk;
        if constexpr (sizeof(T) == 2)
            if (cols % 8 == 0 && aligned16(x) && (reinterpret_cast<uintptr_t>(q) & 7) == 0) {
                quantize_rows8_kernel<<<stream_grid(ceil_div(items, 2 * kRowPairs) * 32, 256), 256, 0, st>>>(x, cols, nblk, items, q,
                                                                                                         scales);
                return check_launch("fp8_quantize_rows");
            }
        const unsigned grid = stream_grid(ceil_div(items, kRowBlocks) * 32, 256);
        if (vec) quantize_rows_kernel<T, true><<<grid, 256, 0, st>>>(x, cols, nblk, items, q, scales);
        else quantize_rows_kernel<T, false><<<grid, 256, 0, st>>>(x, cols, nblk, items, q, scales);
        return check_launch("fp8_quantize_rows");
    }
    const int64_t tiles = ceil_div(rows, kFp8Block) * nblk;
    TLB_REQUIRE(tiles < (int64_t(1) << 31), TLB_EUNSUPPORTED, "fp8_quantize: more than 2^31 blocks of 128 x 128");
    // eight columns a thread: 16 bytes loaded, 8 stored
    const bool vec8 = cols % 8 == 0 && aligned16(x) && (reinterpret_cast<uintptr_t>(q) & 7) == 0;
    if (vec8) quantize_tiles_kernel<T, true><<<unsigned(tiles), kTileThreads, 0, st>>>(x, rows, cols, int(nblk), q, scales);
    else quantize_tiles_kernel<T, false><<<unsigned(tiles), kTileThreads, 0, st>>>(x, rows, cols, int(nblk), q, scales);
    return check_launch("fp8_quantize_tiles");
}

}  // namespace

}  // namespace tlb

using namespace tlb;

extern "C" {

int tlb_fp8_quantize(int32_t type, const void *x, int64_t rows, int64_t cols, int32_t block_rows, uint8_t *q,
                     float *scales, void *stream) {
    clear_error();
    TLB_REQUIRE(type == TLB_W_F32 || type == TLB_W_BF16, TLB_EINVAL, "fp8_quantize: type %d is neither f32 nor bf16", type);
    TLB_REQUIRE(block_rows == 1 || block_rows == kFp8Block, TLB_EINVAL, "fp8_quantize: block_rows must be 1 or 128");
    TLB_REQUIRE(rows >= 0 && cols >= 0, TLB_EINVAL, "fp8_quantize: negative size");
    TLB_REQUIRE(rows <= (int64_t(1) << 40) && cols <= (int64_t(1) << 40) && (rows == 0 || cols <= (int64_t(1) << 48) / rows),
                TLB_EUNSUPPORTED, "fp8_quantize: more than 2^48 values");
    if (rows == 0 || cols == 0) return TLB_OK;
    TLB_REQUIRE(x && q && scales, TLB_EINVAL, "fp8_quantize: null pointer");
    TLB_REQUIRE((reinterpret_cast<uintptr_t>(x) & (type == TLB_W_F32 ? 3 : 1)) == 0 &&
                    (reinterpret_cast<uintptr_t>(scales) & 3) == 0,
                TLB_EINVAL, "fp8_quantize: x and scales must be aligned to their elements");
    if (type == TLB_W_F32)
        return quantize_launch(static_cast<const float *>(x), rows, cols, block_rows, q, scales, as_stream(stream));
    return quantize_launch(static_cast<const __nv_bfloat16 *>(x), rows, cols, block_rows, q, scales, as_stream(stream));
}

}  // extern "C"
