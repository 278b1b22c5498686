// The transposed-weight product of operands in 8-bit blocks:
//   dX[s, i] (+)= sum_kb dy_scales[s, kb] w_scales[i / 128, kb] sum_{o in block kb} dY[s, o] W[i, o]
#include "common.cuh"
#include "fp8.cuh"

namespace tlb {

namespace {

constexpr int kTile = 16;

// One output a thread, 16 x 16 outputs a CTA, 16 columns of both operands in shared memory.
template <typename T>
__global__ void __launch_bounds__(kTile *kTile) linear_fp8_simple_kernel(
    const uint8_t *__restrict__ W, const float *__restrict__ ws, const uint8_t *__restrict__ dY, const float *__restrict__ ys,
    int64_t S, int64_t out, int64_t in, T *__restrict__ dX, int accumulate) {
    __shared__ float a[kTile][kTile + 1], b[kTile][kTile + 1];
    const int64_t nblk = (out + kFp8Block - 1) / kFp8Block;
    const int tx = threadIdx.x % kTile, ty = threadIdx.x / kTile;
    const int64_t i0 = int64_t(blockIdx.x) * kTile, s0 = int64_t(blockIdx.y) * kTile;
    float sum = 0.f;
    for (int64_t kb = 0; kb < nblk; ++kb) {
        float part = 0.f;
        for (int64_t o = kb * kFp8Block; o < min(out, (kb + 1) * kFp8Block); o += kTile) {
            const bool in_k = o + tx < out;
            a[ty][tx] = in_k && s0 + ty < S ? e4m3x2_to_float2(dY[(s0 + ty) * out + o + tx]).x : 0.f;
            b[ty][tx] = in_k && i0 + ty < in ? e4m3x2_to_float2(W[(i0 + ty) * out + o + tx]).x : 0.f;
            __syncthreads();
#pragma unroll
            for (int k = 0; k < kTile; ++k) part = fmaf(a[ty][k], b[tx][k], part);
            __syncthreads();
        }
        if (s0 + ty < S && i0 + tx < in)
            sum = fmaf(part, ys[(s0 + ty) * nblk + kb] * ws[(i0 + tx) / kFp8Block * nblk + kb], sum);
    }
    if (s0 + ty < S && i0 + tx < in) {
        T *p = dX + (s0 + ty) * in + i0 + tx;
        store_float(p, accumulate ? float(*p) + sum : sum);
    }
}

}  // namespace

}  // namespace tlb

using namespace tlb;

extern "C" {

size_t tlb_linear_fp8_workspace_bytes(int64_t S, int64_t out_dim, int64_t in_dim) {
    const int64_t most = int64_t(1) << 24;
    if (S < 0 || out_dim < 0 || in_dim < 0 || S > most || out_dim > most || in_dim > most) return 0;
    return kStatusBytes;
}

int tlb_linear_fp8_backward(const uint8_t *W, const float *w_scales, const uint8_t *dY, const float *dy_scales, int64_t S,
                            int64_t out_dim, int64_t in_dim, int32_t type, void *dX, int32_t accumulate, void *ws,
                            size_t ws_bytes, void *stream) {
    clear_error();
    const int64_t most = int64_t(1) << 24;
    TLB_REQUIRE(type == TLB_W_F32 || type == TLB_W_BF16, TLB_EINVAL, "linear_fp8_backward: type %d is neither f32 nor bf16", type);
    TLB_REQUIRE(S >= 0 && out_dim >= 0 && in_dim >= 0, TLB_EINVAL, "linear_fp8_backward: negative size");
    TLB_REQUIRE(S <= most && out_dim <= most && in_dim <= most, TLB_EUNSUPPORTED, "linear_fp8_backward: a size past 2^24");
    if (S == 0 || in_dim == 0) return TLB_OK;
    TLB_REQUIRE(dX && (out_dim == 0 || (W && w_scales && dY && dy_scales)), TLB_EINVAL, "linear_fp8_backward: null pointer");
    TLB_REQUIRE(aligned16(W) && aligned16(dY) && aligned16(dX), TLB_EINVAL,
                "linear_fp8_backward: W, dY and dX must be 16-byte aligned");
    const size_t need = tlb_linear_fp8_workspace_bytes(S, out_dim, in_dim);
    TLB_REQUIRE(ws != nullptr && ws_bytes >= need, TLB_EINVAL,
                "linear_fp8_backward: workspace of %zu bytes is smaller than the %zu bytes needed", ws_bytes, need);
    TLB_REQUIRE((reinterpret_cast<uintptr_t>(ws) & 255) == 0, TLB_EINVAL, "linear_fp8_backward: workspace must be 256-byte aligned");
    cudaStream_t st = as_stream(stream);
    const dim3 grid(unsigned(ceil_div(in_dim, kTile)), unsigned(ceil_div(S, kTile)));
    TLB_REQUIRE(grid.y <= 65535, TLB_EUNSUPPORTED, "linear_fp8_backward: too many rows");
    if (type == TLB_W_F32)
        linear_fp8_simple_kernel<<<grid, kTile * kTile, 0, st>>>(W, w_scales, dY, dy_scales, S, out_dim, in_dim,
                                                                 static_cast<float *>(dX), accumulate);
    else
        linear_fp8_simple_kernel<<<grid, kTile * kTile, 0, st>>>(W, w_scales, dY, dy_scales, S, out_dim, in_dim,
                                                                 static_cast<__nv_bfloat16 *>(dX), accumulate);
    return check_launch("linear_fp8_simple");
}

}  // extern "C"
