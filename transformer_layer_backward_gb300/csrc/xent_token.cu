// Cross entropy of a linear head for up to four rows (single tokens), and its gradient, in one
// pass over the head.
//
// With so few rows everything is bound by the read of W: 2 V D bytes in bf16.  The tensor-core
// route reads W twice for a gradient (z, then dz W); here a block of head rows is staged
// once in shared memory (bulk copies, one contiguous run of rows each), taken into registers,
// and used for both z and dz W (and the block's rows of d_w), so W crosses once.  All
// arithmetic is fp32: z, the softmax and dz are never rounded to fewer bits.
//
// One CTA of 16 warps an SM, two of 8 or four of 4.  A thread owns the same column pairs of every
// head row: its part of the hidden rows and of d_hidden stays in registers.  Per block of 8 head
// rows (4 of float32):
//   the thread's W values into registers; its share of the 8 N dot products
//   warp sums by exchange (a lane ends with one of the 8 N values), 16 warps' sums in shared
//   memory, one barrier: the slot is free for the copy of a later block, and every warp
//   adds the 16 sums up
//   loss: warp 0 keeps a running maximum and sum per lane; gradient: dz, passed round by
//   shuffles, times the W values still in registers
// A CTA's statistics, or its part of d_hidden, are joined in CTA order by a second kernel.
//
// Measured: one token, 32768 x 2560 bf16 (168 MB, 24.7 us of reading at the copy rate): loss 28 us
// (70 % of DRAM's time busy; 33 us with the join), gradient 31 us (63 %; 37 us with the sum).  The
// first blocks' way from DRAM and the last CTA's end are the rest.
#include <algorithm>
#include <cstring>

#include "async.cuh"
#include "common.cuh"
#include "kernels.cuh"

namespace tlb {

namespace {

constexpr int kMaxStages = 6;
constexpr float kLog2e = 1.4426950408889634f;

struct TokenParams {
    const void *hidden, *w;
    int hidden_f32;
    const int64_t *targets;
    int64_t vocab;
    int D, stages;
    int n;                       // hidden rows: N, or fewer for N = 4
    // loss
    float2 *part;                // (max, sum) [CTA][ld_part]
    int64_t ld_part;
    float *zt;
    // gradient
    const float *lse, *dloss;
    float *partial;              // [CTA][n][D, made even]
    void *dw;                    // [V, D] in hidden's type, or null
    int dw_add;                  // add to it (float32)
    uint32_t *status;
};

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Head rows of one block: 16 D bytes of either type, so that every block starts and ends on
// a multiple of 16 bytes whatever D is.
template <bool W32> constexpr int block_rows() { return W32 ? 4 : 8; }

// A column pair of a head row.
template <bool W32> struct Pair { uint32_t v; };
template <> struct Pair<true> { float2 v; };
template <bool W32>
__device__ __forceinline__ float2 unpack(const Pair<W32> &p) {
    if constexpr (W32) return p.v;
    else return make_float2(bf16_lo(p.v), bf16_hi(p.v));
}

// Pairs of columns a thread's registers hold: of the hidden rows, and for the gradient of
// d_hidden's rows and of a block of head rows too.
// (A round that no column needs costs as much: 256 threads with 6 take 45 us for 2560, with 5 38.)
constexpr int rounds(int64_t N, bool grad, int threads) { return N == 1 && threads == 512 ? 6 : N <= 2 || !grad ? 5 : 3; }

// Sums of the first CNT values over the warp: each exchange halves the values that a lane holds,
// then plain sums, so that s[0] of lane l is the sum of value l >> (5 - log2 CNT).
template <int CNT, int OFF>
__device__ __forceinline__ void warp_sums(float *s, int lane) {
    if constexpr (CNT > 1) {
        const bool up = lane & OFF;
#pragma unroll
        for (int k = 0; k < CNT / 2; ++k) {
            float x0 = s[k], x1 = s[k + CNT / 2];
            asm("" : "+f"(x0), "+f"(x1));                   // values, not places, are chosen: s stays in registers
            s[k] = (up ? x1 : x0) + __shfl_xor_sync(0xffffffffu, up ? x0 : x1, OFF);
        }
    } else {
        s[0] += __shfl_xor_sync(0xffffffffu, s[0], OFF);
    }
    if constexpr (OFF > 1) warp_sums<(CNT > 1 ? CNT / 2 : 1), OFF / 2>(s, lane);
}

// TH threads: 512, one CTA an SM, or 256 or 128, two or four CTAs, which wait at barriers of
// their own: as few threads as hold the columns in R pairs each.
template <int TH, int N, bool W32, bool GRAD>
__global__ void __launch_bounds__(TH, 512 / TH) xent_token_kernel(const __grid_constant__ TokenParams p) {
    constexpr int kThreads = TH, kWarps = TH / 32, R = rounds(N, GRAD, TH);
    constexpr int VB = block_rows<W32>(), NV = VB * N;
    constexpr int SH = NV == 32 ? 0 : NV == 16 ? 1 : NV == 8 ? 2 : 3;      // lane >> SH: the lane's value
    static_assert((NV << SH) == 32, "values a warp reduces");
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ uint64_t full[kMaxStages];
    __shared__ float red[2][kWarps][NV];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int D = p.D, stages = p.stages;
    const bool odd = D & 1;                                 // pairs start at odd elements: loads by element
    const int64_t blocks = (p.vocab + VB - 1) / VB, nfull = p.vocab / VB;  // the last may be short
    const uint32_t bytes = 16u * uint32_t(D);
    const char *w = static_cast<const char *>(p.w);

    if (tid == 0) {
        for (int s = 0; s < stages; ++s) mbar_init(&full[s], 1);
    }
    fence_mbar_init();
    __syncthreads();
    // block number i of this CTA into slot i % stages; a short last block is not staged
    auto fetch = [&](int i) {
        const int64_t b = blockIdx.x + int64_t(i) * gridDim.x;
        if (b >= nfull) return;
        mbar_arrive_expect_tx(&full[i % stages], bytes);
        tma_load_1d(smem + size_t(i % stages) * bytes, w + b * bytes, bytes, &full[i % stages]);
    };
    if (tid == 0)
        for (int i = 0; i < stages; ++i) fetch(i);
    pdl_trigger();                                          // the kernel that joins the parts may be scheduled

    // the lane's value: head row vr of the block, hidden row vn
    const int vi = lane >> SH, vn = vi % N, vr = vi / N;
    const int64_t t = vn < p.n ? p.targets[vn] : -1;
    const bool has = t >= 0 && t < p.vocab;
    float lse = 0.f, g = 0.f;
    if constexpr (GRAD) {
        lse = has ? p.lse[vn] : 0.f;
        g = has ? p.dloss[vn] : 0.f;
    }
    float2 h[N][R], acc[N][R];
#pragma unroll
    for (int n = 0; n < N; ++n) {
        // d_w takes nothing from rows without a target
        const int64_t tn = n < p.n ? p.targets[n] : -1;
        const bool on = n < p.n && (!GRAD || (tn >= 0 && tn < p.vocab));
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int c = 2 * (tid + r * kThreads);
            h[n][r] = acc[n][r] = make_float2(0.f, 0.f);
            if (c < D && on) {
                const int64_t e = int64_t(n) * D + c;
                if (odd) {
                    h[n][r].x = p.hidden_f32 ? static_cast<const float *>(p.hidden)[e] : __bfloat162float(static_cast<const __nv_bfloat16 *>(p.hidden)[e]);
                    if (c + 1 < D)
                        h[n][r].y = p.hidden_f32 ? static_cast<const float *>(p.hidden)[e + 1]
                                                 : __bfloat162float(static_cast<const __nv_bfloat16 *>(p.hidden)[e + 1]);
                } else if (p.hidden_f32) {
                    h[n][r] = *reinterpret_cast<const float2 *>(static_cast<const float *>(p.hidden) + e);
                } else {
                    const uint32_t v = *reinterpret_cast<const uint32_t *>(static_cast<const __nv_bfloat16 *>(p.hidden) + e);
                    h[n][r] = make_float2(bf16_lo(v), bf16_hi(v));
                }
            }
        }
    }
    // x[v][r]: this thread's pairs of the first `rows` head rows at src
    auto take = [&](const void *src, int rows, Pair<W32> (&x)[VB][R]) {
        if (!odd) {
#pragma unroll
            for (int v = 0; v < VB; ++v)
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    const int c = 2 * (tid + r * kThreads);
                    x[v][r] = {};
                    if (c < D && v < rows)
                        x[v][r] = *reinterpret_cast<const Pair<W32> *>(static_cast<const char *>(src) + (size_t(v) * D + c) * (W32 ? 4 : 2));
                }
            return;
        }
#pragma unroll
        for (int v = 0; v < VB; ++v)
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const int c = 2 * (tid + r * kThreads);
                x[v][r] = {};
                if (c >= D || v >= rows) continue;
                if constexpr (W32) {
                    const float *q = static_cast<const float *>(src) + size_t(v) * D + c;
                    x[v][r].v.x = q[0];
                    if (c + 1 < D) x[v][r].v.y = q[1];
                } else {
                    const uint16_t *q = static_cast<const uint16_t *>(src) + size_t(v) * D + c;
                    x[v][r].v = q[0];
                    if (c + 1 < D) x[v][r].v |= uint32_t(q[1]) << 16;
                }
            }
    };
    float m = -INFINITY, sum = 0.f;
    bool ok = true;
    int i = 0;
    for (int64_t b = blockIdx.x; b < blocks; b += gridDim.x, ++i) {
        const bool staged = b < nfull;
        const int rows = staged ? VB : int(p.vocab - b * VB);
        Pair<W32> x[VB][R];
        if (staged) {
            ok = mbar_wait(&full[i % stages], (i / stages) & 1, p.status, 30u);
            take(smem + size_t(i % stages) * bytes, VB, x);
        } else {
            take(w + b * bytes, rows, x);
        }
        float s[NV];
#pragma unroll
        for (int v = 0; v < VB; ++v)
#pragma unroll
            for (int n = 0; n < N; ++n) {
                float a = 0.f;
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    const float2 u = unpack<W32>(x[v][r]);
                    a = fmaf(u.x, h[n][r].x, fmaf(u.y, h[n][r].y, a));
                }
                s[v * N + n] = a;
            }
        warp_sums<NV, 16>(s, lane);
        if ((lane & ((1 << SH) - 1)) == 0) red[i & 1][warp][vi] = s[0];
        if (__syncthreads_or(!ok)) {                        // a copy did not arrive: leave together
            ok = false;
            break;
        }
        if (tid == 0) fetch(i + stages);                    // the slot has been read by all
        if (!GRAD && warp != 0) continue;
        float z = 0.f;
#pragma unroll
        for (int k = 0; k < kWarps; ++k) z += red[i & 1][k][vi];
        const int64_t row = b * VB + vr;
        if constexpr (!GRAD) {
            if (vr < rows) {
                const float mn = fmaxf(m, z), ref = mn == -INFINITY ? 0.f : mn;
                sum = sum * ex2((m - ref) * kLog2e) + ex2((z - ref) * kLog2e);
                m = mn;
                if (row == t && (lane & ((1 << SH) - 1)) == 0) p.zt[vn] = z;
            }
        } else {
            float dz = ex2((z - lse) * kLog2e);
            if (__any_sync(0xffffffffu, row == t))
                dz = row == t ? exp_minus_1(z - lse) : dz;       // p - 1, exact also where p is near 1
            dz = has && vr < rows ? dz * g : 0.f;
#pragma unroll
            for (int v = 0; v < VB; ++v) {
                float d[N];
#pragma unroll
                for (int n = 0; n < N; ++n) d[n] = __shfl_sync(0xffffffffu, dz, (v * N + n) << SH);
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    const float2 u = unpack<W32>(x[v][r]);
#pragma unroll
                    for (int n = 0; n < N; ++n) {
                        acc[n][r].x = fmaf(d[n], u.x, acc[n][r].x);
                        acc[n][r].y = fmaf(d[n], u.y, acc[n][r].y);
                    }
                }
                if (p.dw != nullptr && v < rows) {
#pragma unroll
                    for (int r = 0; r < R; ++r) {
                        const int c = 2 * (tid + r * kThreads);
                        if (c >= D) continue;
                        float2 o = make_float2(0.f, 0.f);
#pragma unroll
                        for (int n = 0; n < N; ++n) {
                            o.x = fmaf(d[n], h[n][r].x, o.x);
                            o.y = fmaf(d[n], h[n][r].y, o.y);
                        }
                        const int64_t e = (b * VB + v) * D + c;
                        if (p.hidden_f32) {
                            float *q = static_cast<float *>(p.dw) + e;
                            if (p.dw_add) {
                                o.x += q[0];
                                if (c + 1 < D) o.y += q[1];
                            }
                            if (odd) {
                                q[0] = o.x;
                                if (c + 1 < D) q[1] = o.y;
                            } else {
                                *reinterpret_cast<float2 *>(q) = o;
                            }
                        } else if (odd) {
                            __nv_bfloat16 *q = static_cast<__nv_bfloat16 *>(p.dw) + e;
                            q[0] = __float2bfloat16(o.x);
                            if (c + 1 < D) q[1] = __float2bfloat16(o.y);
                        } else {
                            const __nv_bfloat162 q = __floats2bfloat162_rn(o.x, o.y);
                            *reinterpret_cast<__nv_bfloat162 *>(static_cast<__nv_bfloat16 *>(p.dw) + e) = q;
                        }
                    }
                }
            }
        }
    }
    if (!ok) {                                              // what is still in flight lands first (bounded)
        if (tid == 0)
            for (int k = i; k < i + stages; ++k)
                if (blockIdx.x + int64_t(k) * gridDim.x < nfull) mbar_wait(&full[k % stages], (k / stages) & 1, nullptr, 0u);
        __syncthreads();
        return;
    }
    if constexpr (!GRAD) {
        if (warp == 0) {
            // lanes of one hidden row: value bits above log2(N)
#pragma unroll
            for (int off = 16; off > 0; off /= 2) {
                if ((off >> SH) != 0 && (off >> SH) < N) continue;       // that bit tells hidden rows apart
                if ((off >> SH) == 0) continue;                          // copies of the same value
                const float om = __shfl_xor_sync(0xffffffffu, m, off), os = __shfl_xor_sync(0xffffffffu, sum, off);
                const float mn = fmaxf(m, om), ref = mn == -INFINITY ? 0.f : mn;
                sum = sum * ex2((m - ref) * kLog2e) + os * ex2((om - ref) * kLog2e);
                m = mn;
            }
            if (vr == 0 && vn < p.n && (lane & ((1 << SH) - 1)) == 0)
                p.part[int64_t(blockIdx.x) * p.ld_part + vn] = make_float2(m, sum);
        }
    } else {
#pragma unroll
        for (int n = 0; n < N; ++n)
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const int c = 2 * (tid + r * kThreads);
                if (c < D && n < p.n)
                    *reinterpret_cast<float2 *>(p.partial + (int64_t(blockIdx.x) * p.n + n) * (D + (D & 1)) + c) = acc[n][r];
            }
    }
}

// d_hidden: the CTAs' parts added up, 32 elements x 32 threads a block, in a fixed order.
__global__ void __launch_bounds__(1024) xent_token_sum_kernel(const float *__restrict__ partial, int parts, int rows, int D,
                                                              float *out32, __nv_bfloat16 *out16) {
    __shared__ float sh[32][33];
    const int x = threadIdx.x & 31, y = threadIdx.x >> 5, e = blockIdx.x * 32 + x;
    const int ld = D + (D & 1), n = rows * D, row = e / D, step = rows * ld;
    const float *src = partial + row * ld + (e - row * D);
    pdl_wait();
    float s = 0.f;
    for (int k = y; k < parts && e < n; k += 256) {
        float v[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) v[u] = k + 32 * u < parts ? src[int64_t(k + 32 * u) * step] : 0.f;
#pragma unroll
        for (int u = 0; u < 8; ++u) s += v[u];
    }
    sh[y][x] = s;
    __syncthreads();
    s = warp_sum(sh[x][y]);                                 // a warp an element
    const int o = blockIdx.x * 32 + y;
    if (x == 0 && o < n) {
        if (out32 != nullptr) out32[o] = s;
        else out16[o] = __float2bfloat16(s);
    }
}

template <int TH, int N, bool W32, bool GRAD>
int launch(TokenParams &p, int grid, cudaStream_t st) {
    constexpr int room = (TH == 512 ? 220 : TH == 256 ? 108 : 52) * 1024;
    p.stages = std::min(kMaxStages, room / (16 * p.D));
    const int smem = p.stages * 16 * p.D;
    auto k = xent_token_kernel<TH, N, W32, GRAD>;
    TLB_CUDA(cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, room));
    k<<<grid, TH, smem, st>>>(p);
    return check_launch(GRAD ? "xent_token_grad" : "xent_token_loss");
}

// Threads of a CTA for N rows of length D; 0: too long.  The smallest CTA whose registers hold the
// rows, and 512 / threads of them an SM: the warps of a CTA wait for one another at every block
// of head rows (the gradient of one token over 32768 x 2560 takes 43 us with one CTA of 512
// threads an SM, 30 us with two of 256).
int token_threads(int64_t N, int64_t D, bool grad) {
    for (int th = 128; th <= 512; th *= 2)
        if (D <= int64_t(2) * th * rounds(N, grad, th)) return th;
    return 0;
}

template <int N, bool W32, bool GRAD>
int by_threads(TokenParams &p, int th, int grid, cudaStream_t st) {
    return th == 128 ? launch<128, N, W32, GRAD>(p, grid, st) : th == 256 ? launch<256, N, W32, GRAD>(p, grid, st)
                                                                          : launch<512, N, W32, GRAD>(p, grid, st);
}

// Up to 4 CTAs an SM, each with a block of head rows at least.
int token_grid(int wtype, int th, int64_t vocab) {
    return int(std::min<int64_t>(512 / th * num_sms(), ceil_div(vocab, wtype == TLB_W_F32 ? 4 : 8)));
}

template <bool W32, bool GRAD>
int by_rows(TokenParams &p, int th, int grid, cudaStream_t st) {
    return p.n == 1 ? by_threads<1, W32, GRAD>(p, th, grid, st) : p.n == 2 ? by_threads<2, W32, GRAD>(p, th, grid, st)
                                                                           : by_threads<4, W32, GRAD>(p, th, grid, st);
}

}  // namespace

bool xent_token_supported(int64_t N, int64_t D, bool grad) { return N >= 1 && N <= 4 && token_threads(N, D, grad) > 0; }

int xent_token_loss(int htype, const void *hidden, int wtype, const void *W, const int64_t *targets, int64_t N, int64_t V,
                    int64_t D, float2 *part, int64_t ld_part, float *zt, uint32_t *status, int *slots, cudaStream_t st) {
    TokenParams p;
    memset(&p, 0, sizeof(p));
    p.hidden = hidden;
    p.w = W;
    p.hidden_f32 = htype == TLB_W_F32;
    p.targets = targets;
    p.vocab = V;
    p.D = int(D);
    p.n = int(N);
    p.part = part;
    p.ld_part = ld_part;
    p.zt = zt;
    p.status = status;
    const int th = token_threads(N, D, false);
    *slots = token_grid(wtype, th, V);
    return wtype == TLB_W_F32 ? by_rows<true, false>(p, th, *slots, st) : by_rows<false, false>(p, th, *slots, st);
}

int xent_token_grad(int htype, const void *hidden, int wtype, const void *W, const int64_t *targets, const float *lse,
                    const float *d_loss, int64_t N, int64_t V, int64_t D, void *d_hidden, void *d_w, float *partial,
                    uint32_t *status, bool dw_add, cudaStream_t st) {
    TokenParams p;
    memset(&p, 0, sizeof(p));
    p.hidden = hidden;
    p.w = W;
    p.hidden_f32 = htype == TLB_W_F32;
    p.targets = targets;
    p.vocab = V;
    p.D = int(D);
    p.n = int(N);
    p.lse = lse;
    p.dloss = d_loss;
    p.partial = partial;
    p.dw = d_w;
    p.dw_add = dw_add;
    p.status = status;
    const int th = token_threads(N, D, true), grid = token_grid(wtype, th, V), n = int(N * D);
    TLB_TRY((wtype == TLB_W_F32 ? by_rows<true, true>(p, th, grid, st) : by_rows<false, true>(p, th, grid, st)));
    TLB_CUDA(launch_dependent(xent_token_sum_kernel, dim3(unsigned(ceil_div(n, 32))), dim3(1024), 0, st, partial, grid, int(N), int(D),
                              htype == TLB_W_F32 ? static_cast<float *>(d_hidden) : nullptr,
                              htype == TLB_W_F32 ? nullptr : static_cast<__nv_bfloat16 *>(d_hidden)));
    return check_launch("xent_token_sum");
}

}  // namespace tlb
