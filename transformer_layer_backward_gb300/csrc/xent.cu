// Softmax cross entropy of a linear head, and its gradient, without the logits in memory:
//   z[i, v] = <hidden[i], W[v]>,  lse[i] = log sum_v exp z[i, v],  loss[i] = lse[i] - z[i, t_i]
//   dz[i, v] = d_loss[i] (exp(z[i, v] - lse[i]) - [v = t_i])
//   d_hidden = dz W,  d_w = dz^T hidden
// with hidden [N, D] (token rows), W [V, D] (one row per vocabulary entry) and t_i a column
// of [0, V) or outside it (no target: loss 0, dz = 0).
//
// Every product runs on one tcgen05 kernel.  Its modes differ in what becomes of an
// accumulator tile (rows x columns of z or of a gradient):
//   kStats  maximum and sum of exponentials of each row over the tile's columns; the logits
//           never leave tensor memory.  A second kernel joins the tiles' pairs in a fixed order.
//   kGrad   dz of the tile, rounded to bf16, by TMA into a piece of the vocabulary's dz
//           [N, piece] in the workspace
//   kOut    d_hidden (+)= dz W over one piece, or d_w of the piece: fp32 sums, stream-K
// Operands of either order: a K-major operand has the summed index along its rows (hidden
// and W in z), an MN-major one across them (W in dz W, dz and hidden in dz^T hidden); both
// are staged by TMA with 128-byte swizzle, so nothing is transposed in memory.
//
// Float32 operands are taken apart into three bf16 terms of 8 bits each, x = x0 + x1 + x2
// exactly, and the product is the sum of the term products down to 2^-24 of the first: three
// with a bf16 partner (exact), six between two float32 operands (x_i y_j with i + j <= 2).  The
// terms are written to the workspace, or (a float32 head, up to 512 rows) made from the float32
// values on their way into shared memory.
// With bf16 operands dz is rounded to bf16 once (2^-8 at most, relative to each dz; the sums
// of it are in fp32).  What the target's dz, the largest of most rows, loses there is kept
// aside in fp32, and the epilogues of both gradients add it back, times the target's row of the
// head to the row's d_hidden, times the hidden row to the target's row of d_w (summed before over the
// rows with that target): so the gradients' error stays near that of their own rounding to bf16.
//
// The tensor core cuts its fp32 sum after every MMA of 16 products (measured: a sum of 160
// MMAs comes out about 1.2e-6 of its size short, one of 6144 3e-5).  Results of float32
// precision are therefore summed in chunks of a few k blocks, which the epilogue adds up in
// registers.  The term products of a k block follow one another, so that its operand tiles
// come from memory once and from L2 then.
//
// The logit of a row's own target decides how exact the loss and p - 1 of a confident row are
// (1 - p may be 1e-3 of p): a kernel of its own sums it in fp32 on the CUDA cores, and both
// epilogues put it in the place of the accumulator's.
//
// Up to 64 bf16 rows give too few roundings of dz to even out (one row's largest dz alone sets
// its error), and the read of W hides a second product: dz is kept in two terms there.
//
// Bounds: N >= 512 rows is bound by the tensor pipe (2 N V D flops a product), few rows by
// the read of W.  Measured at 2048 x 2560 x 131072 in bf16 (727 us a product at the rate of a large
// library product, 1.89 PFLOP/s): loss 769 us, dz 793 us, dz W 798 us each alone, 1.72 to 1.79
// PFLOP/s; 863 and 1766 us for the calls back to back, where the power limit sets the clock.  4096 x
// 2560 x 65536 with d_w: 2.71 ms (2.18).  Float32 rows, 512 x 2560 x 32768: 391 us (273: three
// products), at 2048 x 2560 x 131072 2.23 ms the loss (2.18) and 5.30 ms d_hidden (4.36).
#include <cuda.h>

#include <algorithm>
#include <cstdint>
#include <cstring>
#include <type_traits>

#include "async.cuh"
#include "common.cuh"
#include "kernels.cuh"
#include "tc.cuh"

namespace tlb {

namespace {

constexpr int kBM = 128, kBK = 64;          // rows of a CTA's tile; k block (64 bf16 = 128 bytes)
constexpr int kThreads = 320;               // 10 warps: TMA producer, MMA issuer, 8 epilogue warps
constexpr int kConvWarps = 8;               // ... and those that take a float32 operand apart
constexpr int kConvThreads = kThreads + 32 * kConvWarps;
constexpr int kEpiWarps = 8;                // two per 32 TMEM lanes (rows), each half of the columns
constexpr int kMaxTerms = 3, kMaxProd = 6;
// k blocks (4 MMAs each) of one tensor-memory sum of a float32 result, of z and of a gradient.
// Reading a sum out takes the tensor pipe about 300 cycles (the loss of 2048 x 2560 x 131072, before its
// rows' targets were fetched a tile ahead: 812 us at 8 k blocks, 787 at 20, and 769 since; 512 float32
// rows' gradient 400 us with z in tens, 388), and its error grows with its length.
constexpr int kChunkLoss = 20, kChunkGrad = 10;
constexpr int kConvLoss = 3, kConvGrad = 2;  // of six term products each
constexpr int kGroupM = 16;                 // row tiles that share a column tile before the next one
constexpr int kBox = 4096;                  // bytes of a 32 x 64 bf16 box of dz
constexpr float kLog2e = 1.4426950408889634f;

enum Mode { kStats = 0, kGrad = 1, kOut = 2 };

struct XParams {
    CUtensorMap a[kMaxTerms], b[kMaxTerms];  // operand terms
    CUtensorMap d[kMaxTerms];                // kGrad: dz terms [rows, piece], boxes of 64 x 32
    int nprod;                               // the product is the sum of a[pa[i]] b[pb[i]]
    int8_t pa[kMaxProd + 2], pb[kMaxProd + 2];
    int kb;                                  // k blocks of one term product
    int M, N;                                // rows and columns of the result
    int tiles_m, tiles_n;
    int units;                               // CTAs (pairs): unit u does the whole tiles u, u + units, ...
    int whole;                               // ... below `whole`, then its share of the other tiles'
    int64_t sk_work;                         // k blocks (kOut: split evenly over sk_units units)
    int sk_units;
    // kStats, kGrad
    const int64_t *targets;
    int64_t vocab, v0;                       // columns in all, first column of this piece
    float2 *part;                            // kStats: (max, sum) [slot0 + 2 tile_n + half][ld_part]
    int64_t ld_part;
    const float *zt;                         // logit of each row's target, from xent_target_kernel
    const float *lse, *dloss;                // kGrad
    // kOut
    // What dz of the targets has lost.  d_hidden (more): rest[i] x row targets[i] of the head (rows ld_more
    // apart) is added to row i.  d_w (sums): row first[v] of sums, the sum of rest[i] x hidden row i over
    // the rows with target v, to row v where first[v + 1] > first[v]
    const float *rest;
    const __nv_bfloat16 *more;
    int64_t ld_more;                         // of sums too
    const float *sums;
    const int *first;
    const float *acc;                        // sum of the earlier pieces [M, N], or null
    float *out32;                            // one of the two is written
    __nv_bfloat16 *out16;
    int vec;                                 // N % 4 == 0 and 16-byte rows: four columns an access
    const float *bw;                         // CONV: columns' operand, float32 [b_rows, b_cols], rows b_cols apart
    int b_rows, b_cols, b_vec;               // b_vec: four columns an access
    float *partial;                          // [CTA][2][kBM][BN]
    uint32_t *status;
};

__host__ __device__ __forceinline__ int64_t sk_start(int64_t work, int units, int c) { return work * c / units; }

// Result tile number t: groups of kGroupM row tiles, inside a group the row tiles of one
// column tile first.  The CTAs that run together so share a few column tiles of one operand
// and 16 row tiles of the other (21 MB of 2560-wide rows), which stay in L2.
// (Fewer than 2^31 tiles: 2^24 rows by 2^20 columns at most.)
__device__ __forceinline__ void tile_of(const XParams &p, uint32_t t, int &m, int &n) {
    const uint32_t group = uint32_t(kGroupM) * p.tiles_n, g = t / group, r = t - g * group;
    const uint32_t rows = min(kGroupM, p.tiles_m - int(g) * kGroupM), c = r / rows;
    n = int(c);
    m = int(g * kGroupM + (r - c * rows));
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Shared-memory descriptor of an MN-major tile written by TMA boxes of 64 (MN) x kBK (K)
// with 128-byte swizzle: 128-byte rows, one per k; 8-row groups along k are 1024 bytes apart
// (stride offset), blocks of 64 along MN one box (leading offset).
__device__ __forceinline__ uint64_t sw128_desc_mn(const void *p) {
    uint64_t d = (uint64_t(smem_u32(p)) >> 4) & 0x3FFFull;
    d |= uint64_t((kBK * 128) >> 4) << 16;
    d |= uint64_t(1024 >> 4) << 32;
    d |= uint64_t(1) << 46;
    d |= uint64_t(2) << 61;
    return d;
}

__device__ __forceinline__ void tma_store_2d(const CUtensorMap *map, const void *src, int x, int y) {
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(x), "r"(y), "r"(smem_u32(src))
                 : "memory");
}
__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
__device__ __forceinline__ void bulk_wait_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
__device__ __forceinline__ void bulk_wait_all() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

// The next bf16 term of x: its 8 highest significant bits (cut, so that three terms hold
// all 24 exactly), removed from x.  Infinities and NaN go whole into the first term.
__device__ __forceinline__ uint32_t next_term(float &x) {
    const uint32_t u = __float_as_uint(x);
    if ((u & 0x7F800000u) == 0x7F800000u) {
        x = 0.f;
        return (u >> 16) | ((u & 0x007FFFFFu) ? 0x40u : 0u);
    }
    x -= __uint_as_float(u & 0xFFFF0000u);
    return u >> 16;
}

// ---------------------------------------------------------------- epilogues of a warp

// Columns [col0, col0 + BN / 2) of this thread's row, in registers: z[j] is column col0 + j.

// kStats: maximum and sum of exponentials, with the target's logit as p.zt has it.
template <int BN>
__device__ __forceinline__ void stats_row(const XParams &p, float (&z)[BN / 2], int row, int col0, int slot) {
    const int64_t t = row < p.M ? p.targets[row] : -1;
    const int tc = (t >= p.v0 && t < p.v0 + p.N && t < p.vocab) ? int(t - p.v0) - col0 : -1;
    if (col0 + BN / 2 > p.N) {
#pragma unroll
        for (int c = 0; c < BN / 2; ++c)
            if (col0 + c >= p.N) z[c] = -INFINITY;
    }
    if (tc >= 0 && tc < BN / 2) {
        const float zt = p.zt[row];
        int k = tc;
        asm("" : "+r"(k));                                 // compared, never an index: z stays in registers
#pragma unroll
        for (int c = 0; c < BN / 2; ++c)
            if (c == k) z[c] = zt;
    }
    float m[4] = {z[0], z[1], z[2], z[3]};
#pragma unroll
    for (int c = 4; c < BN / 2; ++c) m[c & 3] = fmaxf(m[c & 3], z[c]);
    const float mx = fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]));
    // nothing but -inf (columns past the last): exponents against 0 give sums of 0.  The maximum's own
    // exponent is 0 exactly (a product mx log2(e) that is rounded before the difference leaves up to half
    // a step of it: the lse of a certain row a step below its largest logit, its loss below 0)
    const float ref = mx == -INFINITY ? 0.f : mx;
    float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int c = 0; c < BN / 2; ++c) sum[c & 3] += ex2((z[c] - ref) * kLog2e);
    if (row < p.M) p.part[int64_t(slot) * p.ld_part + row] = make_float2(mx, (sum[0] + sum[1]) + (sum[2] + sum[3]));
}

// kGrad: what dz needs of this thread's row; fetched a tile ahead.
struct GradRow {
    int64_t t;
    float lse, g, zt;
};
__device__ __forceinline__ GradRow grad_row(const XParams &p, int row) {
    GradRow r{-1, 0.f, 0.f, 0.f};
    if (row < p.M) r = GradRow{p.targets[row], p.lse[row], p.dloss[row], p.zt[row]};
    return r;
}

// kGrad: dz of this warp's 32 rows row0.. and columns col0 .. col0 + 63, from z in y: term by
// term through the warp's 4 KB box and out by TMA, which leaves out
// what lies past the last row or column.
template <int TERMS>
__device__ __forceinline__ void grad_box(const XParams &p, const GradRow &r, float *y, int row0, int col0, uint8_t *box,
                                         int lane) {
    if (row0 >= p.M || col0 >= p.N) return;
    const bool has = r.t >= 0 && r.t < p.vocab;
#pragma unroll
    for (int c = 0; c < 64; ++c) y[c] = ex2((y[c] - r.lse) * kLog2e);
    const int64_t tc = has ? r.t - p.v0 - col0 : -1;       // the target's column in this box
    if (tc >= 0 && tc < min(64, p.N - col0)) {
        int k = int(tc);
        asm("" : "+r"(k));                                 // compared, never an index: y stays in registers
        const float pt1 = exp_minus_1(r.zt - r.lse);            // p - 1 of the target, exact also where p is near 1
#pragma unroll
        for (int c = 0; c < 64; ++c)
            if (c == k) y[c] = pt1;
    }
#pragma unroll
    for (int c = 0; c < 64; ++c) y[c] = has ? y[c] * r.g : 0.f;
#pragma unroll
    for (int k = 0; k < TERMS; ++k) {
        if (lane == 0) bulk_wait_read();                   // the box's last store has read it
        __syncwarp();
#pragma unroll
        for (int c = 0; c < 8; ++c) {
            uint4 w;
            if constexpr (TERMS == 1) {
                const uint2 lo = pack_bf16x4(y[8 * c], y[8 * c + 1], y[8 * c + 2], y[8 * c + 3]);
                const uint2 hi = pack_bf16x4(y[8 * c + 4], y[8 * c + 5], y[8 * c + 6], y[8 * c + 7]);
                w = make_uint4(lo.x, lo.y, hi.x, hi.y);
            } else {
                // the 8 highest significant bits, cut; what is left goes on to the next term
                uint32_t u[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    u[i] = __float_as_uint(y[8 * c + i]);
                    y[8 * c + i] -= __uint_as_float(u[i] & 0xFFFF0000u);
                }
                w = make_uint4(__byte_perm(u[0], u[1], 0x7632), __byte_perm(u[2], u[3], 0x7632),
                               __byte_perm(u[4], u[5], 0x7632), __byte_perm(u[6], u[7], 0x7632));
            }
            *reinterpret_cast<uint4 *>(box + lane * 128 + ((c ^ (lane & 7)) << 4)) = w;
        }
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) {
            tma_store_2d(&p.d[k], box, col0, row0);
            bulk_commit();
        }
    }
}

// Four columns col.. of one row of a result: the earlier pieces' sum is added, the value
// stored in the result's type.
__device__ __forceinline__ void store4(const XParams &p, int row, int col, float (&v)[4]) {
    const int64_t e = int64_t(row) * p.N + col;
    if (p.vec) {
        float4 y = make_float4(v[0], v[1], v[2], v[3]);
        if (p.acc != nullptr) {
            const float4 c = *reinterpret_cast<const float4 *>(p.acc + e);
            y.x += c.x; y.y += c.y; y.z += c.z; y.w += c.w;
        }
        if (p.out32 != nullptr) *reinterpret_cast<float4 *>(p.out32 + e) = y;
        else *reinterpret_cast<uint2 *>(p.out16 + e) = pack_bf16x4(y.x, y.y, y.z, y.w);
        return;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (col + i >= p.N) break;
        const float y = v[i] + (p.acc != nullptr ? p.acc[e + i] : 0.f);
        if (p.out32 != nullptr) p.out32[e + i] = y;
        else p.out16[e + i] = __float2bfloat16(y);
    }
}

// kOut: what the targets' dz have lost, in d_hidden (kTargets) and d_w (kSums).
enum More { kNone = 0, kTargets = 1, kSums = 2 };
// ... for this thread's row of a tile; fetched a tile ahead.
struct MoreRow {
    int64_t row;                                           // of `more` or `sums`, or -1
    float rest;
};
// (the lines of columns col .. col + cols of that row are asked for in L2)
template <int MORE>
__device__ __forceinline__ MoreRow more_row(const XParams &p, int row, int col, int cols) {
    MoreRow r{-1, 0.f};
    if (row >= p.M) return r;
    if constexpr (MORE == kSums) {
        const int at = p.first[row];
        if (at < p.first[row + 1]) r.row = at;
    } else {
        const int64_t t = p.targets[row];
        if (t >= 0 && t < p.vocab) r.row = t;
        r.rest = p.rest[row];
    }
    if (r.row >= 0) {
        constexpr int kLine = MORE == kSums ? 32 : 64;
        const int64_t e = r.row * p.ld_more;
        for (int c = col; c < min(col + cols, p.N); c += kLine) {
            if constexpr (MORE == kSums) asm volatile("prefetch.global.L2 [%0];" ::"l"(p.sums + e + c));
            else asm volatile("prefetch.global.L2 [%0];" ::"l"(p.more + e + c));
        }
    }
    return r;
}
// Columns col .. col + 31 of that row, fetched before the tensor memory is read (d_hidden: where the
// head's rows are whole 16 bytes), and added to the thread's row.
template <int MORE> struct MoreCols {
    uint4 w[MORE == kSums ? 8 : MORE == kTargets ? 4 : 1];
};
template <int MORE>
__device__ __forceinline__ void fetch_more(const XParams &p, const MoreRow &r, MoreCols<MORE> &q, int col) {
    constexpr int C = MORE == kSums ? 4 : 8;
    const bool on = r.row >= 0 && (MORE == kSums || p.ld_more % 8 == 0);
    const int64_t e = r.row * p.ld_more + col;
#pragma unroll
    for (int k = 0; k < 32 / C; ++k) {
        const void *src = MORE == kSums ? static_cast<const void *>(p.sums + e + C * k) : p.more + e + C * k;
        q.w[k] = on && col + C * k < p.N ? *static_cast<const uint4 *>(src) : make_uint4(0, 0, 0, 0);
    }
}
template <int MORE>
__device__ __forceinline__ void add_more(const XParams &p, const MoreRow &r, const MoreCols<MORE> &q, float *y, int col) {
    if (r.row < 0) return;
    if constexpr (MORE == kSums) {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            y[4 * k] += __uint_as_float(q.w[k].x);
            y[4 * k + 1] += __uint_as_float(q.w[k].y);
            y[4 * k + 2] += __uint_as_float(q.w[k].z);
            y[4 * k + 3] += __uint_as_float(q.w[k].w);
        }
    } else if (p.ld_more % 8 == 0) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const uint32_t u[4] = {q.w[k].x, q.w[k].y, q.w[k].z, q.w[k].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                y[8 * k + 2 * i] = fmaf(r.rest, bf16_lo(u[i]), y[8 * k + 2 * i]);
                y[8 * k + 2 * i + 1] = fmaf(r.rest, bf16_hi(u[i]), y[8 * k + 2 * i + 1]);
            }
        }
    } else {
        const __nv_bfloat16 *src = p.more + r.row * p.ld_more + col;
#pragma unroll
        for (int k = 0; k < 32; ++k)
            if (col + k < p.N) y[k] = fmaf(r.rest, __bfloat162float(src[k]), y[k]);
    }
}
// The same for four columns col.. of one row (col % 4 == 0).
template <int MORE>
__device__ __forceinline__ void add_more4(const XParams &p, int row, int col, float (&v)[4]) {
    if constexpr (MORE == kSums) {
        const int at = p.first[row];
        if (at >= p.first[row + 1]) return;
        const float4 c = *reinterpret_cast<const float4 *>(p.sums + at * p.ld_more + col);
        v[0] += c.x; v[1] += c.y; v[2] += c.z; v[3] += c.w;
    } else {
        const int64_t t = p.targets[row];
        if (t < 0 || t >= p.vocab) return;
        const float f = p.rest[row];
        const __nv_bfloat16 *src = p.more + t * p.ld_more + col;
        if (p.ld_more % 4 == 0) {
            const uint2 w = *reinterpret_cast<const uint2 *>(src);
            v[0] = fmaf(f, bf16_lo(w.x), v[0]);
            v[1] = fmaf(f, bf16_hi(w.x), v[1]);
            v[2] = fmaf(f, bf16_lo(w.y), v[2]);
            v[3] = fmaf(f, bf16_hi(w.y), v[3]);
        } else {
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (col + k < p.N) v[k] = fmaf(f, __bfloat162float(src[k]), v[k]);
        }
    }
}

// kOut: columns col0 .. col0 + 31 of a warp's 32 rows row0.. (one row a thread), turned in
// shared memory so that lanes run along the columns (8 column quads x 4 rows an access):
// into the result, or into a partial tile (rows of `ld` floats) where there is one.
__device__ __forceinline__ void out_block(const XParams &p, const float *z, int row0, int col0, float *partial, int ld,
                                          float *blk, int lane) {
    if (row0 >= p.M || col0 >= p.N) return;
#pragma unroll
    for (int t = 0; t < 32; ++t) blk[lane * 33 + t] = z[t];
    __syncwarp();
    const int c4 = (lane & 7) * 4, rl = lane >> 3;
#pragma unroll 4
    for (int k = 0; k < 8; ++k) {
        const int r = 4 * k + rl;
        if (row0 + r >= p.M || col0 + c4 >= p.N) continue;
        const float *a = blk + r * 33 + c4;
        if (partial != nullptr) {
            *reinterpret_cast<float4 *>(partial + int64_t(r) * ld + c4) = make_float4(a[0], a[1], a[2], a[3]);
        } else {
            float v[4] = {a[0], a[1], a[2], a[3]};
            store4(p, row0 + r, col0 + c4, v);
        }
    }
    __syncwarp();
}

// ---------------------------------------------------------------- the kernel

template <int BN, bool PAIR>
struct Shape {
    static constexpr int TM = PAIR ? 2 * kBM : kBM;          // rows of a tile of the schedule
    static constexpr int BH = PAIR ? BN / 2 : BN;            // columns' operand rows that a CTA stages
    static constexpr int A_BYTES = kBM * kBK * 2, B_BYTES = BH * kBK * 2, STAGE = A_BYTES + B_BYTES;
};
// Ring depth: what shared memory leaves beside the epilogue's buffers (8 x 4 KB boxes of dz, 8 x
// 4.2 KB for the turn of kOut, none for kStats).
template <int MODE>
constexpr int epi_bytes() {
    return MODE == kStats ? 0 : MODE == kGrad ? kEpiWarps * kBox : kEpiWarps * 32 * 33 * 4;
}
template <int BN, bool PAIR, int MODE, bool CONV>
constexpr int stages_of() {
    const int n = (226 * 1024 - 1024 - epi_bytes<MODE>()) / ((CONV ? 3 : 1) * Shape<BN, PAIR>::STAGE);   // CONV: all terms
    return n > 6 ? 6 : n;
}

// A float32 head's 64 x 64 block in registers, loaded and taken apart by the converting warps.
// vec: two rows of 16 lanes x 4 columns; else a row of 32 lanes x 2 columns.
constexpr int kConvRows = 64 / kConvWarps, kAhead = 2;
template <bool INSIDE>
__device__ __forceinline__ void conv_fetch(const XParams &p, int row0, int col0, int cw, int lane, float (&v)[2 * kConvRows]) {
    if (p.b_vec) {
        const int c = col0 + 4 * (lane & 15), r = row0 + cw * kConvRows + (lane >> 4);
        const float *src = p.bw + int64_t(r) * p.b_cols + c;
#pragma unroll
        for (int u = 0; u < kConvRows / 2; ++u, src += 2 * p.b_cols) {
            float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
            if (INSIDE || (r + 2 * u < p.b_rows && c < p.b_cols)) x = __ldg(reinterpret_cast<const float4 *>(src));
            v[4 * u] = x.x; v[4 * u + 1] = x.y; v[4 * u + 2] = x.z; v[4 * u + 3] = x.w;
        }
    } else {
        const int c = col0 + 2 * lane, r = row0 + cw * kConvRows;
        const float *src = p.bw + int64_t(r) * p.b_cols + c;
#pragma unroll
        for (int u = 0; u < kConvRows; ++u, src += p.b_cols)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                v[2 * u + k] = 0.f;
                if (INSIDE || (r + u < p.b_rows && c + k < p.b_cols)) v[2 * u + k] = __ldg(src + k);
            }
    }
}
__device__ __forceinline__ void conv_load(const XParams &p, int row0, int col0, int cw, int lane, float (&v)[2 * kConvRows]) {
    if (row0 + 64 <= p.b_rows && col0 + 64 <= p.b_cols) conv_fetch<true>(p, row0, col0, cw, lane, v);
    else conv_fetch<false>(p, row0, col0, cw, lane, v);
}
// A k block's lines on their way to L2, a line a thread: 128 x 64 floats, or 64 x 128 (MN).
template <bool B_MN>
__device__ __forceinline__ void conv_prefetch(const XParams &p, int row0, int col0, int t) {
    static_assert(kConvWarps == 8, "256 lines");
    const int r = row0 + (B_MN ? t >> 2 : t >> 1), c = col0 + 32 * (B_MN ? t & 3 : t & 1);
    if (r < p.b_rows && c < p.b_cols) asm volatile("prefetch.global.L2 [%0];" ::"l"(p.bw + int64_t(r) * p.b_cols + c));
}
// Two neighbours' next terms as a word, removed from them.  (Infinities and NaN leave NaN.)
__device__ __forceinline__ uint32_t cut_terms(float &x, float &y) {
    const uint32_t a = __float_as_uint(x), b = __float_as_uint(y);
    x -= __uint_as_float(a & 0xFFFF0000u);
    y -= __uint_as_float(b & 0xFFFF0000u);
    return __byte_perm(a, b, 0x7632);
}
// ... into the three planes `plane` bytes apart (rows of 128 bytes, 128-byte swizzle).
__device__ __forceinline__ void conv_store(bool vec, uint8_t *dst, int plane, int cw, int lane, float (&v)[2 * kConvRows]) {
    if (vec) {
#pragma unroll
        for (int u = 0; u < kConvRows / 2; ++u) {
            const int r = cw * kConvRows + 2 * u + (lane >> 4), c = lane & 15;
            uint8_t *at = dst + r * 128 + (((c >> 1) ^ (r & 7)) << 4) + (c & 1) * 8;
#pragma unroll
            for (int t = 0; t < 3; ++t) {
                uint2 w;
                w.x = cut_terms(v[4 * u], v[4 * u + 1]);
                w.y = cut_terms(v[4 * u + 2], v[4 * u + 3]);
                *reinterpret_cast<uint2 *>(at + t * plane) = w;
            }
        }
    } else {
#pragma unroll
        for (int u = 0; u < kConvRows; ++u) {
            const int r = cw * kConvRows + u;
            uint8_t *at = dst + r * 128 + (((lane >> 2) ^ (r & 7)) << 4) + (lane & 3) * 4;
#pragma unroll
            for (int t = 0; t < 3; ++t) *reinterpret_cast<uint32_t *>(at + t * plane) = cut_terms(v[2 * u], v[2 * u + 1]);
        }
    }
}

// TERMS: bf16 terms of dz (kGrad; 1 otherwise).  FINE: sums in chunks of k blocks.
// CONV: the columns' operand is float32 in memory, and 8 more warps take it apart into the three
// planes of a stage, beside TMA's three of the rows' operand; a k block is then all six term
// products (24 MMAs, 1536 cycles), and two stages fill shared memory.  It is bound by the
// converting warps: their loads (32 KB in flight an SM, asked for in L2 two k blocks before) and
// the cutting, about 2000 cycles a k block.  Loss of 128 rows, 32768 x 2560: 4 warps 176 us, 8
// warps 139 (although the epilogue then spills some registers), with the prefetch 127, without a
// test for infinities 115.  CTA pairs that share a k block's rows: slower (333 rows 488 against
// 300 us).
template <int BN, bool PAIR, int MODE, int TERMS, bool FINE, bool A_MN, bool B_MN, bool CONV, int MORE>
__global__ void __launch_bounds__(CONV ? kConvThreads : kThreads, 1) xent_gemm_kernel(const __grid_constant__ XParams p) {
    using S = Shape<BN, PAIR>;
    static_assert(!CONV || (BN == 128 && !PAIR && FINE && !A_MN), "one form");
    constexpr int kStages = stages_of<BN, PAIR, MODE, CONV>();
    constexpr int TM = S::TM, BH = S::BH, A_BYTES = (CONV ? 3 : 1) * S::A_BYTES, STAGE = (CONV ? 3 : 1) * S::STAGE;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    __shared__ uint64_t full[kStages], empty[kStages], accfull[2], accempty[2], done;
    __shared__ uint32_t tmem_base;
    __shared__ int s_abort, s_issued, s_consumed;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = PAIR ? int(cluster_rank()) : 0;         // this CTA's half of a tile's rows
    const int unit = PAIR ? int(blockIdx.x >> 1) : int(blockIdx.x);
    const bool leader = rank == 0;                           // issues the MMAs

    // this unit's segments: its whole tiles, then its share of the split tiles, cut at tiles
    const int KB = p.nprod * p.kb;
    // k blocks of one accumulator
    const int chunk = !FINE ? KB : MODE != kOut ? (CONV ? kConvLoss : kChunkLoss) : (CONV ? kConvGrad : kChunkGrad);
    const int nwhole = p.whole > unit ? (p.whole - unit + p.units - 1) / p.units : 0;
    const bool splits = MODE == kOut && p.sk_work > 0 && unit < p.sk_units;
    const int b0 = splits ? int(sk_start(p.sk_work, p.sk_units, unit)) : 0;       // sk_work < units KB < 2^31
    const int b1 = splits ? int(sk_start(p.sk_work, p.sk_units, unit + 1)) : 0;
    struct Seg {
        int tile, kb0, kb1, slot;
    };
    // segment i; `at` walks through [b0, b1) after the whole tiles
    auto next_seg = [&](int i, int &at, Seg &s) {
        if (i < nwhole) {
            s.tile = i * p.units + unit;
            s.kb0 = 0;
            s.kb1 = KB;
            s.slot = 0;
        } else {
            if (at >= b1) return false;
            const int tl = at / KB;
            s.kb0 = at - tl * KB;
            s.kb1 = min(KB, b1 - tl * KB);
            s.slot = at == b0 ? 0 : 1;
            at += s.kb1 - s.kb0;
            s.tile = p.whole + tl;
        }
        return true;
    };
    // this CTA's first row, the first column and the column tile of a tile
    auto place = [&](int tile, int &m0, int &n0, int &tn) {
        int m;
        tile_of(p, uint32_t(tile), m, tn);
        m0 = m * TM + rank * kBM;
        n0 = tn * BN;
    };

    // A part of a tile starts at a multiple of the units' share and wraps round, so that the units
    // are at the same k of different tiles at the same time and share its operand tiles in L2
    auto first_kb = [&](int i, const Seg &s) {
        int kb = s.kb0;
        if (splits && i >= nwhole && s.kb1 - s.kb0 == b1 - b0) {
            const int share = int((p.sk_work + p.sk_units - 1) / p.sk_units);
            kb = (s.kb0 + share - 1) / share * share;
            if (kb >= s.kb1) kb = s.kb0;
        }
        return kb;
    };

    if (threadIdx.x == 0) {
        s_abort = 0;
        s_issued = s_consumed = 0;
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&full[s], CONV ? 1 + kConvWarps : 1);
            mbar_init(&empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&accfull[b], 1);
            mbar_init(&accempty[b], (PAIR ? 2 : 1) * kEpiWarps);
        }
        mbar_init(&done, 1);
    }
    if (warp == 1) {
        if constexpr (PAIR) {
            tmem_alloc_pair(&tmem_base, 2 * BN);
            tmem_relinquish_pair();
        } else {
            tmem_alloc(&tmem_base, 2 * BN);
            tmem_relinquish();
        }
    }
    fence_mbar_init();
    tc_fence_before();
    __syncthreads();
    if constexpr (PAIR) cluster_sync();              // the peer's barriers exist before any remote arrive
    tc_fence_after();
    const uint32_t tmem = tmem_base;
    pdl_trigger();                                           // the kernel that joins the parts may be scheduled

    if (warp == 0) {
        // ------------------------------------------------ TMA producer
        if (lane == 0) {
            int g = 0, at = b0;
            bool ok = true;
            Seg sg;
            for (int i = 0; ok && next_seg(i, at, sg); ++i) {
                int m0, n0, tn;
                place(sg.tile, m0, n0, tn);
                const int nb = n0 + rank * BH;
                int kb = first_kb(i, sg);
                for (int j = sg.kb0; j < sg.kb1; ++j, ++g, kb = kb + 1 < sg.kb1 ? kb + 1 : sg.kb0) {
                    const int s = g % kStages;
                    if (g >= kStages && !mbar_wait(&empty[s], ((g / kStages) - 1) & 1, p.status, 20u)) {
                        ok = false;
                        break;
                    }
                    const int kq = kb / p.nprod, prod = kb - kq * p.nprod, k0 = kq * kBK;
                    const CUtensorMap *ma = &p.a[p.pa[prod]], *mb = &p.b[p.pb[prod]];
                    uint8_t *sa = smem + s * STAGE, *sb = sa + A_BYTES;
                    if constexpr (CONV) {
                        mbar_arrive_expect_tx(&full[s], A_BYTES);
                        for (int t = 0; t < 3; ++t) tma_load_2d(sa + t * S::A_BYTES, &p.a[t], k0, m0, &full[s]);
                    } else if constexpr (PAIR) {
                        if (leader) mbar_arrive_expect_tx(&full[s], 2 * STAGE);   // both CTAs' copies
                        const uint32_t fb = cluster_addr(&full[s], 0);
                        if constexpr (A_MN) {
                            for (int c = 0; c < kBM / 64; ++c)
                                tma_load_2d_pair(sa + c * kBK * 128, ma, m0 + c * 64, k0, fb);
                        } else {
                            tma_load_2d_pair(sa, ma, k0, m0, fb);
                        }
                        if constexpr (B_MN) {
                            for (int c = 0; c < BH / 64; ++c)
                                tma_load_2d_pair(sb + c * kBK * 128, mb, nb + c * 64, k0, fb);
                        } else {
                            tma_load_2d_pair(sb, mb, k0, nb, fb);
                        }
                    } else {
                        mbar_arrive_expect_tx(&full[s], STAGE);
                        if constexpr (A_MN) {
                            for (int c = 0; c < kBM / 64; ++c)
                                tma_load_2d(sa + c * kBK * 128, ma, m0 + c * 64, k0, &full[s]);
                        } else {
                            tma_load_2d(sa, ma, k0, m0, &full[s]);
                        }
                        if constexpr (B_MN) {
                            for (int c = 0; c < BH / 64; ++c)
                                tma_load_2d(sb + c * kBK * 128, mb, nb + c * 64, k0, &full[s]);
                        } else {
                            tma_load_2d(sb, mb, k0, nb, &full[s]);
                        }
                    }
                    s_issued = g + 1;
                }
            }
            if (!ok) s_abort = 1;
        }
    } else if (warp == 1) {
        // ------------------------------------------------ MMA issuer, accumulators alternate
        if (lane == 0 && leader) {
            constexpr uint32_t idesc = (1u << 4) | (1u << 7) | (1u << 10) | (A_MN ? 1u << 15 : 0u) |
                                       (B_MN ? 1u << 16 : 0u) | (uint32_t(BN >> 3) << 17) | (uint32_t(TM >> 4) << 24);
            // 16 k: 32 bytes along a K-major row, 16 rows of 128 bytes of an MN-major tile
            constexpr int ka = A_MN ? 128 : 2, kbs = B_MN ? 128 : 2;
            int g = 0, f = 0, at = b0;                       // k blocks, accumulators so far
            bool ok = true;
            Seg sg;
            for (int i = 0; ok && next_seg(i, at, sg); ++i) {
                for (int k0 = sg.kb0; ok && k0 < sg.kb1; k0 += chunk, ++f) {
                    const int b = f & 1, k1 = min(sg.kb1, k0 + chunk);
                    const uint32_t acc = tmem + uint32_t(b * BN);
                    if (f >= 2 && !mbar_wait(&accempty[b], uint32_t(((f >> 1) - 1) & 1), p.status, 23u)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    for (int kb = k0; kb < k1; ++kb, ++g) {
                        const int s = g % kStages;
                        if (!mbar_wait(&full[s], (g / kStages) & 1, p.status, 21u)) { ok = false; break; }
                        tc_fence_after();
                        const uint8_t *sa = smem + s * STAGE;
                        // CONV: the six products of three terms each, the smallest first
#pragma unroll
                        for (int sum = CONV ? 2 : 0; sum >= 0; --sum)
#pragma unroll
                            for (int ta = 0; ta <= sum; ++ta) {
                                const uint8_t *pa = sa + ta * S::A_BYTES, *pb = sa + A_BYTES + (sum - ta) * S::B_BYTES;
                                const uint64_t ad = A_MN ? sw128_desc_mn(pa) : sw128_desc(pa);
                                const uint64_t bd = B_MN ? sw128_desc_mn(pb) : sw128_desc(pb);
#pragma unroll
                                for (int k = 0; k < kBK / 16; ++k) {
                                    const uint32_t add = (kb > k0 || k > 0 || (CONV && !(sum == 2 && ta == 0))) ? 1u : 0u;
                                    if constexpr (PAIR) mma_bf16_pair(acc, ad + ka * k, bd + kbs * k, idesc, add);
                                    else mma_bf16(acc, ad + ka * k, bd + kbs * k, idesc, add);
                                }
                            }
                        if constexpr (PAIR) mma_commit_pair(&empty[s], 3);   // frees the stage in both CTAs
                        else mma_commit(&empty[s]);
                        s_consumed = g + 1;
                    }
                    if (ok) {
                        if constexpr (PAIR) mma_commit_pair(&accfull[b], 3);
                        else mma_commit(&accfull[b]);
                    }
                }
            }
            if (!ok) s_abort = 1;
            if constexpr (PAIR) mma_commit_pair(&done, 1);
            else mma_commit(&done);
            mbar_wait(&done, 0, nullptr, 0u);
        }
    } else if (CONV && warp >= 2 + kEpiWarps) {
        // ------------------------------------------------ float32 operand -> three terms
        if constexpr (CONV) {
            const int cw = warp - 2 - kEpiWarps;
            int i = 0, at = b0, j = 0, kb = 0, m0, n0 = 0, tn;
            Seg sg;
            // k blocks in the producer's order
            auto enter = [&] {
                if (!next_seg(i, at, sg)) return false;
                place(sg.tile, m0, n0, tn);
                kb = first_kb(i, sg);
                j = sg.kb0;
                return true;
            };
            auto step = [&] {
                if (++j < sg.kb1) {
                    kb = kb + 1 < sg.kb1 ? kb + 1 : sg.kb0;
                    return true;
                }
                ++i;
                return enter();
            };
            float v[2][2 * kConvRows];                        // the two halves of the k block that comes next
            auto load = [&](int h) {
                if constexpr (B_MN) conv_load(p, kb * kBK, n0 + 64 * h, cw, lane, v[h]);
                else conv_load(p, n0 + 64 * h, kb * kBK, cw, lane, v[h]);
            };
            bool more = enter();
            if (more) {
                load(0);
                load(1);
            }
            for (int g = 0; more; ++g) {
                const int s = g % kStages;
                if (g >= kStages && !mbar_wait(&empty[s], ((g / kStages) - 1) & 1, p.status, 24u)) {
                    s_abort = 1;
                    break;
                }
                uint8_t *sb = smem + s * STAGE + A_BYTES;
                more = step();
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    conv_store(p.b_vec != 0, sb + h * 64 * 128, S::B_BYTES, cw, lane, v[h]);
                    if (more) load(h);
                    // DRAM takes longer than a k block does: later ones are asked for too
                    if (more && h == 0)
                        conv_prefetch<B_MN>(p, B_MN ? (kb + kAhead) * kBK : n0, B_MN ? n0 : (kb + kAhead) * kBK, cw * 32 + lane);
                }
                fence_proxy_async();
                __syncwarp();
                if (lane == 0) mbar_arrive(&full[s]);
            }
        }
    } else {
        // ------------------------------------------------ epilogue (warps 2..9)
        const int q = warp & 3, half = (warp - 2) >> 2;       // TMEM lane quarter, half of the columns
        // A fine sum is gathered whole in registers; any other stays in tensor memory while it
        // is read a block at a time.
        constexpr int WN = MODE == kGrad ? 64 : 32, ZN = FINE ? BN / 2 : WN;
        uint8_t *buf = smem + kStages * STAGE;
        uint8_t *box = buf + (warp - 2) * kBox;                                        // kGrad
        float *blk = reinterpret_cast<float *>(buf) + (warp - 2) * 32 * 33;            // kOut
        if constexpr (MODE != kOut) pdl_wait();               // the targets' logits, where their kernel comes just before
        int f = 0, at = b0;
        bool ok = true;
        Seg sg, next;
        bool more = next_seg(0, at, next);
        int m0 = 0, n0 = 0, tn = 0;
        GradRow grn{-1, 0.f, 0.f, 0.f};
        MoreRow mrn{-1, 0.f};
        auto enter = [&] {
            place(next.tile, m0, n0, tn);
            if constexpr (MODE == kGrad) grn = grad_row(p, m0 + q * 32 + lane);
            // (to a split tile the kernel that joins its parts adds it)
            if constexpr (MORE != kNone)
                mrn = next.kb0 == 0 && next.kb1 == KB ? more_row<MORE>(p, m0 + q * 32 + lane, n0 + half * (BN / 2), BN / 2)
                                                      : MoreRow{-1, 0.f};
        };
        if (more) enter();
        for (int i = 0; ok && more; ++i) {
            sg = next;
            const int row0 = m0 + q * 32, colh = n0 + half * (BN / 2), tile_n = tn;
            const GradRow gr = grn;
            const MoreRow mr = mrn;
            more = next_seg(i + 1, at, next);
            if (more) enter();
            float *part = nullptr;                            // kOut: this warp's part of a partial tile
            if (MODE == kOut && (sg.kb0 != 0 || sg.kb1 != KB))
                part = p.partial + ((int64_t(blockIdx.x) * 2 + sg.slot) * kBM + q * 32) * BN + half * (BN / 2);
            float z[ZN];                                      // this thread's row
            MoreCols<MORE> cols;
            auto block = [&](float *y, int c0) {              // WN columns from colh + c0
                if constexpr (MODE == kGrad) grad_box<TERMS>(p, gr, y, row0, colh + c0, box, lane);
                if constexpr (MODE == kOut) {
                    if constexpr (MORE != kNone) add_more<MORE>(p, mr, cols, y, colh + c0);
                    out_block(p, y, row0, colh + c0, part != nullptr ? part + c0 : nullptr, BN, blk, lane);
                }
            };
            for (int k0 = sg.kb0; k0 < sg.kb1; k0 += chunk, ++f) {
                const int b = f & 1;
                if (!mbar_wait(&accfull[b], uint32_t((f >> 1) & 1), p.status, 22u)) {
                    s_abort = 1;
                    ok = false;
                    break;
                }
                __syncwarp();                                 // tensor memory is read by whole warps
                tc_fence_after();
                const uint32_t tm = tmem + uint32_t(b * BN + half * (BN / 2)) + (uint32_t(q * 32) << 16);
                if constexpr (FINE) {
#pragma unroll
                    for (int j = 0; j < BN / 64; ++j) {
                        uint32_t v[32];
                        tmem_ld32(tm + uint32_t(j * 32), v);
                        tmem_wait_ld();
#pragma unroll
                        for (int c = 0; c < 32; ++c)
                            z[j * 32 + c] = (k0 > sg.kb0 ? z[j * 32 + c] : 0.f) + __uint_as_float(v[c]);
                    }
                } else {
#pragma unroll 1
                    for (int c0 = 0; c0 < BN / 2; c0 += WN) {
                        uint32_t v[WN / 32][32];
                        if constexpr (MORE != kNone) fetch_more<MORE>(p, mr, cols, colh + c0);
#pragma unroll
                        for (int j = 0; j < WN / 32; ++j) tmem_ld32(tm + uint32_t(c0 + j * 32), v[j]);
                        tmem_wait_ld();
#pragma unroll
                        for (int c = 0; c < WN; ++c) z[c] = __uint_as_float(v[c / 32][c % 32]);
                        block(z, c0);
                        __syncwarp();
                    }
                }
                tc_fence_before();                            // the accumulator is free again
                __syncwarp();
                if (lane == 0) {
                    if constexpr (PAIR) mbar_arrive_cluster(cluster_addr(&accempty[b], 0));
                    else mbar_arrive(&accempty[b]);
                }
            }
            if (!ok) break;
            if constexpr (MODE == kStats) {
                stats_row<BN>(p, z, row0 + lane, colh, 2 * tile_n + half);
            } else if constexpr (FINE) {
#pragma unroll
                for (int c0 = 0; c0 < BN / 2; c0 += WN) block(z + c0, c0);
            }
        }
        if (MODE == kGrad && lane == 0) bulk_wait_all();
    }
    // wind down.  The MMA thread waited for its last commit; after an abort (a wait ran out)
    // the copies that were issued and not consumed are awaited too, and every CTA then stays
    // for 20 us so that its peer's last copies and arrivals land while it lives.
    tc_fence_before();
    __syncthreads();
    if (s_abort && threadIdx.x == 0) {
        if (leader)
            for (int g = s_consumed; g < s_issued; ++g) mbar_wait(&full[g % kStages], (g / kStages) & 1, nullptr, 0u);
        const long long t0 = clock64();
        while (clock64() - t0 < 40000) {}
    }
    __syncthreads();
    if constexpr (PAIR) cluster_sync();
    if (warp == 1) {
        tc_fence_after();
        if constexpr (PAIR) tmem_dealloc_pair(tmem, 2 * BN);
        else tmem_dealloc(tmem, 2 * BN);
    }
}

// Loads in program order, so that a row of them is in flight together.
__device__ __forceinline__ float4 ld_ordered(const float *p) {
    float4 r;
    asm volatile("ld.global.v4.f32 {%0,%1,%2,%3}, [%4];" : "=f"(r.x), "=f"(r.y), "=f"(r.z), "=f"(r.w) : "l"(p) : "memory");
    return r;
}

// A split tile (number whole + blockIdx.x) is the sum, in unit order, of its units' partial
// tiles; block y does fix_rows of its rows.  (A unit's share is less than a tile: none was written by
// one unit.)  U parts are in flight together: 16 where a tile has more than 24 (200 x 512 x 131072, 38
// units a tile: d_hidden 95 us, 101 with 8), else 8 (128 x 2560 x 32768, 15 units: 79 us, 81 with 16).
template <int BN> constexpr int fix_rows() { return 256 * 4 / BN; }
template <int BN, bool PAIR, int MORE, int U>
__global__ void __launch_bounds__(256) xent_fixup_kernel(const __grid_constant__ XParams p) {
    constexpr int TM = PAIR ? 2 * kBM : kBM;
    const int64_t KB = int64_t(p.nprod) * p.kb, ta = int64_t(blockIdx.x) * KB, tb = ta + KB;
    int c0 = int(ta * p.sk_units / p.sk_work);
    while (c0 > 0 && sk_start(p.sk_work, p.sk_units, c0) > ta) --c0;
    while (c0 + 1 < p.sk_units && sk_start(p.sk_work, p.sk_units, c0 + 1) <= ta) ++c0;
    int c1 = c0;
    while (c1 + 1 < p.sk_units && sk_start(p.sk_work, p.sk_units, c1 + 1) < tb) ++c1;
    const int s0 = sk_start(p.sk_work, p.sk_units, c0) < ta ? 1 : 0;
    int m, n;
    tile_of(p, uint32_t(p.whole + blockIdx.x), m, n);
    // four columns a thread
    const int r = int(blockIdx.y) * fix_rows<BN>() + int(threadIdx.x) / (BN / 4), c4 = int(threadIdx.x) % (BN / 4) * 4;
    const int row = m * TM + r, col = n * BN + c4, h = r / kBM, lr = r % kBM;
    const bool on = c1 > c0 && row < p.M && col < p.N;
    float v[4] = {0.f, 0.f, 0.f, 0.f};
    // (written by kernels before the product: fetched while that still runs)
    if (MORE != kNone && on) add_more4<MORE>(p, row, col, v);
    pdl_wait();
    if (!on) return;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int c = c0; c <= c1; c += U) {
        float4 x[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (c + u <= c1) {
                const int64_t cta = PAIR ? 2 * int64_t(c + u) + h : c + u;
                const int slot = c + u == c0 ? s0 : 0;
                x[u] = ld_ordered(p.partial + ((cta * 2 + slot) * kBM + lr) * BN + c4);
            }
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (c + u <= c1) {
                acc.x += x[u].x; acc.y += x[u].y; acc.z += x[u].z; acc.w += x[u].w;
            }
    }
    v[0] += acc.x; v[1] += acc.y; v[2] += acc.z; v[3] += acc.w;
    store4(p, row, col, v);
}

// The rows of every target, in ascending order: order[first[v]] .. order[first[v + 1] - 1] are those
// with target v; span of each is (first[v], their number).  A block has 32 columns of the vocabulary, a
// lane each, and each of its W warps a share of the rows; they go through them twice, to count and to
// place, so that no order depends on timing.  Launched as a dependent of dz's product: it starts
// where that runs out of tiles.
template <int W>
__global__ void __launch_bounds__(32 * W) xent_list_kernel(const int64_t *__restrict__ targets, int64_t rows, int64_t vocab,
                                                           int *__restrict__ first, int *__restrict__ order,
                                                           int2 *__restrict__ span) {
    __shared__ int cnt[W][32], below[W];
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const uint32_t v0 = blockIdx.x * 32u;
    const int64_t share = (rows + 128 * W - 1) / (128 * W) * 128, i0 = w * share, i1 = min(rows, i0 + share);
    int less = 0;                                            // targets below the block's columns
    int at = 0;                                              // rows of this lane's column; then where they go
    int2 mine;
    auto scan = [&](auto place) {
        constexpr bool PLACE = decltype(place)::value;
#pragma unroll 1
        for (int64_t i = i0; i < i1; i += 128) {
            int64_t t[4];                                    // without branches, so that all are in flight
#pragma unroll
            for (int u = 0; u < 4; ++u) t[u] = targets[min(i + 32 * u + lane, i1 - 1)];
            uint32_t d[4];                                   // column in the block, or 32 and more
            bool hit = false;
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const bool on = (uint64_t(t[u]) >> 32 == 0) & (i + 32 * u + lane < i1);
                if (!PLACE) less += on & (uint32_t(t[u]) < v0);
                d[u] = on ? uint32_t(t[u]) - v0 : ~0u;
                hit |= d[u] < 32u;
            }
            if (!__any_sync(0xffffffffu, hit)) continue;     // most steps have none of the block's columns
#pragma unroll
            for (int u = 0; u < 4; ++u)
                for (uint32_t here = __ballot_sync(0xffffffffu, d[u] < 32u); here != 0; here &= here - 1) {
                    const int s = __ffs(here) - 1;
                    if (__shfl_sync(0xffffffffu, d[u], s) != lane) continue;
                    if constexpr (PLACE) {
                        order[at] = int(i) + 32 * u + s;
                        span[at] = mine;
                    }
                    ++at;
                }
        }
    };
    scan(std::false_type{});
#pragma unroll
    for (int o = 16; o > 0; o /= 2) less += __shfl_xor_sync(0xffffffffu, less, o);
    cnt[w][lane] = at;
    if (lane == 0) below[w] = less;
    __syncthreads();
    int all = 0, before = 0;                                 // of this lane's column; in the warps before
    less = 0;
#pragma unroll
    for (int k = 0; k < W; ++k) {
        if (k < w) before += cnt[k][lane];
        all += cnt[k][lane];
        less += below[k];
    }
    int sum = all;                                           // of this lane's and the lower lanes' columns
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
        const int x = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += x;
    }
    const bool any = __any_sync(0xffffffffu, at > 0);
    at = less + sum - all;
    if (w == 0) {                                            // (columns past the last list targets outside: past first[vocab])
        if (v0 + lane < vocab) first[v0 + lane] = at;
        if (v0 + lane == vocab - 1) first[vocab] = at + all;
    }
    mine = make_int2(at, all);
    at += before;
    if (any) scan(std::true_type{});
    // The grid is done no earlier than the product before it: one block waits for that.  (All of them would
    // keep the blocks that find no room beside it from starting before its end.)
    if (blockIdx.x == 0) pdl_wait();
}

// What the targets' dz have lost in d_w: row first[v] of sums is the sum of rest[i] x hidden row i over
// the rows i with target v, in their order.  gridDim.y warps an entry of `order`; the warps of one
// target's c entries share its row's chunks of columns.  Four entries or more are split over the warp's
// groups of lanes, four of 64 columns or sixteen of 16; fewer: a chunk of 64 columns a group.  Launched
// as a dependent of dz W, as the lists of dz's product.
__global__ void __launch_bounds__(256) xent_sums_kernel(int64_t vocab, const int *__restrict__ first,
                                                        const int *__restrict__ order, const int2 *__restrict__ span,
                                                        const float *__restrict__ rest, const __nv_bfloat16 *__restrict__ h,
                                                        int64_t ld, float *__restrict__ sums) {
    pdl_trigger();                                           // the fix-up may be scheduled
    const int e = int(blockIdx.x) * 8 + int(threadIdx.x >> 5), lane = threadIdx.x & 31, rl = lane >> 3;
    auto add = [](float (&a)[8], float f, uint4 w) {
        const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            a[2 * q] = fmaf(f, bf16_lo(x[q]), a[2 * q]);
            a[2 * q + 1] = fmaf(f, bf16_hi(x[q]), a[2 * q + 1]);
        }
    };
    auto put = [](float *out, const float (&a)[8]) {
        reinterpret_cast<float4 *>(out)[0] = make_float4(a[0], a[1], a[2], a[3]);
        reinterpret_cast<float4 *>(out)[1] = make_float4(a[4], a[5], a[6], a[7]);
    };
    if (e < first[vocab]) {
        const int lo = span[e].x, c = span[e].y, j = e - lo + c * int(blockIdx.y), warps = c * int(gridDim.y);
        const int64_t mine = 8 * (lane & 7);                 // first column of eight in a chunk; ld % 8 == 0
        if (c < 4) {
            const __nv_bfloat16 *src[3];
            float f[3];
#pragma unroll
            for (int u = 0; u < 3; ++u) {
                const int i = order[lo + min(u, c - 1)];
                f[u] = u < c ? rest[i] : 0.f;
                src[u] = h + i * ld;
            }
#pragma unroll 2
            for (int64_t col = (4 * int64_t(j) + rl) * 64 + mine; col < ld; col += 256 * int64_t(warps)) {
                float a[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int u = 0; u < 3; ++u)
                    if (u < c) add(a, f[u], *reinterpret_cast<const uint4 *>(src[u] + col));
                put(sums + lo * ld + col, a);
            }
        } else {
            // G groups of 32 / G lanes, G entries and 8 x 32 / G columns at a time
            auto split = [&](auto groups) {
                constexpr int G = decltype(groups)::value, L = 32 / G, U = 4;
                const int g = lane / L;
                for (int64_t k = int64_t(j) * 8 * L; k < ld; k += int64_t(warps) * 8 * L) {
                    const int64_t col = k + 8 * (lane % L);
                    const bool on = col < ld;
                    float a[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
                    for (int s = g; s < c; s += U * G) {
                        int i[U];
                        float f[U];
                        uint4 w[U];
#pragma unroll
                        for (int u = 0; u < U; ++u) i[u] = order[lo + min(s + u * G, c - 1)];
#pragma unroll
                        for (int u = 0; u < U; ++u) {
                            f[u] = s + u * G < c ? rest[i[u]] : 0.f;
                            w[u] = on ? *reinterpret_cast<const uint4 *>(h + i[u] * ld + col) : make_uint4(0, 0, 0, 0);
                        }
#pragma unroll
                        for (int u = 0; u < U; ++u)
                            if (s + u * G < c) add(a, f[u], w[u]);
                    }
#pragma unroll
                    for (int o = L; o < 32; o *= 2)
#pragma unroll
                        for (int q = 0; q < 8; ++q) a[q] += __shfl_xor_sync(0xffffffffu, a[q], o);
                    if (on && g == 0) put(sums + lo * ld + col, a);
                }
            };
            // a token that many rows have as target
            if (c >= 32) split(std::integral_constant<int, 16>{});
            else split(std::integral_constant<int, 4>{});
        }
    }
    if (blockIdx.x == 0 && blockIdx.y == 0) pdl_wait();      // done no earlier than the product before it
}

// zt[i] = <hidden[i], W[t_i]> in fp32: a warp a row.  rest (dz of one bf16 term): what the target's
// dz loses when it is rounded.
template <typename HT, typename WT>
__global__ void __launch_bounds__(256) xent_target_kernel(const HT *__restrict__ hidden, const WT *__restrict__ W,
                                                          const int64_t *__restrict__ targets, int64_t rows, int64_t vocab,
                                                          int64_t dim, float *__restrict__ zt, const float *__restrict__ lse,
                                                          const float *__restrict__ dloss, float *__restrict__ rest) {
    pdl_trigger();
    const int64_t row = int64_t(blockIdx.x) * 8 + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    if (row >= rows) return;
    const int64_t t = targets[row];
    if (t < 0 || t >= vocab) {
        if (lane == 0) {
            zt[row] = 0.f;
            if (rest != nullptr) rest[row] = 0.f;
        }
        return;
    }
    const HT *h = hidden + row * dim;
    const WT *w = W + t * dim;
    float s[4] = {0.f, 0.f, 0.f, 0.f};
    if (dim % 8 == 0) {                                      // rows of whole 16 bytes
        for (int64_t c = lane * 8; c < dim; c += 256) {
            alignas(16) HT a[8];
            alignas(16) WT b[8];
#pragma unroll
            for (int k = 0; k < int(sizeof(a) / 16); ++k) reinterpret_cast<uint4 *>(a)[k] = reinterpret_cast<const uint4 *>(h + c)[k];
#pragma unroll
            for (int k = 0; k < int(sizeof(b) / 16); ++k) reinterpret_cast<uint4 *>(b)[k] = reinterpret_cast<const uint4 *>(w + c)[k];
#pragma unroll
            for (int k = 0; k < 8; ++k) s[k & 3] = fmaf(float(a[k]), float(b[k]), s[k & 3]);
        }
    } else {
        for (int64_t c = lane; c < dim; c += 128)
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (c + 32 * k < dim) s[k] = fmaf(float(h[c + 32 * k]), float(w[c + 32 * k]), s[k]);
    }
    const float v = warp_sum((s[0] + s[1]) + (s[2] + s[3]));
    if (lane == 0) {
        zt[row] = v;
        if (rest != nullptr) {
            const float dz = exp_minus_1(v - lse[row]) * dloss[row], lost = dz - __bfloat162float(__float2bfloat16(dz));
            rest[row] = isfinite(lost) ? lost : 0.f;
        }
    }
}

// Joins the (max, sum) pairs of a row's tiles: rx rows x 256 / rx threads a block.  Each
// thread joins slots y, y + 256 / rx, ..., eight at a time, then the block its threads' pairs
// in a fixed tree.
__global__ void __launch_bounds__(256) xent_join_kernel(const float2 *__restrict__ part, int64_t ld, int slots, int rows,
                                                        int rx, const float *__restrict__ zt,
                                                        const int64_t *__restrict__ targets, int64_t vocab,
                                                        float *__restrict__ loss, float *__restrict__ lse) {
    __shared__ float2 sh[256];
    const int x = threadIdx.x % rx, y = threadIdx.x / rx, ny = 256 / rx;
    const int row = blockIdx.x * rx + x;
    pdl_wait();
    auto scaled = [](float2 a, float ref) { return a.y * ex2((a.x - ref) * kLog2e); };
    float2 a = make_float2(-INFINITY, 0.f);
    for (int s = y; s < slots && row < rows; s += 8 * ny) {
        float2 v[8];
        float m = a.x;
#pragma unroll
        for (int u = 0; u < 8; ++u)
            v[u] = s + u * ny < slots ? part[int64_t(s + u * ny) * ld + row] : make_float2(-INFINITY, 0.f);
#pragma unroll
        for (int u = 0; u < 8; ++u) m = fmaxf(m, v[u].x);
        const float ref = m == -INFINITY ? 0.f : m;
        float sum = scaled(a, ref);
#pragma unroll
        for (int u = 0; u < 8; ++u) sum += scaled(v[u], ref);
        a = make_float2(m, sum);
    }
    sh[threadIdx.x] = a;
    for (int h = ny / 2; h > 0; h /= 2) {
        __syncthreads();
        if (y < h) {
            const float2 b = sh[threadIdx.x + h * rx], c = sh[threadIdx.x];
            const float m = fmaxf(b.x, c.x), ref = m == -INFINITY ? 0.f : m;
            sh[threadIdx.x] = make_float2(m, scaled(c, ref) + scaled(b, ref));
        }
    }
    if (y == 0 && row < rows) {
        const float2 r = sh[threadIdx.x];
        // the sum is 1 at least, and no logit is above r.x: the loss is not below 0, and keeps digits that
        // the difference lse - z_t has lost
        const float l = logf(r.y);
        const int64_t t = targets[row];
        lse[row] = r.x + l;
        loss[row] = (t >= 0 && t < vocab) ? (r.x - zt[row]) + l : 0.f;
    }
}

// Rows of float32 or bf16 -> T bf16 terms [T][rows][ld], columns past `cols` zero; with
// `targets`, rows without a target are zero (what padding holds must not reach a sum over
// the rows).
template <typename SRC>
__global__ void __launch_bounds__(256) xent_pack_kernel(const SRC *__restrict__ x, int64_t rows, int cols, int ld, int terms,
                                                        const int64_t *__restrict__ targets, int64_t vocab,
                                                        __nv_bfloat16 *__restrict__ y) {
    const int64_t n = rows * (ld / 8), plane = rows * int64_t(ld);
    const uint32_t per = uint32_t(ld / 8);
    for (int64_t i = int64_t(blockIdx.x) * blockDim.x + threadIdx.x; i < n; i += int64_t(gridDim.x) * blockDim.x) {
        const int64_t r = n >> 32 ? i / per : int64_t(uint32_t(i) / per);
        const int c = int(i - r * per) * 8;
        bool on = true;
        if (targets != nullptr) {
            const int64_t t = targets[r];
            on = t >= 0 && t < vocab;
        }
        if constexpr (std::is_same<SRC, __nv_bfloat16>::value) {
            // bf16 into one term: the bits as they are, by words, half a word apart in odd places
            const int64_t e = r * cols + c, total = rows * cols;
            const uint16_t *half = reinterpret_cast<const uint16_t *>(x);
            const uint32_t *word = reinterpret_cast<const uint32_t *>(x) + (e >> 1);
            uint32_t w[5], o[4];
#pragma unroll
            for (int k = 0; k < 5; ++k) {
                const int64_t at = (e & ~int64_t(1)) + 2 * k;
                w[k] = !on || at >= total || 2 * k > 8 + int(e & 1) - 1 ? 0u : at + 1 < total ? word[k] : uint32_t(half[at]);
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                o[k] = e & 1 ? __byte_perm(w[k], w[k + 1], 0x5432) : w[k];
                const int left = cols - c - 2 * k;           // columns from here to the row's end
                if (left < 2) o[k] = left == 1 ? o[k] & 0xFFFFu : 0u;
            }
            *reinterpret_cast<uint4 *>(y + r * ld + c) = make_uint4(o[0], o[1], o[2], o[3]);
            continue;
        }
        const SRC *src = x + r * cols + c;
        float v[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = on && c + k < cols ? float(src[k]) : 0.f;
        for (int t = 0; t < terms; ++t) {
            uint32_t w[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) w[k] = next_term(v[k]);
            *reinterpret_cast<uint4 *>(y + t * plane + r * ld + c) =
                make_uint4(w[0] | (w[1] << 16), w[2] | (w[3] << 16), w[4] | (w[5] << 16), w[6] | (w[7] << 16));
        }
    }
}

// ---------------------------------------------------------------- host side

// bf16 [rows, cols] with rows `ld` elements apart, boxes of 64 columns x `box_rows`, 128-byte
// swizzle, zero fill past the edges.
int make_map(CUtensorMap *m, const void *base, int64_t rows, int64_t cols, int64_t ld, int box_rows) {
    EncodeTiled enc = encode_fn();
    TLB_REQUIRE(enc != nullptr, TLB_ECUDA, "xent: cuTensorMapEncodeTiled unavailable");
    const cuuint64_t dims[2] = {cuuint64_t(cols), cuuint64_t(rows)};
    const cuuint64_t strides[1] = {cuuint64_t(ld) * 2};
    const cuuint32_t box[2] = {cuuint32_t(kBK), cuuint32_t(box_rows)};
    const cuuint32_t estr[2] = {1, 1};
    CUresult r = enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void *>(base), dims, strides, box, estr,
                     CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    TLB_REQUIRE(r == CUDA_SUCCESS, TLB_ECUDA, "xent: tensor map encoding failed (%d)", int(r));
    return TLB_OK;
}

// A matrix operand: `terms` bf16 planes [rows, cols], `plane` elements apart, rows ld apart.
struct Mat {
    const __nv_bfloat16 *p;
    int64_t rows, cols, ld, plane;
    int terms;
    const float *f32 = nullptr;  // instead: the float32 matrix, rows cols apart, taken apart by the product
};

// beside: launches what may run beside the product (and waits for its end).
struct Nothing {
    int operator()() const { return TLB_OK; }
};
template <int BN, bool PAIR, int MODE, int TERMS, bool FINE, bool A_MN, bool B_MN, bool CONV = false, typename F = Nothing>
int launch(XParams &p, const Mat &a, const Mat &b, cudaStream_t st, bool dependent = false, F beside = F()) {
    using S = Shape<BN, PAIR>;
    constexpr int stages = stages_of<BN, PAIR, MODE, CONV>();
    constexpr int smem = stages * (CONV ? 3 : 1) * S::STAGE + epi_bytes<MODE>() + 1024;
    static_assert(stages >= (CONV ? 2 : 3) && smem <= 227 * 1024 - 512, "shared memory of one CTA");
    for (int t = 0; t < a.terms; ++t)
        TLB_TRY(make_map(&p.a[t], a.p + t * a.plane, a.rows, a.cols, a.ld, A_MN ? kBK : kBM));
    for (int t = 0; t < b.terms && !CONV; ++t)
        TLB_TRY(make_map(&p.b[t], b.p + t * b.plane, b.rows, b.cols, b.ld, B_MN ? kBK : S::BH));
    if (CONV) {
        p.bw = b.f32;
        p.b_rows = int(b.rows);
        p.b_cols = int(b.cols);
        p.b_vec = b.cols % 4 == 0;
    }
    // term products, the smallest first: i + j <= 2 of three and three, all of one and three
    p.nprod = 0;
    for (int sum = kMaxTerms - 1; sum >= 0; --sum)
        for (int i = 0; i < a.terms; ++i) {
            const int j = sum - i;
            if (j < 0 || j >= b.terms) continue;
            p.pa[p.nprod] = int8_t(i);
            p.pb[p.nprod] = int8_t(j);
            ++p.nprod;
        }
    if (CONV) p.nprod = 1;                                   // all six are a k block's
    const int64_t K = A_MN ? a.rows : a.cols;
    p.kb = int(ceil_div(K, kBK));
    p.tiles_m = int(ceil_div(p.M, S::TM));
    p.tiles_n = int(ceil_div(p.N, BN));
    const int64_t tiles = int64_t(p.tiles_m) * p.tiles_n, KB = int64_t(p.nprod) * p.kb;
    const int most = PAIR ? num_sms() / 2 : num_sms();
    TLB_REQUIRE(tiles < (int64_t(1) << 31), TLB_EUNSUPPORTED, "xent: too many tiles");
    p.whole = int(tiles);
    p.sk_work = 0;
    p.sk_units = 1;
    p.units = int(std::min<int64_t>(tiles, most));
    if (MODE == kOut) {
        // The tiles past the last full wave are split along K over all units unless a wave of
        // them costs less: a split ends in partial tiles and a second kernel, about 24 k blocks
        const int64_t rest = tiles % most;
        if (rest > 0 && KB > KB * rest / most + (CONV ? 4 : 24)) {
            p.whole = int(tiles - rest);
            p.sk_work = rest * KB;
            p.sk_units = int(std::max<int64_t>(1, std::min<int64_t>(most, p.sk_work / (CONV ? 2 : 8))));
            p.units = p.whole > 0 ? most : p.sk_units;
        }
    }
    // (a form of its own: the code costs the others 1 to 2 us; split tiles get it from the fix-up)
    constexpr int MORE = MODE != kOut || FINE ? kNone : A_MN ? kSums : kTargets;
    const bool more = MORE != kNone && p.rest != nullptr;
    auto k = xent_gemm_kernel<BN, PAIR, MODE, TERMS, FINE, A_MN, B_MN, CONV, kNone>;
    if constexpr (MORE != kNone)
        if (more && p.whole > 0) k = xent_gemm_kernel<BN, PAIR, MODE, TERMS, FINE, A_MN, B_MN, CONV, MORE>;
    TLB_CUDA(cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, smem));
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned((PAIR ? 2 : 1) * p.units));
    cfg.blockDim = dim3(CONV ? kConvThreads : kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = PAIR ? 2 : 1;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = dependent ? 2 : 1;
    TLB_CUDA(cudaLaunchKernelEx(&cfg, k, p));
    TLB_TRY(check_launch(MODE == kStats ? "xent_stats" : MODE == kGrad ? "xent_grad" : A_MN ? "xent_dw" : "xent_dh"));
    TLB_TRY(beside());
    if (p.sk_work > 0) {
        const int64_t rest = p.sk_work / KB;
        auto fix = p.sk_units > 24 * rest ? (more ? xent_fixup_kernel<BN, PAIR, MORE, 16> : xent_fixup_kernel<BN, PAIR, kNone, 16>)
                                         : (more ? xent_fixup_kernel<BN, PAIR, MORE, 8> : xent_fixup_kernel<BN, PAIR, kNone, 8>);
        TLB_CUDA(launch_dependent(fix, dim3(unsigned(rest), S::TM / fix_rows<BN>()), dim3(256), 0, st, p));
        TLB_TRY(check_launch("xent_fixup"));
    }
    return TLB_OK;
}

// Tile form.  More than 128 rows: CTA pairs on 256 x 256 tiles.  Up to 128 rows there is one
// row tile, and 128 columns a tile even out the few tiles over the SMs better than 256 when
// their last wave is fuller.
// after_targets: the kernel before it in the stream is xent_target_kernel, beside which it may start.
template <int MODE, int TERMS>
int launch_z(XParams &p, const Mat &h, const Mat &w, bool after_targets, cudaStream_t st) {
    constexpr bool fine = MODE == kStats || TERMS > 1;       // the loss is float32 whatever the operands
    if constexpr (MODE == kStats || TERMS == 3)
        if (w.f32 != nullptr)
            return launch<128, false, MODE, TERMS, true, false, false, true>(p, h, w, st, after_targets);
    if constexpr (TERMS != 2)                                // two terms: up to 64 rows
        if (p.M > kBM) return launch<256, true, MODE, TERMS, fine, false, false>(p, h, w, st, after_targets);
    const int64_t n = num_sms(), t256 = ceil_div(p.N, 256), t128 = ceil_div(p.N, 128);
    if (2 * ceil_div(t256, n) <= ceil_div(t128, n))
        return launch<256, false, MODE, TERMS, fine, false, false>(p, h, w, st, after_targets);
    return launch<128, false, MODE, TERMS, fine, false, false>(p, h, w, st, after_targets);
}

template <bool A_MN, bool FINE, typename F = Nothing>
int launch_out(XParams &p, const Mat &a, const Mat &b, cudaStream_t st, F beside = F()) {
    if constexpr (FINE && !A_MN)
        if (b.f32 != nullptr)
            return launch<128, false, kOut, 1, true, false, true, true>(p, a, b, st);
    if (p.M > kBM) return launch<256, true, kOut, 1, FINE, A_MN, true>(p, a, b, st, false, beside);
    return launch<256, false, kOut, 1, FINE, A_MN, true>(p, a, b, st, false, beside);
}

constexpr int64_t kPieceBytes = int64_t(512) << 20;   // of dz, and of packed head rows, in the workspace
constexpr int64_t kFewRows = 64;                      // bf16 rows up to which dz has two terms
// Rows up to which a float32 head is taken apart by the product itself, once for every 128 rows,
// instead of being written as three terms (2.5 times its bytes) before.  Loss, gradient in us:
//   32768 x 2560    128 rows: 115, 248 against 269, 395   333: 300, 656 against 489, 852   512: 356, 827 against 496, 871
//   50021 x 1001    128 rows:  89, 192 against 207, 297   333: 189, 439 against 309, 564   512: 255, 586 against 315, 578
//   32768 x 2560    600 rows: 446, 1004 against 667, 1180   1024: 690, 1545 against 750, 1426   2048: 1308, 3071 against 1345, 2666
// (the larger tiles of the other form pay for the gradient from about 1000 rows on, for the loss not yet at 2048).
constexpr int64_t kConvMost = 512;
constexpr int64_t kRowChunk = 16384;                  // rows of one pass of the loss (its pairs' buffer)

struct Plan {
    int h_terms, w_terms, z_terms;
    bool pack_h, pack_w, conv_w;
    int64_t dp;                  // packed row length
    int64_t piece;               // vocabulary rows of one piece (multiple of 256)
    int64_t part_ld, slots;
    size_t h, w, dz, part, zt, rest, first, order, span, sums, acc, partial, total;
    bool keep_rest, list;        // what the targets' dz lose, and its sums over the rows of each target (d_w)
};

Plan plan_of(int htype, int wtype, int64_t N, int64_t V, int64_t D, bool grad, bool grad_w) {
    Plan q;
    q.h_terms = htype == TLB_W_F32 ? 3 : 1;
    q.w_terms = wtype == TLB_W_F32 ? 3 : 1;
    q.z_terms = htype == TLB_W_F32 ? 3 : N <= kFewRows ? 2 : 1;
    q.dp = ceil_div(D, 8) * 8;
    // d_w sums over the rows: those without a target are zeroed in a copy
    q.pack_h = htype == TLB_W_F32 || D % 8 != 0 || grad_w;
    q.conv_w = wtype == TLB_W_F32 && N <= kConvMost;
    q.pack_w = !q.conv_w && (wtype == TLB_W_F32 || D % 8 != 0);
    int64_t piece = ceil_div(V, 256) * 256;
    if (grad) piece = std::min(piece, kPieceBytes / (2 * q.z_terms * std::max<int64_t>(N, 1)));
    if (q.pack_w) piece = std::min(piece, kPieceBytes / (2 * q.w_terms * q.dp));
    piece = std::min(std::max<int64_t>(piece / 256 * 256, 2048), ceil_div(V, 256) * 256);
    q.piece = ceil_div(ceil_div(V, ceil_div(V, piece)), 256) * 256;      // pieces of nearly one size
    WsPlan w;
    q.h = q.pack_h ? w.take(size_t(q.h_terms) * N * q.dp * 2) : 0;
    q.w = q.pack_w ? w.take(size_t(q.w_terms) * q.piece * q.dp * 2) : 0;
    q.part_ld = q.slots = 0;
    q.part = q.zt = q.rest = q.first = q.order = q.span = q.sums = q.dz = q.acc = q.partial = 0;
    q.keep_rest = grad && q.z_terms == 1;
    q.list = q.keep_rest && grad_w;
    if (!grad) {
        q.part_ld = ceil_div(std::min(N, kRowChunk), 32) * 32;
        // 128-wide tiles: the most slots; four an SM for up to four rows
        q.slots = std::max<int64_t>(2 * (ceil_div(V, 128) + ceil_div(V, q.piece)), 4 * num_sms());
        q.part = w.take(size_t(q.part_ld) * q.slots * 8);
        q.zt = w.take(size_t(N) * 4);
    } else {
        q.dz = w.take(size_t(q.z_terms) * N * q.piece * 2);
        q.zt = w.take(size_t(N) * 4);
        if (q.keep_rest) q.rest = w.take(size_t(N) * 4);
        if (q.list) {
            q.first = w.take(size_t(V + 1) * 4);
            q.order = w.take(size_t(N) * 4);
            q.span = w.take(size_t(N) * 8);
            q.sums = w.take(size_t(N) * q.dp * 4);
        }
        if (htype != TLB_W_F32 && q.piece < V) q.acc = w.take(size_t(N) * D * 4);
        q.partial = w.take(size_t(num_sms() + 1) * 2 * kBM * 256 * 4);
    }
    q.total = w.off;
    return q;
}

int pack(const void *x, int type, int64_t rows, int64_t cols, int64_t ld, int terms, const int64_t *targets, int64_t vocab,
         __nv_bfloat16 *y, cudaStream_t st) {
    const unsigned grid = stream_grid(rows * (ld / 8), 256);
    if (type == TLB_W_F32)
        xent_pack_kernel<float><<<grid, 256, 0, st>>>(static_cast<const float *>(x), rows, int(cols), int(ld), terms, targets,
                                                      vocab, y);
    else
        xent_pack_kernel<__nv_bfloat16><<<grid, 256, 0, st>>>(static_cast<const __nv_bfloat16 *>(x), rows, int(cols), int(ld),
                                                              terms, targets, vocab, y);
    return check_launch("xent_pack");
}

size_t elem(int type) { return type == TLB_W_F32 ? 4 : 2; }

int check_types(const char *fn, int htype, int wtype, int64_t N, int64_t V, int64_t D) {
    TLB_REQUIRE((htype == TLB_W_F32 || htype == TLB_W_BF16) && (wtype == TLB_W_F32 || wtype == TLB_W_BF16), TLB_EINVAL,
                "%s: hidden and head are float32 or bfloat16", fn);
    TLB_REQUIRE(!(htype == TLB_W_BF16 && wtype == TLB_W_F32), TLB_EUNSUPPORTED,
                "%s: bfloat16 hidden rows with a float32 head", fn);
    TLB_REQUIRE(N >= 0 && V >= 1 && D >= 1, TLB_EINVAL, "%s: needs rows >= 0, vocab >= 1, dim >= 1", fn);
    TLB_REQUIRE(N <= (int64_t(1) << 24) && V <= (int64_t(1) << 24) && D <= (int64_t(1) << 20), TLB_EUNSUPPORTED,
                "%s: rows and vocab up to 2^24, dim up to 2^20", fn);
    return TLB_OK;
}

// hidden rows as an operand, packed into the workspace where its plan asks for it
int hidden_operand(const Plan &q, int htype, const void *hidden, int64_t N, int64_t D, const int64_t *mask, int64_t V,
                   void *ws, cudaStream_t st, Mat &h) {
    if (!q.pack_h) {
        h = Mat{static_cast<const __nv_bfloat16 *>(hidden), N, D, D, 0, 1};
        return TLB_OK;
    }
    __nv_bfloat16 *y = ws_at<__nv_bfloat16>(ws, q.h);
    h = Mat{y, N, D, q.dp, N * q.dp, q.h_terms};
    return pack(hidden, htype, N, D, q.dp, q.h_terms, mask, V, y, st);
}

// rows v0 .. v0 + n of the head as an operand
int head_operand(const Plan &q, int wtype, const void *W, int64_t v0, int64_t n, int64_t D, void *ws, cudaStream_t st,
                 Mat &w) {
    const char *src = static_cast<const char *>(W) + size_t(v0) * D * elem(wtype);
    if (q.conv_w) {
        w = Mat{nullptr, n, D, D, 0, q.w_terms, reinterpret_cast<const float *>(src)};
        return TLB_OK;
    }
    if (!q.pack_w) {
        w = Mat{reinterpret_cast<const __nv_bfloat16 *>(src), n, D, D, 0, 1};
        return TLB_OK;
    }
    __nv_bfloat16 *y = ws_at<__nv_bfloat16>(ws, q.w);
    w = Mat{y, n, D, q.dp, n * q.dp, q.w_terms};
    return pack(src, wtype, n, D, q.dp, q.w_terms, nullptr, 0, y, st);
}

// Up to four rows take the kernel that reads the head once, and with a float32 head up to eight,
// in two turns.  Measured, loss and gradient in us, 32768 x 2560 | 110656 x 832, against tensor cores:
//   bf16                4 rows: 40, 77 against 44, 91 | 1024 wide, 151936: 75, 153 against 78, 154
//   float32 and bf16    4 rows: 38, 76 against 82, 147 | 56, 114 against 77, 162;   8 rows: 75, 152 | 111, 226
//   float32             8 rows: 111, 189 | 137, 280;   12: 165, 284 | 204, 419 against 112, 239 | 126, 295
bool by_tokens(const Plan &q, int64_t rows, int64_t dim, bool grad) {
    const int64_t turns = ceil_div(rows, 4), last = rows - 4 * (turns - 1);
    return turns <= (q.w_terms > 1 ? 2 : 1) && xent_token_supported(std::min<int64_t>(rows, 4), dim, grad) &&
           xent_token_supported(last, dim, grad);
}

int target_logits(int htype, const void *hidden, int wtype, const void *W, const int64_t *targets, int64_t rows, int64_t vocab,
                  int64_t dim, float *zt, const float *lse, const float *dloss, float *rest, cudaStream_t st) {
    const unsigned grid = unsigned(ceil_div(rows, 8));
    const float *hf = static_cast<const float *>(hidden);
    const __nv_bfloat16 *hb = static_cast<const __nv_bfloat16 *>(hidden), *wb = static_cast<const __nv_bfloat16 *>(W);
    if (wtype == TLB_W_F32)
        xent_target_kernel<<<grid, 256, 0, st>>>(hf, static_cast<const float *>(W), targets, rows, vocab, dim, zt, lse, dloss, rest);
    else if (htype == TLB_W_F32)
        xent_target_kernel<<<grid, 256, 0, st>>>(hf, wb, targets, rows, vocab, dim, zt, lse, dloss, rest);
    else
        xent_target_kernel<<<grid, 256, 0, st>>>(hb, wb, targets, rows, vocab, dim, zt, lse, dloss, rest);
    return check_launch("xent_target");
}

// Which rows have each target, and what their dz lose, summed; both beside a product.
int list_targets(const Plan &q, void *ws, const int64_t *targets, int64_t rows, int64_t vocab, cudaStream_t st) {
    const int64_t blocks = ceil_div(vocab, 32);
    // 32 warps a block where all blocks run at once (both gradients of 4096 x 1024 x 4096 122 us, of 100000 x
    // 64 x 1000 363, with 8 warps 128 and 570), 8 where there are many
    const bool wide = blocks <= 2 * num_sms();
    TLB_CUDA(launch_dependent(wide ? xent_list_kernel<32> : xent_list_kernel<8>, dim3(unsigned(blocks)), dim3(wide ? 1024 : 256), 0,
                              st, targets, rows, vocab, ws_at<int>(ws, q.first), ws_at<int>(ws, q.order), ws_at<int2>(ws, q.span)));
    return check_launch("xent_list");
}
int sum_rests(const Plan &q, void *ws, int64_t rows, int64_t vocab, const Mat &h, cudaStream_t st) {
    TLB_CUDA(launch_dependent(xent_sums_kernel, dim3(unsigned(ceil_div(rows, 8)), unsigned(ceil_div(h.ld, 512))), dim3(256), 0, st,
                              vocab, ws_at<int>(ws, q.first), ws_at<int>(ws, q.order), ws_at<int2>(ws, q.span),
                              ws_at<float>(ws, q.rest), h.p, h.ld, ws_at<float>(ws, q.sums)));
    return check_launch("xent_sums");
}

const void *row_of(const void *x, int type, int64_t r, int64_t dim) {
    return static_cast<const char *>(x) + size_t(r) * dim * elem(type);
}

int join(const Plan &q, void *ws, int64_t r0, int64_t n, int slots, const int64_t *targets, int64_t vocab, float *loss,
         float *lse, cudaStream_t st) {
    int rx = 1;                                              // a block for every SM first, then whole sectors
    while (rx < 8 && 2 * rx * int64_t(num_sms()) <= n) rx *= 2;
    TLB_CUDA(launch_dependent(xent_join_kernel, dim3(unsigned(ceil_div(n, rx))), dim3(256), 0, st,
                              ws_at<float2>(ws, q.part), q.part_ld, slots, int(n), rx, ws_at<float>(ws, q.zt) + r0,
                              targets + r0, vocab, loss + r0, lse + r0));
    return check_launch("xent_join");
}

}  // namespace

}  // namespace tlb

using namespace tlb;

extern "C" {

size_t tlb_xent_workspace_bytes(int32_t htype, int32_t wtype, int64_t rows, int64_t vocab, int64_t dim, int32_t grad_w) {
    clear_error();
    if (check_types("xent_workspace_bytes", htype, wtype, rows, vocab, dim) != TLB_OK) return 0;
    return std::max(plan_of(htype, wtype, rows, vocab, dim, false, false).total,
                    plan_of(htype, wtype, rows, vocab, dim, true, grad_w != 0).total);
}

size_t tlb_xent_forward_workspace_bytes(int32_t htype, int32_t wtype, int64_t rows, int64_t vocab, int64_t dim) {
    clear_error();
    if (check_types("xent_forward_workspace_bytes", htype, wtype, rows, vocab, dim) != TLB_OK) return 0;
    return plan_of(htype, wtype, rows, vocab, dim, false, false).total;
}

int tlb_xent_forward(int32_t htype, const void *hidden, int32_t wtype, const void *W, const int64_t *targets, int64_t rows,
                     int64_t vocab, int64_t dim, float *loss, float *lse, void *ws, size_t ws_bytes, void *stream) {
    clear_error();
    TLB_TRY(check_types("xent_forward", htype, wtype, rows, vocab, dim));
    if (rows == 0) return TLB_OK;
    TLB_REQUIRE(hidden && W && targets && loss && lse, TLB_EINVAL, "xent_forward: null pointer");
    TLB_REQUIRE(aligned16(hidden) && aligned16(W), TLB_EINVAL, "xent_forward: hidden and W must be 16-byte aligned");
    const Plan q = plan_of(htype, wtype, rows, vocab, dim, false, false);
    TLB_REQUIRE(ws != nullptr && (reinterpret_cast<uintptr_t>(ws) & 255) == 0 && ws_bytes >= q.total, TLB_EINVAL,
                "xent_forward: needs a 256-byte aligned workspace of %zu bytes", q.total);
    cudaStream_t st = as_stream(stream);
    if (by_tokens(q, rows, dim, false)) {
        for (int64_t r0 = 0; r0 < rows; r0 += 4) {
            const int64_t n = std::min<int64_t>(4, rows - r0);
            int slots = 0;
            TLB_TRY(xent_token_loss(htype, row_of(hidden, htype, r0, dim), wtype, W, targets + r0, n, vocab, dim,
                                    ws_at<float2>(ws, q.part), q.part_ld, ws_at<float>(ws, q.zt) + r0,
                                    ws_at<uint32_t>(ws, 0), &slots, st));
            TLB_TRY(join(q, ws, r0, n, slots, targets, vocab, loss, lse, st));
        }
        return TLB_OK;
    }
    Mat h;
    TLB_TRY(hidden_operand(q, htype, hidden, rows, dim, nullptr, vocab, ws, st, h));
    const int64_t step = q.pack_w ? q.piece : vocab;
    for (int64_t r0 = 0; r0 < rows; r0 += kRowChunk) {
        const int64_t n = std::min(kRowChunk, rows - r0);
        Mat hr = h;
        hr.p += r0 * h.ld;
        hr.rows = n;
        int slot = 0;
        for (int64_t v0 = 0; v0 < vocab; v0 += step) {
            Mat w;
            const int64_t nv = std::min(step, vocab - v0);
            TLB_TRY(head_operand(q, wtype, W, v0, nv, dim, ws, st, w));
            if (v0 == 0)
                TLB_TRY(target_logits(htype, row_of(hidden, htype, r0, dim), wtype, W, targets + r0, n, vocab, dim,
                                      ws_at<float>(ws, q.zt) + r0, nullptr, nullptr, nullptr, st));
            XParams p;
            memset(&p, 0, sizeof(p));
            p.M = int(n);
            p.N = int(nv);
            p.targets = targets + r0;
            p.vocab = vocab;
            p.v0 = v0;
            p.part = ws_at<float2>(ws, q.part) + int64_t(slot) * q.part_ld;
            p.ld_part = q.part_ld;
            p.zt = ws_at<float>(ws, q.zt) + r0;
            p.status = ws_at<uint32_t>(ws, 0);
            TLB_TRY((launch_z<kStats, 1>(p, hr, w, v0 == 0, st)));
            slot += 2 * p.tiles_n;
        }
        TLB_TRY(join(q, ws, r0, n, slot, targets, vocab, loss, lse, st));
    }
    return TLB_OK;
}

int tlb_xent_backward(int32_t htype, const void *hidden, int32_t wtype, const void *W, const int64_t *targets,
                      const float *lse, const float *d_loss, int64_t rows, int64_t vocab, int64_t dim, void *d_hidden,
                      void *d_w, void *ws, size_t ws_bytes, void *stream) {
    clear_error();
    TLB_TRY(check_types("xent_backward", htype, wtype, rows, vocab, dim));
    cudaStream_t st = as_stream(stream);
    if (rows == 0) {
        if (d_w != nullptr) TLB_CUDA(cudaMemsetAsync(d_w, 0, size_t(vocab) * dim * elem(htype), st));
        return TLB_OK;
    }
    TLB_REQUIRE(hidden && W && targets && lse && d_loss && d_hidden, TLB_EINVAL, "xent_backward: null pointer");
    TLB_REQUIRE(aligned16(hidden) && aligned16(W), TLB_EINVAL, "xent_backward: hidden and W must be 16-byte aligned");
    const Plan q = plan_of(htype, wtype, rows, vocab, dim, true, d_w != nullptr);
    TLB_REQUIRE(ws != nullptr && (reinterpret_cast<uintptr_t>(ws) & 255) == 0 && ws_bytes >= q.total, TLB_EINVAL,
                "xent_backward: needs a 256-byte aligned workspace of %zu bytes", q.total);
    // (several turns add to d_w, in float32: a float32 head goes with float32 rows)
    if (by_tokens(q, rows, dim, true) && aligned16(d_w)) {
        for (int64_t r0 = 0; r0 < rows; r0 += 4)
            TLB_TRY(xent_token_grad(htype, row_of(hidden, htype, r0, dim), wtype, W, targets + r0, lse + r0, d_loss + r0,
                                    std::min<int64_t>(4, rows - r0), vocab, dim,
                                    const_cast<void *>(row_of(d_hidden, htype, r0, dim)), d_w, ws_at<float>(ws, q.partial),
                                    ws_at<uint32_t>(ws, 0), r0 > 0, st));
        return TLB_OK;
    }
    Mat h;
    TLB_TRY(hidden_operand(q, htype, hidden, rows, dim, d_w != nullptr ? targets : nullptr, vocab, ws, st, h));
    const bool wide = htype == TLB_W_F32;
    float *rest = q.keep_rest ? ws_at<float>(ws, q.rest) : nullptr;
    for (int64_t v0 = 0; v0 < vocab; v0 += q.piece) {
        const int64_t nv = std::min(q.piece, vocab - v0);
        Mat w;
        TLB_TRY(head_operand(q, wtype, W, v0, nv, dim, ws, st, w));
        if (v0 == 0)
            TLB_TRY(target_logits(htype, hidden, wtype, W, targets, rows, vocab, dim, ws_at<float>(ws, q.zt), lse, d_loss, rest, st));
        const Mat dz{ws_at<__nv_bfloat16>(ws, q.dz), rows, nv, q.piece, rows * q.piece, q.z_terms};
        {
            XParams p;
            memset(&p, 0, sizeof(p));
            p.M = int(rows);
            p.N = int(nv);
            p.targets = targets;
            p.vocab = vocab;
            p.v0 = v0;
            p.lse = lse;
            p.dloss = d_loss;
            p.zt = ws_at<float>(ws, q.zt);
            for (int t = 0; t < q.z_terms; ++t)
                TLB_TRY(make_map(&p.d[t], dz.p + t * dz.plane, rows, nv, dz.ld, 32));
            p.status = ws_at<uint32_t>(ws, 0);
            if (q.z_terms == 3) TLB_TRY((launch_z<kGrad, 3>(p, h, w, v0 == 0, st)));
            else if (q.z_terms == 2) TLB_TRY((launch_z<kGrad, 2>(p, h, w, v0 == 0, st)));
            else TLB_TRY((launch_z<kGrad, 1>(p, h, w, v0 == 0, st)));
            if (q.list && v0 == 0) TLB_TRY(list_targets(q, ws, targets, rows, vocab, st));
        }
        {
            XParams p;
            memset(&p, 0, sizeof(p));
            p.M = int(rows);
            p.N = int(dim);
            float *sum = wide ? static_cast<float *>(d_hidden) : ws_at<float>(ws, q.acc);
            const bool last = v0 + nv == vocab;
            p.acc = v0 > 0 ? sum : nullptr;
            if (q.keep_rest && v0 == 0) {                    // once, whatever piece the target is in
                p.targets = targets;
                p.vocab = vocab;
                p.rest = rest;
                p.more = static_cast<const __nv_bfloat16 *>(W);
                p.ld_more = dim;
            }
            if (wide || !last) p.out32 = sum;
            else p.out16 = static_cast<__nv_bfloat16 *>(d_hidden);
            p.vec = dim % 4 == 0 && aligned16(d_hidden);
            p.partial = ws_at<float>(ws, q.partial);
            p.status = ws_at<uint32_t>(ws, 0);
            auto beside = [&] { return q.list && v0 == 0 ? sum_rests(q, ws, rows, vocab, h, st) : TLB_OK; };
            TLB_TRY((wide ? launch_out<false, true>(p, dz, w, st) : launch_out<false, false>(p, dz, w, st, beside)));
        }
        if (d_w != nullptr) {
            XParams p;
            memset(&p, 0, sizeof(p));
            p.M = int(nv);
            p.N = int(dim);
            char *out = static_cast<char *>(d_w) + size_t(v0) * dim * elem(htype);
            if (wide) p.out32 = reinterpret_cast<float *>(out);
            else p.out16 = reinterpret_cast<__nv_bfloat16 *>(out);
            p.vec = dim % 4 == 0 && aligned16(d_w);
            if (q.list) {
                p.rest = rest;
                p.sums = ws_at<float>(ws, q.sums);
                p.ld_more = h.ld;
                p.first = ws_at<int>(ws, q.first) + v0;
            }
            p.partial = ws_at<float>(ws, q.partial);
            p.status = ws_at<uint32_t>(ws, 0);
            TLB_TRY((wide ? launch_out<true, true>(p, dz, h, st) : launch_out<true, false>(p, dz, h, st)));
        }
    }
    return TLB_OK;
}

}  // extern "C"
