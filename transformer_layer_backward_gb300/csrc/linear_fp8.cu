// The transposed-weight product of operands in 8-bit blocks:
//   dX[s, i] (+)= sum_kb dy_scales[s, kb] w_scales[i / 128, kb] sum_{o in block kb} dY[s, o] W[i, o]
// with both operands K-major e4m3.  The scales change with every 128 columns, so the tensor cores sum 128
// columns at a time (exact products, float32 sums) and each of these sums is multiplied by its two scales
// and added up in registers.
//
// More than kFewRows rows: tcgen05 (kind::f8f6f4), persistent CTA pairs on 256 x 256 super-tiles:
//   warp 0       TMA producer: 128 x 128 bytes of dY and of W a stage and CTA (128-byte swizzle: one scale
//                block is one swizzle row)
//   warps 1, 2   of the even CTA, one elected lane each, issue four MMAs (M = 256, N = 128, K = 32) a k block for
//                one half of the columns, into two accumulators of 128 columns in turn: all of the tensor memory
//   warps 4..19  a thread has one row and 64 of the columns: it keeps their sums in registers and adds each
//                k block's accumulator times its scale while the next one is multiplied
// Tiles that do not fill a last wave are shared by CTA pairs along K; their parts go to the workspace and
// are joined in a fixed order by a second kernel.
// What bounds it: an accumulator is in use from its MMA's start until both CTAs have read it out, about 1700 cycles
// (MMA 260 to 400, commit to the readers 400, reading 350, arrival to the next MMA 500), and two k blocks fill the
// tensor memory: 830 cycles a k block where the MMAs need 512.  2048 x 9728 x 2560: 54.3 us (1.88 PFLOP/s), of which
// about 33 us are the 76 k blocks of the whole tiles, 5 us the start and first blocks, 5 us the results' way out, 6 us the
// shared tiles' join; the rest is not told apart.
// Measured on the way there, same sizes: MMAs issued by a lane on its own 108 us and a release arrival of cluster scope
// (it waits for the scales' loads) on top; one issuer and two accumulators of 256 columns 57 us; eight warps for the
// sums with 128 columns each 62 to 71 us; waits that spin 71 us.
//
// Up to kFewRows rows: bound by the read of W.  A warp multiplies 16 rows of W by up to 8 rows of dY an mma.sync
// (m16n8k32), straight from global memory: the 128 columns of a block may be summed in any order, so a lane's
// 16 consecutive bytes of W and of dY serve as the operands' registers as they are.  The warps of a CTA, and
// the CTAs of a cluster, share the columns of 16 rows and add up through shared memory in a fixed order.
// 1 x 9728 x 2560: 8.9 us (25 MB: 2.8 TB/s; launch, one or two rounds of loads, the sums through the cluster).  Five CTAs an
// SM leave 48 registers, of which 112 bytes a thread go to local memory.  8 x 9728 x 2560: 10.0 us.
#include <cuda.h>

#include <algorithm>
#include <cstring>

#include "async.cuh"
#include "common.cuh"
#include "fp8.cuh"
#include "tc.cuh"

namespace tlb {

namespace {

constexpr int kFewRows = 8;             // from nine on the tensor cores win: 2560 x 9728, 16 rows 14 us against 22
constexpr int64_t kMost = int64_t(1) << 24;

// ------------------------------------------------------------------ results

// Four consecutive values of a row of dX (col % 4 == 0), the last ones past `cols` left out; WIDE: cols % 4 == 0.
template <typename T, bool WIDE>
__device__ __forceinline__ void put4(T *p, int col, int cols, float4 y, bool add) {
    if (WIDE) {
        if (col >= cols) return;
        if (add) {
            const float4 c = load_float4(p);
            y.x += c.x; y.y += c.y; y.z += c.z; y.w += c.w;
        }
        store_float4(p, y);
        return;
    }
    const float v[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
    for (int k = 0; k < 4; ++k)
        if (col + k < cols) store_float(p + k, add ? v[k] + load_float(p + k) : v[k]);
}

// A warp's 32 x 32 results out of shared memory (16-byte pieces turned by their row's last three bits), four rows of
// eight lanes at a time; what they are added to is loaded kAhead rows ahead.
template <typename T>
__device__ __forceinline__ void put_rows4(T *dX, int row0, int rows, int col, int cols, const float4 *blk, int ch, int rl, bool add) {
    constexpr int kAhead = 8;
    if (col >= cols) return;
    T *p = dX + int64_t(row0 + rl) * cols + col;
#pragma unroll 1
    for (int k0 = 0; k0 < 8; k0 += kAhead) {
        float4 old[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k)
            old[k] = add && row0 + 4 * (k0 + k) + rl < rows ? load_float4(p + int64_t(4 * (k0 + k)) * cols) : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const int r = 4 * (k0 + k) + rl;
            float4 y = blk[r * 8 + (ch ^ (r & 7))];
            if (row0 + r >= rows) continue;
            if (add) { y.x += old[k].x; y.y += old[k].y; y.z += old[k].z; y.w += old[k].w; }
            store_float4(p + int64_t(4 * (k0 + k)) * cols, y);
        }
    }
}

// The same where rows do not start at multiples of four elements: a row of 32 lanes at a time.
template <typename T>
__device__ __forceinline__ void put_rows1(T *dX, int row0, int rows, int col, int cols, const float *blk, int lane, bool add) {
    constexpr int kAhead = 16;
    if (col >= cols) return;
    T *p = dX + int64_t(row0) * cols + col;
#pragma unroll 1
    for (int r0 = 0; r0 < 32 && row0 + r0 < rows; r0 += kAhead) {
        float old[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) old[k] = add && row0 + r0 + k < rows ? load_float(p + int64_t(r0 + k) * cols) : 0.f;
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const int r = r0 + k;
            const float y = blk[r * 32 + (((lane >> 2) ^ (r & 7)) << 2) + (lane & 3)];
            if (row0 + r < rows) store_float(p + int64_t(r) * cols, add ? y + old[k] : y);
        }
    }
}

// ------------------------------------------------------------------ few rows

constexpr int kRowWarps = 8;

__device__ __forceinline__ void mma_e4m3(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

struct RowsParams {
    const uint8_t *W, *dY;
    const float *ws, *ys;
    int64_t ld_w, ld_y;          // bytes from row to row, multiples of 16
    int S, out, in, nblk;
    int add;
    void *dX;
};

// 16 bytes of a row at column `col`, zeros past its end (the rows are padded to 16 bytes)
__device__ __forceinline__ uint4 piece(const uint8_t *row, int col, int out, bool there) {
    return there && col < out ? ld_stream_u4(row + col) : make_uint4(0, 0, 0, 0);
}

template <typename T>
__global__ void __launch_bounds__(kRowWarps * 32, 5) linear_fp8_rows_kernel(const RowsParams p) {
    __shared__ float part[kRowWarps][16][kFewRows + 1];
    __shared__ float mine[16][kFewRows];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    uint32_t rank, size;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
    asm("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(size));
    const int i0 = int(blockIdx.x / size) * 16;
    const int u = int(rank) * kRowWarps + warp, U = int(size) * kRowWarps;
    const int kb0 = int(int64_t(p.nblk) * u / U), kb1 = int(int64_t(p.nblk) * (u + 1) / U);
    const uint8_t *w0 = p.W + int64_t(min(i0 + g, p.in - 1)) * p.ld_w, *w1 = p.W + int64_t(min(i0 + g + 8, p.in - 1)) * p.ld_w;
    const bool r0 = i0 + g < p.in, r1 = i0 + g + 8 < p.in, there = g < p.S;
    const float *wsc = p.ws + int64_t(i0 / kFp8Block) * p.nblk;
    const uint8_t *y = p.dY + int64_t(there ? g : 0) * p.ld_y;
    float acc[4] = {};
#pragma unroll 2
    for (int kb = kb0; kb < kb1; ++kb) {
        const int c = kb * kFp8Block + t * 16;
        const uint4 a0 = piece(w0, c, p.out, r0), a1 = piece(w1, c, p.out, r1);
        const uint4 a2 = piece(w0, c + 64, p.out, r0), a3 = piece(w1, c + 64, p.out, r1);
        const float sw = __ldg(wsc + kb);
        uint4 b0 = make_uint4(0, 0, 0, 0), b1 = b0;
        if (there && c < p.out) b0 = __ldg(reinterpret_cast<const uint4 *>(y + c));
        if (there && c + 64 < p.out) b1 = __ldg(reinterpret_cast<const uint4 *>(y + c + 64));
        float d[4] = {0.f, 0.f, 0.f, 0.f};
        mma_e4m3(d, a0.x, a1.x, a0.y, a1.y, b0.x, b0.y);
        mma_e4m3(d, a0.z, a1.z, a0.w, a1.w, b0.z, b0.w);
        mma_e4m3(d, a2.x, a3.x, a2.y, a3.y, b1.x, b1.y);
        mma_e4m3(d, a2.z, a3.z, a2.w, a3.w, b1.z, b1.w);
        const int s0 = 2 * t;
        const float f0 = s0 < p.S ? sw * __ldg(p.ys + int64_t(s0) * p.nblk + kb) : 0.f;
        const float f1 = s0 + 1 < p.S ? sw * __ldg(p.ys + int64_t(s0 + 1) * p.nblk + kb) : 0.f;
        acc[0] = fmaf(d[0], f0, acc[0]);
        acc[1] = fmaf(d[1], f1, acc[1]);
        acc[2] = fmaf(d[2], f0, acc[2]);
        acc[3] = fmaf(d[3], f1, acc[3]);
    }
    part[warp][g][2 * t] = acc[0];
    part[warp][g][2 * t + 1] = acc[1];
    part[warp][g + 8][2 * t] = acc[2];
    part[warp][g + 8][2 * t + 1] = acc[3];
    __syncthreads();
    const int r = threadIdx.x & 15, s = threadIdx.x >> 4;      // consecutive threads: consecutive columns of dX
    if (s < kFewRows) {
        float sum = 0.f;
#pragma unroll
        for (int w = 0; w < kRowWarps; ++w) sum += part[w][r][s];
        mine[r][s] = sum;
    }
    if (size > 1) cluster_sync();
    else __syncthreads();
    if (rank == 0 && s < p.S && i0 + r < p.in) {
        float sum = mine[r][s];
        for (uint32_t c = 1; c < size; ++c) {
            float x;
            asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(x) : "r"(cluster_addr(&mine[r][s], c)));
            sum += x;
        }
        T *o = static_cast<T *>(p.dX) + int64_t(s) * p.in + i0 + r;
        store_float(o, p.add ? sum + load_float(o) : sum);
    }
    if (size > 1) cluster_sync();                             // no CTA leaves while its sums are read
}

template <typename T>
int rows_launch(const RowsParams &p, cudaStream_t st) {
    // A CTA takes 16 rows of W; clusters of up to eight share their columns until there are four CTAs an SM, each
    // warp having a block of 128 columns at least.
    const int64_t groups = ceil_div(p.in, 16);
    int c = 1;
    while (c < 8 && groups * c < int64_t(num_sms()) * 4 && p.nblk >= 2 * c * kRowWarps) c *= 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(groups * c));
    cfg.blockDim = dim3(kRowWarps * 32);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = unsigned(c);
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    TLB_CUDA(cudaLaunchKernelEx(&cfg, linear_fp8_rows_kernel<T>, p));
    return check_launch("linear_fp8_rows");
}

// ------------------------------------------------------------------ tcgen05

constexpr int kTM = 256, kTN = 256;      // super-tile of a CTA pair
constexpr int kHalf = 128;               // rows of dY, and of W, that one CTA stages
constexpr int kStageBytes = 2 * kHalf * kFp8Block;
constexpr int kStages = 5;
constexpr int kFirstEpi = 4;             // warps before: producer, two for the MMAs, one that only holds its place
constexpr int kEpiWarps = 16;              // four for each 32 rows, 64 columns each
constexpr int kThreads = 32 * (kFirstEpi + kEpiWarps);
// Registers a thread after the split between the two kinds of warps (setmaxnreg): 128 sums and 64 on their way.
constexpr int kFewRegs = 64, kManyRegs = 104;
constexpr int kSplitRegs = 32 * (kFirstEpi * kFewRegs + kEpiWarps * kManyRegs);
constexpr int kBlkBytes = 32 * 32 * 4;   // a warp's 32 x 32 results on their way out
constexpr int kTcSmem = kStages * kStageBytes + kEpiWarps * kBlkBytes + 1024;
static_assert(kTcSmem <= 227 * 1024, "shared memory of one CTA");

struct TcParams {
    CUtensorMap y, w;                    // e4m3 [S, out] and [in, out], boxes of 128 x 128
    const float *ys, *ws;
    int M, N, KB;
    int add;
    void *dX;
    float *partial;                      // [pairs][2 CTAs][2 slots][128][256]
    // Pair c does its share [work c / sk_pairs, work (c + 1) / sk_pairs) of the (tile, k block) units of the last
    // sk_tiles tiles (c < sk_pairs), cut at the tiles' ends, and the whole tiles c, c + pairs, ...: even pairs the
    // share first, odd pairs last, so that they do not all write at the same time.
    int tiles, sk_tiles, sk_pairs, pairs;
    uint32_t *status;
};

__host__ __device__ __forceinline__ int64_t share(int64_t work, int pairs, int c) { return work * c / pairs; }

// The segments of one pair, in order: tile, rows, columns, k blocks [kb0, kb1).  Few registers: the threads
// that add up have none to spare.
struct Walk {
    int at, end, begin;                  // units of the shared tiles still to do (at most 75 tiles of 2^17 k blocks)
    int whole;                           // next whole tile
    bool first;                          // the share before the whole tiles
    __device__ __forceinline__ Walk(const TcParams &p, int c) {
        const int64_t work = int64_t(p.sk_tiles) * p.KB;
        begin = at = c < p.sk_pairs ? int(share(work, p.sk_pairs, c)) : 0;
        end = c < p.sk_pairs ? int(share(work, p.sk_pairs, c + 1)) : 0;
        whole = c;
        first = (c & 1) == 0;
    }
    // false when there is none left; slot: where a part of a tile goes
    __device__ __forceinline__ bool next(const TcParams &p, int &m, int &n, int &kb0, int &kb1, int &slot) {
        int tile = p.tiles - p.sk_tiles;
        if (at < end && (first || whole >= tile)) {
            const int t = at / p.KB;
            slot = at == begin ? 0 : 1;
            kb0 = at - t * p.KB;
            kb1 = min(p.KB, end - t * p.KB);
            at += kb1 - kb0;
            tile += t;
        } else {
            if (whole >= tile) return false;
            tile = whole;
            whole += p.pairs;
            kb0 = 0;
            kb1 = p.KB;
            slot = 0;
        }
        const int tiles_m = (p.M + kTM - 1) / kTM;
        m = (tile % tiles_m) * kTM;
        n = (tile / tiles_m) * kTN;
        return true;
    }
};

__device__ __forceinline__ void mma_e4m3_pair(uint32_t tmem_d, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(tmem_d),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// One lane of the (converged) warp.
__device__ __forceinline__ bool elect_one() {
    uint32_t ok;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(ok));
    return ok != 0;
}

// Arrive on an mbarrier of either CTA once this warp's tensor-memory loads are done (tcgen05.wait::ld, and
// tcgen05.fence::before_thread_sync).  No data goes through other memory, so the arrival orders none: a
// release waits for the scales' loads as well, and took three quarters of the product's time.
__device__ __forceinline__ void mbar_arrive_drained(uint32_t bar_cluster) {
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar_cluster) : "memory");
}

template <typename T, bool WIDE>
__global__ void __launch_bounds__(kThreads, 1) linear_fp8_tc_kernel(const __grid_constant__ TcParams p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    __shared__ uint64_t full[kStages], empty[kStages], accfull[2][2], accempty[2][2], done;
    __shared__ uint32_t tmem_base;
    __shared__ int s_abort, s_issued, s_consumed[2];
    const int warp = __shfl_sync(0xffffffffu, int(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
    const int rank = int(cluster_rank()), pair = int(blockIdx.x >> 1);
    const bool leader = rank == 0;

    if (threadIdx.x == 0) {
        s_abort = 0;
        s_issued = s_consumed[0] = s_consumed[1] = 0;
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 2);                         // both halves of the columns
        }
        for (int i = 0; i < 4; ++i) {
            mbar_init(&accfull[i >> 1][i & 1], 1);
            mbar_init(&accempty[i >> 1][i & 1], kEpiWarps);  // half of the warps of both CTAs
        }
        mbar_init(&done, 2);
    }
    if (warp == 1) {
        tmem_alloc_pair(&tmem_base, 512);
        tmem_relinquish_pair();
    }
    fence_mbar_init();
    tc_fence_before();
    __syncthreads();
    cluster_sync();
    tc_fence_after();
    const uint32_t tmem = tmem_base;
    if (threadIdx.x == 0) {
        asm volatile("prefetch.tensormap [%0];" ::"l"(&p.y) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(&p.w) : "memory");
    }
    pdl_trigger();                                            // the join may be scheduled
    pdl_wait();                                               // padded copies of the operands

    Walk walk(p, pair);
    int m, n, kb0, kb1, slot;
    if (warp < kFirstEpi) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kFewRegs));
        // The whole warp goes through the loops and one elected lane issues, so that addresses and descriptors
        // stay in uniform registers: issued by a lane on its own, the four MMAs and two commits of a k block
        // took longer than the tensor cores need for them (1160 cycles a k block instead of 512).
        if (warp == 0) {
            // -------------------------------------------- TMA producer
            int g = 0, s = 0, phase = 1;
            bool ok = true;
            const uint32_t fb = cluster_addr(&full[0], 0);
            while (ok && walk.next(p, m, n, kb0, kb1, slot)) {
                for (int kb = kb0; kb < kb1; ++kb, ++g) {
                    if (g >= kStages && !mbar_wait(&empty[s], phase, p.status, 40u)) {
                        ok = false;
                        break;
                    }
                    if (elect_one()) {
                        uint8_t *sa = smem + s * kStageBytes;
                        if (leader) mbar_arrive_expect_tx(&full[s], 2 * kStageBytes);   // both CTAs' copies count here
                        tma_load_2d_pair(sa, &p.y, kb * kFp8Block, m + rank * kHalf, fb + 8 * s);
                        tma_load_2d_pair(sa + kStageBytes / 2, &p.w, kb * kFp8Block, n + rank * kHalf, fb + 8 * s);
                        s_issued = g + 1;
                    }
                    if (++s == kStages) { s = 0; phase ^= 1; }
                }
            }
            if (!ok) s_abort = 1;
        } else if (warp <= 2 && leader) {
            // -------------------------------------------- MMA issuers: one for each half of the columns
            // D float32, A and B e4m3, both K-major, M = 256, N = 128
            const uint32_t idesc = (1u << 4) | (uint32_t(kTN / 2 >> 3) << 17) | (uint32_t(kTM >> 4) << 24);
            const int h = warp - 1;
            // a half takes 64 of the rows of W that each CTA stages
            const uint64_t ad0 = sw128_desc(smem), bd0 = sw128_desc(smem + kStageBytes / 2 + h * 64 * kFp8Block);
            int g = 0, s = 0, phase = 0;
            bool ok = true;
            while (ok && walk.next(p, m, n, kb0, kb1, slot)) {
                for (int kb = kb0; kb < kb1; ++kb, ++g) {
                    const int b = g & 1;
                    // the copies first, which are mostly there: the accumulator is what the next MMA waits for
                    if (!mbar_wait(&full[s], phase, p.status, 41u)) { ok = false; break; }
                    if (!mbar_wait(&accempty[h][b], ((g >> 1) & 1) ^ 1, p.status, 43u)) { ok = false; break; }
                    tc_fence_after();
                    if (elect_one()) {
                        const uint64_t ad = ad0 + uint64_t(s * (kStageBytes / 16)), bd = bd0 + uint64_t(s * (kStageBytes / 16));
                        const uint32_t acc = tmem + uint32_t(h * 256 + b * 128);
#pragma unroll
                        for (int k = 0; k < kFp8Block / 32; ++k)  // 32 bytes = 2 descriptor units
                            mma_e4m3_pair(acc, ad + 2 * k, bd + 2 * k, idesc, k > 0 ? 1u : 0u);
                        mma_commit_pair(&accfull[h][b], 3);
                        s_consumed[h] = g + 1;
                    }
                    if (++s == kStages) { s = 0; phase ^= 1; }
                }
            }
            if (!ok) s_abort = 1;
            if (elect_one()) mma_commit_pair(&done, 1);
            mbar_wait(&done, 0, nullptr, 0u);
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kManyRegs));
        // ------------------------------------------------ sums in registers
        const int q = warp & 3, cq = (warp - kFirstEpi) >> 2;     // this warp's TMEM lanes and quarter of the columns
        const int h = cq >> 1;                                // the half that holds it: columns 64 h.. of each 128
        float4 *blk = reinterpret_cast<float4 *>(smem + kStages * kStageBytes + (warp - kFirstEpi) * kBlkBytes);
        const uint32_t tbase = tmem + (uint32_t(q * 32) << 16) + uint32_t(h * 256 + (cq & 1) * 64);
        int g = 0, st = 0;
        bool ok = true;
        while (ok && walk.next(p, m, n, kb0, kb1, slot)) {
            const int rows0 = m + rank * kHalf + q * 32, in_tile = (cq & 1) * 128 + h * 64, cols0 = n + in_tile;
            const bool any = rows0 < p.M && cols0 < p.N;      // the warp has results to write
            const int yrow = min(rows0 + lane, p.M - 1), wrow = any ? cols0 / kFp8Block : 0;
            auto scale_of = [&](const float *scales, int row, int kb) { return __ldg(scales + int64_t(row) * p.KB + kb); };
            float acc[64];
#pragma unroll
            for (int c = 0; c < 64; ++c) acc[c] = 0.f;
            float sy = scale_of(p.ys, yrow, kb0), sw = scale_of(p.ws, wrow, kb0);
            for (int kb = kb0; kb < kb1; ++kb, ++g) {
                const int b = g & 1;
                const float s = sy * sw;
                if (kb + 1 < kb1) {
                    sy = scale_of(p.ys, yrow, kb + 1);
                    sw = scale_of(p.ws, wrow, kb + 1);
                }
                if (!mbar_wait(&accfull[h][b], (g >> 1) & 1, p.status, 42u)) { ok = false; break; }
                // the MMAs that read this stage are done, in both CTAs
                if (q == 0 && (cq & 1) == 0 && lane == 0) mbar_arrive(&empty[st]);
                if (++st == kStages) st = 0;
                tc_fence_after();
                if (any) {
                    uint32_t v[2][16];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        // 16 columns on their way while the 16 before are added
                        if (j == 0) tmem_ld16(tbase + uint32_t(b * 128), v[0]);
                        tmem_wait_ld();
                        if (j < 3) tmem_ld16(tbase + uint32_t(b * 128 + (j + 1) * 16), v[(j + 1) & 1]);
#pragma unroll
                        for (int c = 0; c < 16; ++c) acc[j * 16 + c] = fmaf(__uint_as_float(v[j & 1][c]), s, acc[j * 16 + c]);
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_drained(cluster_addr(&accempty[h][b], 0));
            }
            if (!ok) break;
            if (!any) continue;
            // 32 x 32 at a time through shared memory, so that lanes run along columns: 16 bytes a lane, whose places in
            // a row are turned by the row's last three bits (no bank is met twice either way)
            const bool whole = kb0 == 0 && kb1 == p.KB;
            const int ch = lane & 7, rl = lane >> 3;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
#pragma unroll
                for (int c = 0; c < 8; ++c)
                    blk[lane * 8 + (c ^ (lane & 7))] =
                        make_float4(acc[j * 32 + 4 * c], acc[j * 32 + 4 * c + 1], acc[j * 32 + 4 * c + 2], acc[j * 32 + 4 * c + 3]);
                __syncwarp();
                if (!whole) {
#pragma unroll 2
                    for (int k = 0; k < 8; ++k) {
                        const int r = 4 * k + rl;
                        if (rows0 + r < p.M)
                            *reinterpret_cast<float4 *>(p.partial + ((int64_t(blockIdx.x) * 2 + slot) * kHalf + q * 32 + r) * kTN +
                                                        in_tile + j * 32 + ch * 4) = blk[r * 8 + (ch ^ (r & 7))];
                    }
                } else if (WIDE) {
                    put_rows4(static_cast<T *>(p.dX), rows0, p.M, cols0 + j * 32 + ch * 4, p.N, blk, ch, rl, p.add != 0);
                } else {
                    put_rows1(static_cast<T *>(p.dX), rows0, p.M, cols0 + j * 32 + lane, p.N, reinterpret_cast<const float *>(blk),
                              lane, p.add != 0);
                }
                __syncwarp();
            }
        }
        if (!ok) s_abort = 1;
    }
    // wind down: the MMA thread waited for its last commit; after an abort also wait (bounded) for the copies
    // that were issued and never consumed
    tc_fence_before();
    __syncthreads();
    if (s_abort && threadIdx.x == 0 && leader) {
        for (int g = min(s_consumed[0], s_consumed[1]); g < s_issued; ++g) mbar_wait(&full[g % kStages], (g / kStages) & 1, nullptr, 0u);
    }
    __syncthreads();
    cluster_sync();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc_pair(tmem, 512);
    }
}

// Joins the parts of the shared tiles in the pairs' order.  Block (tile, y) does rows 2 y and 2 y + 1.
template <typename T, bool WIDE>
__global__ void __launch_bounds__(128) linear_fp8_join_kernel(const __grid_constant__ TcParams p) {
    const int tiles_m = (p.M + kTM - 1) / kTM, tile = p.tiles - p.sk_tiles + int(blockIdx.x);
    const int m = (tile % tiles_m) * kTM, n = (tile / tiles_m) * kTN;
    const int64_t work = int64_t(p.sk_tiles) * p.KB, ta = int64_t(blockIdx.x) * p.KB, tb = ta + p.KB;
    int c0 = int(ta * p.sk_pairs / work);                     // the pair whose share holds unit ta
    while (share(work, p.sk_pairs, c0 + 1) <= ta) ++c0;
    int c1 = c0;
    while (share(work, p.sk_pairs, c1 + 1) < tb) ++c1;
    pdl_wait();                                               // before any block leaves: what comes next waits for this kernel
    if (c1 == c0) return;                                     // done whole by one pair
    const int s0 = share(work, p.sk_pairs, c0) < ta ? 1 : 0;  // that pair began in the tile before
    const int c4 = (threadIdx.x & 63) * 4;
    for (int r = int(blockIdx.y) * 2 + (threadIdx.x >> 6); r < min(kTM, p.M - m); r += int(gridDim.y) * 2) {
        const int h = r / kHalf, lr = r % kHalf;
        float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
        constexpr int kAhead = 8;                             // loads in flight (20 took registers: 512 x 9728 x 2560 32 us, 8: 26)
        for (int c = c0; c <= c1; c += kAhead) {
            float4 v[kAhead];
#pragma unroll
            for (int u = 0; u < kAhead; ++u)
                if (c + u <= c1)
                    v[u] = __ldcg(reinterpret_cast<const float4 *>(
                        p.partial + ((int64_t(2 * (c + u) + h) * 2 + (c + u == c0 ? s0 : 0)) * kHalf + lr) * kTN + c4));
#pragma unroll
            for (int u = 0; u < kAhead; ++u)
                if (c + u <= c1) {
                    y.x += v[u].x; y.y += v[u].y; y.z += v[u].z; y.w += v[u].w;
                }
        }
        if (n + c4 < p.N)
            put4<T, WIDE>(static_cast<T *>(p.dX) + int64_t(m + r) * p.N + n + c4, n + c4, p.N, y, p.add != 0);
    }
}

// How the tiles are spread over the CTA pairs.
struct Plan {
    int tiles, sk_tiles, sk_pairs, pairs;
};

Plan plan_of(int64_t M, int64_t N, int64_t KB) {
    const int P = std::max(1, num_sms() / 2);
    const int64_t tiles = ceil_div(M, kTM) * ceil_div(N, kTN);
    Plan pl{int(tiles), 0, 0, int(std::min<int64_t>(tiles, P))};
    const int rest = int(tiles % P);
    if (rest == 0) return pl;
    // The tiles of the last wave: whole on `rest` pairs, or shared by more along K, evenly (a multiple of `rest`) or
    // by all P.  In k blocks of a pair: a part of a tile costs kPart more where it is written, and kJoin (for 256 rows)
    // where it is read.  Fitted to 1000 x 9728 x 2560 (40 tiles of 76 k blocks: whole 42 us, by 76 pairs 55),
    // 1500 x 4096 x 4096 (20 of 32 beyond a wave: whole 41, by 60 pairs 39), 2048 x 2560 x 2560 (four of 20: whole 29, by 20
    // and more 25) and 2048 x 9728 x 2560 (four of 76: by 76 pairs 60, by 24 to 44 55).
    constexpr double kPart = 6.0, kJoin = 0.22;
    const double join = kJoin * double(std::min<int64_t>(M, kTM)) / kTM;
    double best = double(KB);
    auto consider = [&](int pairs) {
        if (pairs <= rest || pairs > P) return;
        const int64_t most = ceil_div(int64_t(rest) * KB, pairs);
        const int parts = pairs % rest == 0 ? 1 : 2;          // of a pair
        const double cost = double(most) + parts * (kPart + join * pairs);
        if (most >= 1 && cost < best) {
            best = cost;
            pl.sk_tiles = rest;
            pl.sk_pairs = pairs;
            pl.pairs = tiles > P ? P : pairs;
        }
    };
    for (int s = 2; s * rest <= P && s <= KB; ++s) consider(s * rest);
    if (int64_t(rest) * KB >= P) consider(P);
    return pl;
}

int map_of(CUtensorMap *map, const void *base, int64_t rows, int64_t cols, int64_t ld) {
    EncodeTiled enc = encode_fn();
    TLB_REQUIRE(enc != nullptr, TLB_ECUDA, "linear_fp8_backward: cuTensorMapEncodeTiled unavailable");
    const cuuint64_t dims[2] = {cuuint64_t(cols), cuuint64_t(rows)};
    const cuuint64_t strides[1] = {cuuint64_t(ld)};
    const cuuint32_t box[2] = {cuuint32_t(kFp8Block), cuuint32_t(kHalf)};
    const cuuint32_t estr[2] = {1, 1};
    const CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void *>(base), dims, strides, box, estr,
                           CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    TLB_REQUIRE(r == CUDA_SUCCESS, TLB_ECUDA, "linear_fp8_backward: tensor map encoding failed (%d)", int(r));
    return TLB_OK;
}

template <typename T, bool WIDE>
int tc_launch(const TcParams &p, bool after_copies, cudaStream_t st) {
    auto kernel = linear_fp8_tc_kernel<T, WIDE>;
    TLB_CUDA(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kTcSmem));
    static const int regs = [&] {                             // the split shares out what the block is launched with
        cudaFuncAttributes a;
        return cudaFuncGetAttributes(&a, kernel) == cudaSuccess ? a.numRegs : 0;
    }();
    TLB_REQUIRE(regs * kThreads >= kSplitRegs, TLB_ECUDA, "linear_fp8_backward: built with %d registers a thread, needs %d", regs,
                kSplitRegs / kThreads + 1);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(2 * p.pairs));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kTcSmem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;   // behind the copies of padded operands
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = after_copies ? 2 : 1;
    TLB_CUDA(cudaLaunchKernelEx(&cfg, kernel, p));
    TLB_TRY(check_launch("linear_fp8_tc"));
    if (p.sk_tiles == 0) return TLB_OK;
    const int64_t rows = std::min<int64_t>(kTM, p.M);
    TLB_CUDA(launch_dependent(linear_fp8_join_kernel<T, WIDE>, dim3(unsigned(p.sk_tiles), unsigned(ceil_div(rows, 2))), dim3(128), 0,
                              st, p));
    return check_launch("linear_fp8_join");
}

// ------------------------------------------------------------------ operands whose rows are not multiples of 16 bytes

// [rows, cols] bytes to rows of ld bytes (a multiple of 16), zeros behind each; a thread writes 16.
__global__ void __launch_bounds__(256) pad_rows_kernel(const uint8_t *__restrict__ a, int64_t a_rows, uint8_t *__restrict__ a_to,
                                                       const uint8_t *__restrict__ b, int64_t b_rows,
                                                       uint8_t *__restrict__ b_to, int64_t cols, int64_t ld) {
    pdl_trigger();                                            // the product's CTAs may be set up meanwhile
    const int64_t per = ld / 16, n = (a_rows + b_rows) * per;
    for (int64_t i = int64_t(blockIdx.x) * blockDim.x + threadIdx.x; i < n; i += int64_t(gridDim.x) * blockDim.x) {
        int64_t row = i / per;
        const int64_t c = (i - row * per) * 16;
        const bool first = row < a_rows;
        row = first ? row : row - a_rows;
        const uint8_t *src = first ? a : b;
        const int64_t at = row * cols + c, total = (first ? a_rows : b_rows) * cols;
        uint32_t w[4];
        if (c + 16 <= cols && (at & ~int64_t(3)) + 20 <= total) {
            // five aligned words, shifted to the row's own alignment (src is 16-byte aligned)
            const uint32_t *p = reinterpret_cast<const uint32_t *>(src + (at & ~int64_t(3)));
            uint32_t v[5];
#pragma unroll
            for (int k = 0; k < 5; ++k) v[k] = __ldg(p + k);
            const uint32_t shift = uint32_t(at & 3) * 8;
#pragma unroll
            for (int k = 0; k < 4; ++k) w[k] = __funnelshift_r(v[k], v[k + 1], shift);
        } else {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                w[k] = 0;
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (c + 4 * k + e < cols) w[k] |= uint32_t(__ldg(src + at + 4 * k + e)) << (8 * e);
            }
        }
        *reinterpret_cast<uint4 *>((first ? a_to : b_to) + row * ld + c) = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

// ------------------------------------------------------------------ the call

struct Layout {
    size_t partial, w, y, bytes;
};

int64_t padded(int64_t out) { return (out + 15) & ~int64_t(15); }

Layout layout_of(int64_t S, int64_t out, int64_t in) {
    Layout l{};
    WsPlan ws;
    if (S > kFewRows && in > 0 && out > 0) {
        const Plan pl = plan_of(S, in, ceil_div(out, kFp8Block));
        l.partial = ws.take(pl.sk_tiles ? size_t(pl.sk_pairs) * 4 * kHalf * kTN * sizeof(float) : 0);
    }
    if (out % 16 != 0 && S > 0) {
        l.w = ws.take(size_t(in) * padded(out));
        l.y = ws.take(size_t(S) * padded(out));
    }
    l.bytes = ws.off;
    return l;
}

template <typename T>
int run(const uint8_t *W, const float *w_scales, const uint8_t *dY, const float *dy_scales, int64_t S, int64_t out,
        int64_t in, T *dX, bool add, void *ws, cudaStream_t st) {
    const Layout l = layout_of(S, out, in);
    int64_t ld = out;
    if (out % 16 != 0) {
        ld = padded(out);
        uint8_t *w = ws_at<uint8_t>(ws, l.w), *y = ws_at<uint8_t>(ws, l.y);
        pad_rows_kernel<<<stream_grid((in + S) * (ld / 16), 256), 256, 0, st>>>(W, in, w, dY, S, y, out, ld);
        TLB_TRY(check_launch("linear_fp8_pad"));
        W = w;
        dY = y;
    }
    const int KB = int(ceil_div(out, kFp8Block));
    if (S <= kFewRows) {
        const RowsParams p{W, dY, w_scales, dy_scales, ld, ld, int(S), int(out), int(in), KB, add ? 1 : 0, dX};
        return rows_launch<T>(p, st);
    }
    TcParams p;
    memset(&p, 0, sizeof(p));
    TLB_TRY(map_of(&p.y, dY, S, out, ld));
    TLB_TRY(map_of(&p.w, W, in, out, ld));
    const Plan pl = plan_of(S, in, KB);
    p.ys = dy_scales;
    p.ws = w_scales;
    p.M = int(S);
    p.N = int(in);
    p.KB = KB;
    p.add = add ? 1 : 0;
    p.dX = dX;
    p.partial = ws_at<float>(ws, l.partial);
    p.tiles = pl.tiles;
    p.sk_tiles = pl.sk_tiles;
    p.sk_pairs = pl.sk_pairs;
    p.pairs = pl.pairs;
    p.status = static_cast<uint32_t *>(ws);
    return in % 4 == 0 ? tc_launch<T, true>(p, ld != out, st) : tc_launch<T, false>(p, ld != out, st);
}

// Sums of nothing.
template <typename T>
__global__ void zero_kernel(T *p, int64_t n) {
    for (int64_t i = int64_t(blockIdx.x) * blockDim.x + threadIdx.x; i < n; i += int64_t(gridDim.x) * blockDim.x) store_float(p + i, 0.f);
}

template <typename T>
int zero_launch(T *p, int64_t n, cudaStream_t st) {
    zero_kernel<<<stream_grid(n, 256), 256, 0, st>>>(p, n);
    return check_launch("linear_fp8_zero");
}

}  // namespace

}  // namespace tlb

using namespace tlb;

extern "C" {

size_t tlb_linear_fp8_workspace_bytes(int64_t S, int64_t out_dim, int64_t in_dim) {
    if (S < 0 || out_dim < 0 || in_dim < 0 || S > kMost || out_dim > kMost || in_dim > kMost) return 0;
    return layout_of(S, out_dim, in_dim).bytes;
}

int tlb_linear_fp8_backward(const uint8_t *W, const float *w_scales, const uint8_t *dY, const float *dy_scales, int64_t S,
                            int64_t out_dim, int64_t in_dim, int32_t type, void *dX, int32_t accumulate, void *ws,
                            size_t ws_bytes, void *stream) {
    clear_error();
    TLB_REQUIRE(type == TLB_W_F32 || type == TLB_W_BF16, TLB_EINVAL, "linear_fp8_backward: type %d is neither f32 nor bf16", type);
    TLB_REQUIRE(S >= 0 && out_dim >= 0 && in_dim >= 0, TLB_EINVAL, "linear_fp8_backward: negative size");
    TLB_REQUIRE(S <= kMost && out_dim <= kMost && in_dim <= kMost, TLB_EUNSUPPORTED, "linear_fp8_backward: a size past 2^24");
    TLB_REQUIRE(ceil_div(S, kTM) * ceil_div(in_dim, kTN) < (int64_t(1) << 31), TLB_EUNSUPPORTED, "linear_fp8_backward: dX is too large");
    if (S == 0 || in_dim == 0) return TLB_OK;
    TLB_REQUIRE(dX && (out_dim == 0 || (W && w_scales && dY && dy_scales)), TLB_EINVAL, "linear_fp8_backward: null pointer");
    TLB_REQUIRE(aligned16(W) && aligned16(dY) && aligned16(dX), TLB_EINVAL,
                "linear_fp8_backward: W, dY and dX must be 16-byte aligned");
    TLB_REQUIRE(aligned_to(w_scales, 4) && aligned_to(dy_scales, 4), TLB_EINVAL, "linear_fp8_backward: the scales must be aligned");
    const size_t need = tlb_linear_fp8_workspace_bytes(S, out_dim, in_dim);
    TLB_REQUIRE(ws != nullptr && ws_bytes >= need, TLB_EINVAL,
                "linear_fp8_backward: workspace of %zu bytes is smaller than the %zu bytes needed", ws_bytes, need);
    TLB_REQUIRE((reinterpret_cast<uintptr_t>(ws) & 255) == 0, TLB_EINVAL, "linear_fp8_backward: workspace must be 256-byte aligned");
    cudaStream_t st = as_stream(stream);
    if (type == TLB_W_F32) {
        float *x = static_cast<float *>(dX);
        if (out_dim == 0) return accumulate ? TLB_OK : zero_launch(x, S * in_dim, st);
        return run(W, w_scales, dY, dy_scales, S, out_dim, in_dim, x, accumulate != 0, ws, st);
    }
    __nv_bfloat16 *x = static_cast<__nv_bfloat16 *>(dX);
    if (out_dim == 0) return accumulate ? TLB_OK : zero_launch(x, S * in_dim, st);
    return run(W, w_scales, dY, dy_scales, S, out_dim, in_dim, x, accumulate != 0, ws, st);
}

}  // extern "C"
