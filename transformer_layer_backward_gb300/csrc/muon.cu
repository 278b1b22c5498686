// Muon step of adapter matrices: momentum, the update made orthogonal by Newton-Schulz
// steps, and the parameters moved along it.
//   m <- mu m + g;  u = g + mu m (nesterov) or m;  X0 = u / (|u|_F + eps)
//   X <- a X + b (X X^T) X + c (X X^T)^2 X     (steps times)
//   p <- p - lr (wd p + scale X)
// A matrix is taken as [r, n] with r its smaller side (a tall one through its transpose,
// which the steps commute with), r <= 64.
//
// A step is X <- P X with P = a I + b G + c G^2 a polynomial of the r x r Gram matrix
// G = X X^T, and the next Gram matrix is P G P.  So several steps need one pass over X: the
// steps' polynomials are multiplied up in the r x r space and applied to X once.  The catch
// is rounding: an error d in G (norm 1) moves the factor of a singular value s by up to d / s^2
// of it, so weak directions suffer from long runs.  At most two steps are therefore taken from
// the first Gram matrix, whose spectrum is the widest, and at most three from each later one,
// formed anew from X.  Relative L2 error of X against float64 after five steps, spectra falling
// by 1e2, emulated in fp32: 3e-7 to 3e-6, as five steps each with a Gram matrix of its own have
// (4e-7 to 1e-6); three steps before two give up to 1.3e-5, five in one run up to 5e-5.
//
// Two ways, chosen by shape; all matrices of one rank class (r rounded up to 8, 16, 32 or 64) and
// way go in one launch (of each kind):
//   cluster  X fits the shared memory of up to eight CTAs (n <= 8192, 5632, 4096, 2048 by class; a
//            class 64 of few matrices only, see in_cluster): one launch, X never leaves the SMs
//   passes   five launches for five steps, with r x r work between reads of the matrix:
//     pass   m', u = f(g, m); partial Gram matrices of column chunks
//     poly   sums them in order, |u|_F from the trace, two steps' product M
//     pass   u again from g and m'; Y = M u to the workspace; partial Gram matrices of Y
//     poly   three steps' product M
//     pass   X = M Y; p updated
//   The passes run on the CUDA cores for r <= 32, on tcgen05 with every float as three bf16 terms
//   for r > 32, where 3 r FMAs an element would bound them.
//
// Bounds, and measured (five steps):
//   one 16 x 2560 matrix: latency of the phases, 16 us in one launch (20 bytes an element are 0.1 us)
//   144 rank-16 matrices of a 36-layer stack, 118 MB to move (17.4 us): 51 us in one launch.  Its CTAs
//     go through reading, r x r products and writing in step, so that HBM idles in the middle:
//     two reads and two Gram sums of X in shared memory, then two chains of r x r products
//   seven 5 x 1001 and three 999 x 33 matrices: 62 us in two launches, chains of 14 r x r products
//   144 rank-64 matrices, 472 MB (69.6 us; 189 MB read by each pass): 342 us, passes of 76, 115 and
//     91 us and r x r products of 24 and 33 us; the passes wait for loads, for taking floats apart and
//     for their Gram matrices, which leave tile by tile (sums of two tiles in tensor memory: five
//     times the error, 1e-6 against 2e-7 in p)
#include <algorithm>
#include <cmath>
#include <cstring>
#include <type_traits>

#include "common.cuh"
#include "kernels.cuh"
#include "tc.cuh"

namespace tlb {

namespace {

constexpr int kMaxMats = 256;            // matrices of one launch (their table is a kernel parameter)
constexpr int kFirstRun = 2, kRun = 3;    // steps from the first and from each later Gram matrix
// Steps of the run after `done`: the later ones as even as they can be (of six steps 2, 2, 2, not 2, 3, 1).
__host__ __device__ __forceinline__ int run_length(int done, int steps) {
    const int rest = steps - done, runs = (rest + kRun - 1) / kRun;
    return done == 0 ? (rest < kFirstRun ? rest : kFirstRun) : (rest + runs - 1) / runs;
}
constexpr int kCluster = 8;              // CTAs of a cluster; one to all of them hold one matrix
constexpr int NT = 256;                  // threads of every kernel

struct Mat {
    float *p, *m;
    const float *g;
    int64_t y, part;                     // offsets in the workspace, in floats: Y tiles, partial Gram matrices
    int32_t r, n;
    int32_t tall;                        // stored [n, r] (else [r, n])
    int32_t vec;                         // 16-byte accesses (aligned; r % 4 == 0 of a tall one, n % 4 == 0 of a wide one)
    int32_t block0, ctas;                // first block of this matrix, and how many (one a tile for r > 32)
    float lr, lr_scale;                  // lr lr_mult, and times scale
};

struct Params {
    Mat mat[kMaxMats];
    int nmat, tiles_per_block;
    int tiles;                           // r > 32: column tiles of all matrices, numbered through (block0: a matrix's first)
    float *ws;
    int64_t mpoly;                       // offset of the products M [nmat][RP * RP]
    uint32_t *status;
    float mu, wd;
    int nesterov;
    float a, b, c, eps;                  // Newton-Schulz
    int steps;
};

// What a pass reads, and what it does with X.
enum Source { kMomentum = 0, kUpdate = 1, kY = 2 };   // m' and u; u from g and m'; Y
enum Sink { kGram = 0, kGramY = 1, kParam = 2 };      // Gram matrix; X to Y and its Gram matrix; p

// A tile of up to JT columns of X [r, n], in shared memory as [RP][LD]: 33 to 66 KB.  LD = JT + 4: the same column of eight neighbouring rows lies in eight different
// groups of four banks.
template <int RP> struct Tile {
    static constexpr int JT = RP == 8 ? 1024 : RP == 16 ? 704 : RP == 32 ? 512 : 256;
    static constexpr int LD = JT + 4, XF = RP * LD;
    static constexpr int LM = RP + 4;                       // row length of an r x r matrix in shared memory
    // Gram blocks of B x B a thread (row k of block b is b + NB k); the upper PAIRS of them
    static constexpr int B = RP == 64 ? 8 : 4, NB = RP / B, PAIRS = NB * (NB + 1) / 2;
    static constexpr int GSIZE = PAIRS * B * B;             // floats of a Gram matrix's upper blocks
};
// The threads form a Gram matrix in GROUPS groups, each with every GROUPS-th column quad.  A
// warp holds GW whole groups, which it adds up itself, for r <= 16; groups of 36 pairs run
// across warps.  PARTS shares then meet in shared memory.
template <int RP> struct Gram {
    static constexpr int GW = RP == 8 ? 8 : RP == 16 ? 3 : 0;
    static constexpr int GROUPS = GW ? GW * (NT / 32) : NT / Tile<RP>::PAIRS, PARTS = GW ? NT / 32 : GROUPS;
    static constexpr int RF = PARTS * Tile<RP>::GSIZE;      // floats where they meet
    static constexpr int OWN = (Tile<RP>::GSIZE + NT - 1) / NT;
    // this thread's group (GROUPS: none) and pair
    __device__ static void mine(int &grp, int &pair) {
        constexpr int PAIRS = Tile<RP>::PAIRS;
        if constexpr (GW > 0) {
            const int lane = threadIdx.x & 31, g = lane / PAIRS;
            grp = g < GW ? int(threadIdx.x >> 5) * GW + g : GROUPS;
            pair = lane % PAIRS;
        } else {
            grp = min(int(threadIdx.x) / PAIRS, GROUPS);
            pair = threadIdx.x % PAIRS;
        }
    }
};

// Row block and column block of upper pair `q` of an NB x NB grid.
template <int NB>
__device__ __forceinline__ void pair_of(int q, int &bi, int &bk) {
    bi = 0;
    while (q >= NB - bi) {
        q -= NB - bi;
        ++bi;
    }
    bk = bi + q;
}

// All of them into a table in shared memory (a barrier follows before its use): a search for every
// element of a Gram matrix would cost more than the rest of its sum.
template <int RP>
__device__ __forceinline__ void fill_pairs(uchar2 *pairs) {
    if (threadIdx.x < Tile<RP>::PAIRS) {
        int bi, bk;
        pair_of<Tile<RP>::NB>(threadIdx.x, bi, bk);
        pairs[threadIdx.x] = make_uchar2(uint8_t(bi), uint8_t(bk));
    }
}

// Walks through a tile's elements (columns j0 .. j0 + jn): f(C, S, e, de, at, dat, n) for runs of
// n pieces of this thread.  A piece is C::value contiguous elements; piece s starts at element
// e + s de of the matrix and stands at at + s dat of the tile, its elements S::value places
// apart.  Addresses go by increments only.
template <int RP, typename F>
__device__ __forceinline__ void visit(const Mat &a, int j0, int jn, F f) {
    constexpr int LD = Tile<RP>::LD, WARPS = NT / 32;
    constexpr std::integral_constant<int, 1> one{};
    constexpr std::integral_constant<int, 4> four{};
    constexpr std::integral_constant<int, LD> ld{};
    constexpr std::integral_constant<int, 32> k32{};
    constexpr std::integral_constant<int, 8 * WARPS> k64{};
    constexpr std::integral_constant<int, 128> k128{};
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (jn <= 0) return;                                     // a CTA past the last column
    if (!a.tall && a.vec) {                                  // a warp a row, a lane four columns
        const int n = (jn / 4 - lane + 31) >> 5;             // jn % 4 == 0
#pragma unroll 1
        for (int i = warp; i < a.r; i += WARPS)
            f(four, one, int64_t(i) * a.n + j0 + 4 * lane, k128, i * LD + 4 * lane, k128, n);
    } else if (!a.tall) {
        const int n = (jn - lane + 31) >> 5;
#pragma unroll 1
        for (int i = warp; i < a.r; i += WARPS)
            f(one, one, int64_t(i) * a.n + j0 + lane, k32, i * LD + lane, k32, n);
    } else if (a.vec) {                                      // a warp 8 columns x 16 rows: 64 contiguous bytes a column
        const int j = warp * 8 + (lane >> 2), n = (jn - j + 8 * WARPS - 1) / (8 * WARPS);
#pragma unroll 1
        for (int i = (lane & 3) * 4; i < a.r; i += 16)
            f(four, ld, int64_t(j0 + j) * a.r + i, 8 * WARPS * a.r, i * LD + j, k64, n);
    } else {                                                 // a thread a column, or some of its rows
        const int w = (jn + 31) & ~31, parts = max(1, NT / w), rows = (a.r + parts - 1) / parts;
        const int i0 = parts > 1 ? int(threadIdx.x) / w * rows : 0, n = min(rows, a.r - i0);
#pragma unroll 1
        for (int j = parts > 1 ? int(threadIdx.x) % w : int(threadIdx.x); j < jn; j += NT)
            f(one, ld, int64_t(j0 + j) * a.r + i0, one, i0 * LD + j, ld, n);
    }
}

template <int C>
__device__ __forceinline__ void load_piece(const float *p, float (&v)[C]) {
    if constexpr (C == 4) {
        const float4 x = *reinterpret_cast<const float4 *>(p);
        v[0] = x.x; v[1] = x.y; v[2] = x.z; v[3] = x.w;
    } else {
        v[0] = *p;
    }
}
template <int C>
__device__ __forceinline__ void keep_piece(float *p, const float (&v)[C]) {
    if constexpr (C == 4) *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
    else *p = v[0];
}
// To and from the tile, S places apart.
template <int C, int S>
__device__ __forceinline__ void put_piece(float *x, const float (&v)[C]) {
    if constexpr (S == 1) {
        keep_piece<C>(x, v);
    } else {
#pragma unroll
        for (int c = 0; c < C; ++c) x[c * S] = v[c];
    }
}
template <int C, int S>
__device__ __forceinline__ void take_piece(const float *x, float (&v)[C]) {
    if constexpr (S == 1) {
        load_piece<C>(x, v);
    } else {
#pragma unroll
        for (int c = 0; c < C; ++c) v[c] = x[c * S];
    }
}

// Rows past r, and columns jn .. up to a whole quad, count as 0.
template <int RP>
__device__ __forceinline__ void clear_rest(const Mat &a, float *x, int jn) {
    constexpr int LD = Tile<RP>::LD;
    const int j4 = (jn + 3) & ~3;
#pragma unroll 1
    for (int k = threadIdx.x; k < (RP - a.r) * j4; k += NT) x[(a.r + k / j4) * LD + k % j4] = 0.f;
    if (j4 > jn)
#pragma unroll 1
        for (int k = threadIdx.x; k < a.r * (j4 - jn); k += NT) x[(k / (j4 - jn)) * LD + jn + k % (j4 - jn)] = 0.f;
}

constexpr int kFlight = 4;               // pieces of a thread whose loads are in flight together

// The tile of u, from g and the momentum, which FIRST brings up to date.
template <int RP, bool FIRST>
__device__ __forceinline__ void load_update(const Params &p, const Mat &a, float *x, int j0, int jn) {
    const float mu = p.mu;
    const bool nesterov = p.nesterov != 0;
    clear_rest<RP>(a, x, jn);
    visit<RP>(a, j0, jn, [&](auto cc, auto ss, int64_t e, auto de, int at, auto dat, int n) {
        constexpr int C = decltype(cc)::value, S = decltype(ss)::value, U = kFlight;
        const float *gp = a.g + e;
        float *mp = a.m + e, *xp = x + at;
#pragma unroll 1
        for (int s = 0; s < n; s += U, gp += U * de, mp += U * de, xp += U * dat) {
            float g[U][C], m[U][C];
#pragma unroll
            for (int u = 0; u < U; ++u)
                {
                    const int o = min(u, n - 1 - s) * de;
                    load_piece<C>(gp + o, g[u]);
                    load_piece<C>(mp + o, m[u]);
                }
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (s + u < n) {
                    if constexpr (FIRST) {
#pragma unroll
                        for (int c = 0; c < C; ++c) m[u][c] = fmaf(mu, m[u][c], g[u][c]);
                        keep_piece<C>(mp + u * de, m[u]);
                    }
                    if (nesterov) {
#pragma unroll
                        for (int c = 0; c < C; ++c) m[u][c] = fmaf(mu, m[u][c], g[u][c]);
                    }
                    put_piece<C, S>(xp + u * dat, m[u]);
                }
        }
    });
}

// p moved along the tile.
template <int RP>
__device__ __forceinline__ void move_params(const Params &p, const Mat &a, const float *x, int j0, int jn) {
    const float decay = a.lr * p.wd, move = a.lr_scale;
    visit<RP>(a, j0, jn, [&](auto cc, auto ss, int64_t e, auto de, int at, auto dat, int n) {
        constexpr int C = decltype(cc)::value, S = decltype(ss)::value, U = kFlight;
        float *pp = a.p + e;
        const float *xp = x + at;
#pragma unroll 1
        for (int s = 0; s < n; s += U, pp += U * de, xp += U * dat) {
            float v[U][C];
#pragma unroll
            for (int u = 0; u < U; ++u)
                load_piece<C>(pp + min(u, n - 1 - s) * de, v[u]);
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (s + u < n) {
                    float o[C];
                    take_piece<C, S>(xp + u * dat, o);
#pragma unroll
                    for (int c = 0; c < C; ++c) v[u][c] -= fmaf(move, o[c], __fmul_rn(decay, v[u][c]));
                    keep_piece<C>(pp + u * de, v[u]);
                }
        }
    });
}

// X <- M X on the shared tile: a thread owns a column pair (for r > 32 half of its rows), so
// the product goes back in place, past one barrier where two threads share a column.  mt: M's
// columns as rows; the same for all threads, as x is for the rows of a column.  kr: r rounded up to
// 8, past which rows are 0.
template <int RP>
__device__ __forceinline__ void apply(float *x, const float *mt, int jn, int kr) {
    constexpr int LD = Tile<RP>::LD, LM = Tile<RP>::LM;
    constexpr int RH = RP > 32 ? 32 : RP, HALVES = RP / RH, W = NT / HALVES;
    static_assert(HALVES == 1 || 2 * W >= Tile<RP>::JT, "all columns at once where a barrier stands between");
    const int i0 = HALVES == 1 ? 0 : (threadIdx.x / W) * RH;
#pragma unroll 1
    for (int jb = 0; jb < jn; jb += 2 * W) {
        const int j = jb + 2 * (threadIdx.x % W);
        float2 y[RH];
#pragma unroll
        for (int i = 0; i < RH; ++i) y[i] = make_float2(0.f, 0.f);
        if (j < jn) {
#pragma unroll 2
            for (int k = 0; k < (RP > 32 ? kr : RP); ++k) {
                const float2 v = *reinterpret_cast<const float2 *>(x + k * LD + j);
#pragma unroll
                for (int i = 0; i < RH; i += 4) {
                    const float4 w = *reinterpret_cast<const float4 *>(mt + k * LM + i0 + i);
                    y[i].x = fmaf(w.x, v.x, y[i].x); y[i].y = fmaf(w.x, v.y, y[i].y);
                    y[i + 1].x = fmaf(w.y, v.x, y[i + 1].x); y[i + 1].y = fmaf(w.y, v.y, y[i + 1].y);
                    y[i + 2].x = fmaf(w.z, v.x, y[i + 2].x); y[i + 2].y = fmaf(w.z, v.y, y[i + 2].y);
                    y[i + 3].x = fmaf(w.w, v.x, y[i + 3].x); y[i + 3].y = fmaf(w.w, v.y, y[i + 3].y);
                }
            }
        }
        if constexpr (HALVES > 1) __syncthreads();
        if (j < jn) {
#pragma unroll
            for (int i = 0; i < RH; ++i) *reinterpret_cast<float2 *>(x + (i0 + i) * LD + j) = y[i];
        }
    }
}

// This thread's share of the tile's Gram matrix: block (bi, bk) over the column
// quads grp, grp + GROUPS, ...
template <int RP>
__device__ __forceinline__ void gram_tile(const uchar2 *pairs, const float *x, int jn, float (&acc)[Tile<RP>::B][Tile<RP>::B]) {
    using T = Tile<RP>;
    constexpr int B = T::B, NB = T::NB, LD = T::LD;
    int grp, pair;
    Gram<RP>::mine(grp, pair);
#pragma unroll
    for (int k = 0; k < B * B; ++k) acc[k / B][k % B] = 0.f;
    if (grp >= Gram<RP>::GROUPS) return;
    const int bi = pairs[pair].x, bk = pairs[pair].y;
    const int quads = (jn + 3) / 4;
#pragma unroll 1
    for (int q = grp; q < quads; q += Gram<RP>::GROUPS) {
        float4 s[B];
#pragma unroll
        for (int k = 0; k < B; ++k) s[k] = *reinterpret_cast<const float4 *>(x + (bi + NB * k) * LD + 4 * q);
#pragma unroll
        for (int l = 0; l < B; ++l) {
            const float4 t = *reinterpret_cast<const float4 *>(x + (bk + NB * l) * LD + 4 * q);
#pragma unroll
            for (int k = 0; k < B; ++k)
                acc[k][l] = fmaf(s[k].x, t.x, fmaf(s[k].y, t.y, fmaf(s[k].z, t.z, fmaf(s[k].w, t.w, acc[k][l]))));
        }
    }
}

// The groups' shares added up in a fixed order, through red (RF floats), onto s: this thread's
// elements threadIdx.x + o NT of the order [B * B][pair].
template <int RP>
__device__ __forceinline__ void gram_sum(float (&acc)[Tile<RP>::B][Tile<RP>::B], float *red, float (&s)[Gram<RP>::OWN]) {
    using T = Tile<RP>;
    using G = Gram<RP>;
    constexpr int B = T::B;
    int grp, pair;
    G::mine(grp, pair);
    const int part = G::GW ? int(threadIdx.x >> 5) : grp;
    if constexpr (G::GW == 3) {
#pragma unroll
        for (int k = 0; k < B * B; ++k) {
            const float v = acc[k / B][k % B];
            acc[k / B][k % B] = v + __shfl_down_sync(0xffffffffu, v, T::PAIRS) + __shfl_down_sync(0xffffffffu, v, 2 * T::PAIRS);
        }
    } else if constexpr (G::GW == 8) {
#pragma unroll
        for (int o = 4; o > 0; o /= 2)
#pragma unroll
            for (int k = 0; k < B * B; ++k)
                acc[k / B][k % B] += __shfl_down_sync(0xffffffffu, acc[k / B][k % B], o * T::PAIRS);
    }
    __syncthreads();
    if (G::GW ? int(threadIdx.x & 31) < T::PAIRS : grp < G::GROUPS) {
#pragma unroll
        for (int k = 0; k < B * B; ++k) red[part * T::GSIZE + k * T::PAIRS + pair] = acc[k / B][k % B];
    }
    __syncthreads();
#pragma unroll
    for (int o = 0; o < G::OWN; ++o) {
        const int e = threadIdx.x + o * NT;
        if (e < T::GSIZE) {
#pragma unroll
            for (int k = 0; k < G::PARTS; ++k) s[o] += red[k * T::GSIZE + e];
        }
    }
}
template <int RP>
__device__ __forceinline__ void gram_keep(const float (&s)[Gram<RP>::OWN], float *out) {
#pragma unroll
    for (int o = 0; o < Gram<RP>::OWN; ++o) {
        const int e = threadIdx.x + o * NT;
        if (e < Tile<RP>::GSIZE) out[e] = s[o];
    }
}

// Element e of [B * B][pair]: its row and column.
template <int RP>
__device__ __forceinline__ void gram_place(const uchar2 *pairs, int e, int &i, int &k) {
    using T = Tile<RP>;
    const uint32_t q = uint32_t(e) / T::PAIRS;
    const uchar2 b = pairs[uint32_t(e) - q * T::PAIRS];
    i = b.x + T::NB * int(q / T::B);
    k = b.y + T::NB * int(q % T::B);
}

// The product of `steps` Newton-Schulz polynomials P of G, times `scale`, in mm.  gm: G
// (symmetric; changed); sq, pm: scratch; all [RP][LM].  G and P are kept symmetric (the upper
// triangle, mirrored), so that a row stands for a column.  r <= 16: one warp, without block
// barriers, while the others wait; else all threads.  Then only the first kr rows and
// columns (r rounded up to 8) are formed; mm is 0 outside.
template <int RP, int PT = NT>
__device__ __forceinline__ void polynomial(float *gm, float *sq, float *pm, float *mm, int steps, int kr, float a, float b, float c,
                                           float scale) {
    constexpr int LM = Tile<RP>::LM;
    constexpr bool WARP = RP <= 16;
    // a thread's DR x DC elements
    constexpr int DC = RP == 64 ? 1024 / PT : RP == 8 ? 1 : 2, DR = RP == 64 || RP == 16 ? 4 : 2;
    static_assert((RP / DC) * (RP / DR) <= (WARP ? 32 : PT), "threads of a product");
    if constexpr (WARP) kr = RP;                             // unrolled whole
    // as few warps as hold the kr x kr elements, so that no scheduler has more of them than another
    const int tid = threadIdx.x, W = (WARP ? RP : kr) / DC, r0 = (tid / W) * DR, c0 = (tid % W) * DC;
    const bool on = r0 < kr;
    auto sync = [] {
        if constexpr (WARP) __syncwarp();
        else __syncthreads();
    };
    // out = sum_k x[k][r] y[k][c]; SYM: only the upper triangle counts and is mirrored
    enum { PLAIN, SYM, POLY };
    auto product = [&](const float *x, const float *y, float *out, auto kind) {
        constexpr int KIND = decltype(kind)::value;
        float acc[DR][DC];
#pragma unroll
        for (int s = 0; s < DR; ++s)
#pragma unroll
            for (int t = 0; t < DC; ++t) acc[s][t] = 0.f;
        const bool mine = on && (KIND == PLAIN || r0 < c0 + DC);
        if (mine) {
            constexpr int KU = WARP ? RP : 8;
#pragma unroll 1
            for (int k0 = 0; k0 < kr; k0 += KU)
#pragma unroll
            for (int k = k0; k < k0 + KU; ++k) {
                float u[DR], v[DC];
                if constexpr (DR == 4) {
                    const float4 q = *reinterpret_cast<const float4 *>(x + k * LM + r0);
                    u[0] = q.x; u[1] = q.y; u[2] = q.z; u[3] = q.w;
                } else {
                    const float2 q = *reinterpret_cast<const float2 *>(x + k * LM + r0);
                    u[0] = q.x; u[1] = q.y;
                }
                if constexpr (DC == 4) {
                    const float4 q = *reinterpret_cast<const float4 *>(y + k * LM + c0);
                    v[0] = q.x; v[1] = q.y; v[2] = q.z; v[3] = q.w;
                } else if constexpr (DC == 2) {
                    const float2 q = *reinterpret_cast<const float2 *>(y + k * LM + c0);
                    v[0] = q.x; v[1] = q.y;
                } else {
                    v[0] = y[k * LM + c0];
                }
#pragma unroll
                for (int s = 0; s < DR; ++s)
#pragma unroll
                    for (int t = 0; t < DC; ++t) acc[s][t] = fmaf(u[s], v[t], acc[s][t]);
            }
            if constexpr (KIND == POLY) {                    // a I + b x + c x^2
#pragma unroll
                for (int s = 0; s < DR; ++s)
#pragma unroll
                    for (int t = 0; t < DC; ++t)
                        acc[s][t] = fmaf(c, acc[s][t], fmaf(b, x[(r0 + s) * LM + c0 + t], r0 + s == c0 + t ? a : 0.f));
            }
        }
        sync();                                              // out may be x or y
        if (mine) {
#pragma unroll
            for (int s = 0; s < DR; ++s)
#pragma unroll
                for (int t = 0; t < DC; ++t) {
                    const int i = r0 + s, k = c0 + t;
                    if (KIND == PLAIN || i <= k) out[i * LM + k] = acc[s][t];
                    if (KIND != PLAIN && i < k) out[k * LM + i] = acc[s][t];
                }
        }
        sync();
    };
    constexpr std::integral_constant<int, PLAIN> plain{};
    constexpr std::integral_constant<int, SYM> sym{};
    constexpr std::integral_constant<int, POLY> poly{};
    for (int e = threadIdx.x; e < RP * LM; e += PT) mm[e] = 0.f;
    __syncthreads();
    if (!WARP || tid < 32) {
        for (int s = 0; s < steps; ++s) {
            product(gm, gm, pm, poly);
            if (s == 0) {
                if (on) {
#pragma unroll
                    for (int u = 0; u < DR; ++u)
#pragma unroll
                        for (int t = 0; t < DC; ++t) mm[(r0 + u) * LM + c0 + t] = pm[(r0 + u) * LM + c0 + t] * scale;
                }
                sync();
            } else {
                product(pm, mm, mm, plain);
            }
            if (s + 1 < steps) {
                // G of the next X: P G P with one factor on either side (G P P, equal but for
                // rounding, or a G left unsymmetric, cost a digit in X)
                product(gm, pm, sq, plain);                  // G P
                product(sq, pm, gm, sym);                    // (G P)^T P
            }
        }
    }
    __syncthreads();
}

// 1 / (|u|_F + eps) from the Gram matrix of u, which becomes that of X0.  A zero update stays
// zero, also for eps = 0.
template <int RP, int PT = NT>
__device__ __forceinline__ float normalise(float *gm, float *s_inv, float eps) {
    constexpr int LM = Tile<RP>::LM;
    if (threadIdx.x < 32) {
        float t = 0.f;
        for (int k = threadIdx.x; k < RP; k += 32) t += gm[k * LM + k];
        t = sqrtf(warp_sum(t)) + eps;
        if (threadIdx.x == 0) *s_inv = t > 0.f ? 1.f / t : t == 0.f ? 0.f : t;      // NaN stays
    }
    __syncthreads();
    const float inv = *s_inv;
    for (int e = threadIdx.x; e < RP * RP; e += PT) gm[(e / RP) * LM + e % RP] *= inv * inv;
    __syncthreads();
    return inv;
}

// Every thread of the cluster meets here.  The cluster's barrier wants whole warps, whose
// threads come apart in the loops over ragged tiles: the block's barrier brings them together.
__device__ __forceinline__ void cluster_meet() {
    __syncthreads();
    cluster_sync();
}

__device__ __forceinline__ float ld_cluster(const float *p, int rank) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(cluster_addr(p, uint32_t(rank))) : "memory");
    return v;
}

// ---------------------------------------------------------------- one matrix a cluster

// The whole step of a matrix whose X fits the shared memory of a.ctas CTAs of a cluster: CTA c
// of them holds columns [c w, (c + 1) w).  X never leaves the SMs: 20 bytes an element cross,
// as they must.  Gram matrices are summed through distributed shared memory, by every CTA in
// rank order, and every CTA forms the r x r products for itself.  Several matrices share a
// cluster and meet at its barriers; CTAs left over in it only do that.  r <= 16: 57 KB and 64
// registers, four CTAs an SM, so that the 576 CTAs of a 36-layer stack's rank-16 adapters run
// at once.
template <int RP> constexpr int cluster_floats() {
    return Tile<RP>::XF + Gram<RP>::RF + 2 * Tile<RP>::GSIZE + 4 * RP * Tile<RP>::LM;
}

template <int RP>
__global__ void __launch_bounds__(NT, RP <= 16 ? 4 : 1) muon_cluster_kernel(const __grid_constant__ Params p) {
    using T = Tile<RP>;
    constexpr int LM = T::LM, B = T::B;
    extern __shared__ __align__(16) float sh[];
    float *x = sh, *gm = x + T::XF, *sq = gm + RP * LM, *pm = sq + RP * LM, *mm = pm + RP * LM;
    float *part = mm + RP * LM, *red = part + 2 * T::GSIZE;  // part: two, for alternate runs
    __shared__ float s_inv;
    __shared__ uchar2 pairs[T::PAIRS];
    fill_pairs<RP>(pairs);
    int lo = 0, hi = p.nmat - 1;                            // this CTA's matrix
    while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if (p.mat[mid].block0 <= int(blockIdx.x)) lo = mid;
        else hi = mid - 1;
    }
    const Mat &a = p.mat[lo];
    const int rank = int(blockIdx.x) - a.block0, ctas = a.ctas;
    if (rank >= ctas) {
        for (int done = 0; done < p.steps; done += run_length(done, p.steps)) cluster_meet();
        cluster_meet();
        return;
    }
    const int peer0 = int(cluster_rank()) - rank;
    const int w = ((a.n + ctas - 1) / ctas + 3) & ~3;
    const int j0 = min(a.n, rank * w), jn = min(w, a.n - j0), kr = (a.r + 7) & ~7;
    load_update<RP, true>(p, a, x, j0, jn);
    float scale = 1.f;
    for (int done = 0, run = 0; done < p.steps; ++run) {
        __syncthreads();
        float *mine = part + (run & 1) * T::GSIZE;
        {
            float acc[B][B], s[Gram<RP>::OWN] = {};
            gram_tile<RP>(pairs, x, jn, acc);
            gram_sum<RP>(acc, red, s);
            gram_keep<RP>(s, mine);
        }
        cluster_meet();
        constexpr int EU = Gram<RP>::OWN % 3 == 0 ? 3 : 1;  // elements whose peers' shares are in flight together
        for (int e0 = threadIdx.x; e0 < T::GSIZE; e0 += EU * NT) {
            float v[EU][kCluster];
#pragma unroll
            for (int o = 0; o < EU; ++o)
#pragma unroll
                for (int c = 0; c < kCluster; ++c)
                    v[o][c] = c < ctas && e0 + o * NT < T::GSIZE ? ld_cluster(mine + e0 + o * NT, peer0 + c) : 0.f;
#pragma unroll
            for (int o = 0; o < EU; ++o) {
                const int e = e0 + o * NT;
                if (e >= T::GSIZE) break;
                float s = 0.f;
#pragma unroll
                for (int c = 0; c < kCluster; ++c) s += v[o][c];
                int i, k;
                gram_place<RP>(pairs, e, i, k);
                gm[i * LM + k] = s;
                gm[k * LM + i] = s;
            }
        }
        __syncthreads();
        if (run == 0) scale = normalise<RP>(gm, &s_inv, p.eps);
        const int steps = run_length(done, p.steps);
        polynomial<RP>(gm, sq, pm, mm, steps, kr, p.a, p.b, p.c, run == 0 ? scale : 1.f);
        done += steps;
        apply<RP>(x, mm, jn, kr);
    }
    __syncthreads();
    move_params<RP>(p, a, x, j0, jn);
    cluster_meet();                                          // peers have read the last partial sums
}

// ---------------------------------------------------------------- passes over longer matrices

template <int RP> constexpr int pass_floats() {
    static_assert(Gram<RP>::RF <= Tile<RP>::XF, "the groups meet in the tile's place");
    return Tile<RP>::XF + RP * Tile<RP>::LM;
}

template <int RP, int SOURCE, int SINK>
__global__ void __launch_bounds__(NT) muon_pass_kernel(const __grid_constant__ Params p) {
    using T = Tile<RP>;
    constexpr int JT = T::JT, LD = T::LD, LM = T::LM, B = T::B;
    extern __shared__ __align__(16) float sh[];
    float *x = sh, *mt = x + T::XF;
    __shared__ uchar2 pairs[T::PAIRS];
    fill_pairs<RP>(pairs);
    int lo = 0, hi = p.nmat - 1;                            // this block's matrix
    while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if (p.mat[mid].block0 <= int(blockIdx.x)) lo = mid;
        else hi = mid - 1;
    }
    const Mat &a = p.mat[lo];
    const int bl = blockIdx.x - a.block0, t0 = bl * p.tiles_per_block;
    const int t1 = min((a.n + JT - 1) / JT, t0 + p.tiles_per_block);
    if constexpr (SOURCE != kMomentum) {
        const float *src = p.ws + p.mpoly + int64_t(lo) * RP * RP;
        for (int k = threadIdx.x; k < RP * RP; k += NT) mt[(k / RP) * LM + k % RP] = src[k];
    }
    float s[Gram<RP>::OWN] = {};
    for (int t = t0; t < t1; ++t) {
        const int j0 = t * JT, jn = min(JT, a.n - j0);
        float *y = p.ws + a.y + int64_t(t) * RP * JT;       // this tile of Y: [RP][JT]
        __syncthreads();                                    // the last tile is used up (and M is there)
        if constexpr (SOURCE == kY) {
            for (int k = threadIdx.x; k < RP * (JT / 4); k += NT)
                *reinterpret_cast<float4 *>(x + (k / (JT / 4)) * LD + (k % (JT / 4)) * 4) = reinterpret_cast<const float4 *>(y)[k];
        } else {
            load_update<RP, SOURCE == kMomentum>(p, a, x, j0, jn);
        }
        __syncthreads();
        if constexpr (SOURCE != kMomentum) {
            apply<RP>(x, mt, jn, RP);
            __syncthreads();
        }
        if constexpr (SINK == kParam) {
            move_params<RP>(p, a, x, j0, jn);
        } else {
            if constexpr (SINK == kGramY) {
                const int jq = (jn + 3) / 4;
                for (int k = threadIdx.x; k < RP * jq; k += NT)
                    *reinterpret_cast<float4 *>(y + (k / jq) * JT + (k % jq) * 4) =
                        *reinterpret_cast<const float4 *>(x + (k / jq) * LD + (k % jq) * 4);
            }
            float acc[B][B];
            gram_tile<RP>(pairs, x, jn, acc);
            gram_sum<RP>(acc, x, s);       // the tile is used up
        }
    }
    if constexpr (SINK != kParam) gram_keep<RP>(s, p.ws + a.part + int64_t(bl) * T::GSIZE);
}

// ---------------------------------------------------------------- the passes for r > 32, on the tensor cores

// With r near 64 the passes' 3 r FMAs an element would bound them on the CUDA cores (180 us for
// one pass over the 94 MB of a rank-64 36-layer stack).  Here both products run on tcgen05
// with every float taken apart into three bf16 terms of 8 bits (x = x0 + x1 + x2 exactly):
//   Y^T = X^T M^T     128 columns as the MMA's rows, K = 64 rows of X, the six term products
//                     x_a m_b with a + b <= 2, the smallest first; fp32 in tensor memory
//   G = D1 + D2 + D2^T, D1 = x1 x1^T + x0 x0^T, D2 = x0 x2^T + x0 x1^T, over the columns
// What is left out is 2^-24 of a product.  A term of X lies in shared memory as [64 rows][64
// columns] blocks of 128-byte rows with 128-byte swizzle, which is an MN-major operand for the
// first product and a K-major one for the second.
constexpr int kTcJ = 128;                                   // columns of a tile
constexpr int kXPlane = 64 * kTcJ * 2, kMPlane = 64 * 64 * 2;
// Shared memory: 3 planes of X, then 3 of M.  An MMA of G reads 128 rows: 64 of a block and the
// 64 rows behind it, whose results are not looked at, so 8 KB have to lie behind X's last
// block.  Tensor memory: 64 columns each for Y, D1 and D2.  Three CTAs an SM (registers), two
// of the pass that has all of it.
template <int SOURCE, int SINK> constexpr int tc_smem() {
    return 1024 + 3 * kXPlane + (SOURCE == kMomentum ? 64 * 128 : SINK == kParam ? 3 * kMPlane : 84 * 1024 - 1024 - 3 * kXPlane);
}
template <int SOURCE, int SINK> constexpr int tc_columns() { return SINK == kParam ? 64 : SOURCE == kMomentum ? 128 : 256; }
template <int SOURCE, int SINK> constexpr int tc_ctas() { return SOURCE == kMomentum || SINK == kParam ? 3 : 2; }

// Byte offset of element (i, j) in a plane of X (blocks of 64 columns), or of M with j < 64.
__device__ __forceinline__ int plane_at(int i, int j) {
    return (j >> 6) * (64 * 128) + i * 128 + ((((j & 63) >> 3) ^ (i & 7)) << 4) + (j & 7) * 2;
}
// Cuts the 8 highest significant bits off x.
__device__ __forceinline__ uint32_t cut_term(float &x) {
    const uint32_t u = __float_as_uint(x);
    x -= __uint_as_float(u & 0xFFFF0000u);
    return u;
}
// Values into the planes: C = 4 along the columns (S = 1) or down the rows (S = 0), or one.
template <int C, int S>
__device__ __forceinline__ void put_terms(uint8_t *planes, int plane, int i, int j, float (&v)[C]) {
#pragma unroll
    for (int t = 0; t < 3; ++t, planes += plane) {
        uint32_t u[C];
#pragma unroll
        for (int c = 0; c < C; ++c) u[c] = cut_term(v[c]);
        if constexpr (C == 4 && S == 1) {
            *reinterpret_cast<uint2 *>(planes + plane_at(i, j)) =
                make_uint2(__byte_perm(u[0], u[1], 0x7632), __byte_perm(u[2], u[3], 0x7632));
        } else {
#pragma unroll
            for (int c = 0; c < C; ++c)
                *reinterpret_cast<uint16_t *>(planes + plane_at(i + (S == 0 ? c : 0), j + (S == 1 ? c : 0))) = uint16_t(u[c] >> 16);
        }
    }
}

// This thread's pieces of a tile of u, or of p: f(C, S, N, item) with item(k) the k-th of N
// pieces, {whether it exists, element offset, row, column}; S as in put_terms.
struct Piece {
    bool on;
    int64_t e;
    int i, j;
};
template <typename F>
__device__ __forceinline__ void tc_visit(const Mat &a, int j0, int jn, F f) {
    constexpr std::integral_constant<int, 0> down{};
    constexpr std::integral_constant<int, 1> one{};
    constexpr std::integral_constant<int, 4> four{};
    constexpr std::integral_constant<int, 8> n8{};
    constexpr std::integral_constant<int, 32> n32{};
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (!a.tall && a.vec) {                                  // a warp a row, a lane four columns
        f(four, one, n8, [&](int k) {
            const int i = warp + 8 * k, j = 4 * lane;
            return Piece{i < a.r && j < jn, int64_t(i) * a.n + j0 + j, i, j};
        });
    } else if (!a.tall) {
        f(one, one, n32, [&](int k) {
            const int i = warp + 8 * (k >> 2), j = lane + 32 * (k & 3);
            return Piece{i < a.r && j < jn, int64_t(i) * a.n + j0 + j, i, j};
        });
    } else if (a.vec) {                                      // a warp 8 columns x 16 rows
        f(four, down, n8, [&](int k) {
            const int j = (warp + 8 * (k >> 2)) * 8 + (lane >> 2), i = (k & 3) * 16 + (lane & 3) * 4;
            return Piece{i < a.r && j < jn, int64_t(j0 + j) * a.r + i, i, j};
        });
    } else {                                                 // a thread half a column
        f(one, down, n32, [&](int k) {
            const int j = threadIdx.x & 127, i = (threadIdx.x >> 7) * 32 + k;
            return Piece{i < a.r && j < jn, int64_t(j0 + j) * a.r + i, i, j};
        });
    }
}

// The terms of u into the planes, from g and the momentum, which FIRST brings up to date.
template <bool FIRST>
__device__ __forceinline__ void tc_load_update(const Params &p, const Mat &a, uint8_t *planes, int j0, int jn) {
    const float mu = p.mu;
    const bool nesterov = p.nesterov != 0;
    tc_visit(a, j0, jn, [&](auto cc, auto ss, auto nn, auto item) {
        constexpr int C = decltype(cc)::value, S = decltype(ss)::value, U = 4;
#pragma unroll 1
        for (int k = 0; k < decltype(nn)::value; k += U) {
            float g[U][C], m[U][C];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const Piece q = item(k + u);
                const int64_t e = q.on ? q.e : 0;
                load_piece<C>(a.g + e, g[u]);
                load_piece<C>(a.m + e, m[u]);
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const Piece q = item(k + u);
                if (!q.on) continue;
                if constexpr (FIRST) {
#pragma unroll
                    for (int c = 0; c < C; ++c) m[u][c] = fmaf(mu, m[u][c], g[u][c]);
                    keep_piece<C>(a.m + q.e, m[u]);
                }
                if (nesterov) {
#pragma unroll
                    for (int c = 0; c < C; ++c) m[u][c] = fmaf(mu, m[u][c], g[u][c]);
                }
                put_terms<C, S>(planes, kXPlane, q.i, q.j, m[u]);
            }
        }
    });
}

// Partial Gram matrices here are the upper 8 x 8 blocks one after another, each by rows: the row
// and column of element e.
__device__ __forceinline__ void block_place(const uchar2 *pairs, int e, int &i, int &k) {
    const uchar2 b = pairs[e >> 6];
    i = b.x * 8 + ((e >> 3) & 7);
    k = b.y * 8 + (e & 7);
}

// The lines of a pass's next tile on their way to L2 while this one is worked on.
__device__ __forceinline__ void prefetch_l2(const float *p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }
__device__ __forceinline__ void prefetch_tile(const Mat &a, const float *x, int j0, int jn) {
    if (a.tall) {
        for (int k = threadIdx.x * 32; k < jn * a.r; k += NT * 32) prefetch_l2(x + int64_t(j0) * a.r + k);
    } else {
        for (int k = threadIdx.x; k < a.r * (kTcJ / 32); k += NT) {
            const int c = (k % (kTcJ / 32)) * 32;
            if (c < jn) prefetch_l2(x + int64_t(k / (kTcJ / 32)) * a.n + j0 + c);
        }
    }
}
template <int SOURCE, int SINK>
__device__ __forceinline__ void tc_prefetch(const Params &p, int lo, int g) {
    if (lo + 1 < p.nmat && p.mat[lo + 1].block0 <= g) ++lo;
    const Mat &a = p.mat[lo];
    const int t = g - a.block0, j0 = t * kTcJ, jn = min(kTcJ, a.n - j0);
    if constexpr (SOURCE == kY) {
        prefetch_l2(p.ws + a.y + int64_t(t) * 64 * kTcJ + threadIdx.x * 32);
    } else {
        prefetch_tile(a, a.g, j0, jn);
        prefetch_tile(a, a.m, j0, jn);
    }
    if constexpr (SINK == kParam) prefetch_tile(a, a.p, j0, jn);
}

template <int SOURCE, int SINK>
__global__ void __launch_bounds__(NT, tc_ctas<SOURCE, SINK>()) muon_tc_pass_kernel(const __grid_constant__ Params p) {
    using T = Tile<64>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *planes = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t *mplanes = planes + 3 * kXPlane;
    __shared__ uint64_t bar_y, bar_g;
    __shared__ uint32_t tmem_base;
    __shared__ uchar2 pairs[T::PAIRS];
    fill_pairs<64>(pairs);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    // this block's share of all matrices' tiles, and the matrix of the first
    const int g0 = int(int64_t(p.tiles) * blockIdx.x / gridDim.x), g1 = int(int64_t(p.tiles) * (blockIdx.x + 1) / gridDim.x);
    int lo = 0, hi = p.nmat - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if (p.mat[mid].block0 <= g0) lo = mid;
        else hi = mid - 1;
    }
    if (warp == 0) {
        tmem_alloc(&tmem_base, tc_columns<SOURCE, SINK>());
        tmem_relinquish();
    }
    if (tid == 0) {
        mbar_init(&bar_y, 1);
        mbar_init(&bar_g, 1);
    }
    fence_mbar_init();
    tc_fence_before();
    auto clear = [&] {
        for (int k = tid; k < 3 * kXPlane / 16; k += NT) reinterpret_cast<uint4 *>(planes)[k] = make_uint4(0, 0, 0, 0);
    };
    auto load_m = [&] {
        const float *src = p.ws + p.mpoly + int64_t(lo) * 64 * 64;
        for (int k = tid; k < 64 * 16; k += NT) {
            float v[4];
            load_piece<4>(src + 4 * k, v);
            put_terms<4, 1>(mplanes, kMPlane, k / 16, (k % 16) * 4, v);
        }
    };
    if constexpr (SOURCE != kMomentum) load_m();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_base, td1 = tmem, td2 = tmem + 64, ty = SINK == kParam ? tmem : tmem + 128;
    // D f32, A and B bf16, 128 x 64; A MN-major for Y
    constexpr uint32_t idesc = (1u << 4) | (1u << 7) | (1u << 10) | (uint32_t(64 >> 3) << 17) | (uint32_t(128 >> 4) << 24);
    const int q = warp & 3, half = warp >> 2;               // TMEM lanes (columns of X), half of the rows
    // After a wait that gives up (ok: of this warp) p stays as it is, and all leave together at the next
    // barrier; `pending` is then what the last products will still arrive at.
    bool ok = true;
    uint64_t *pending = nullptr;
    int done = 0;
    for (int g = g0; g < g1; ++g, ++done) {
        if (lo + 1 < p.nmat && p.mat[lo + 1].block0 <= g) {  // the next matrix
            ++lo;
            if constexpr (SOURCE != kMomentum) load_m();
        }
        const Mat &a = p.mat[lo];
        const int t = g - a.block0, j0 = t * kTcJ, jn = min(kTcJ, a.n - j0);
        float *y = p.ws + a.y + int64_t(t) * 64 * kTcJ;      // this tile of Y: [64][128]
        // columns past the last count as 0, and so do rows past r (Y has them)
        if (SOURCE != kY && (jn < kTcJ || a.r < 64)) {
            clear();
            __syncthreads();
        }
        if constexpr (SOURCE == kY) {
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                float v[4];
                const int i = warp + 8 * k;
                load_piece<4>(y + i * kTcJ + 4 * lane, v);
                put_terms<4, 1>(planes, kXPlane, i, 4 * lane, v);
            }
        } else {
            tc_load_update<SOURCE == kMomentum>(p, a, planes, j0, jn);
        }
        fence_proxy_async();
        tc_fence_before();
        __syncthreads();
        if (g + 1 < g1) tc_prefetch<SOURCE, SINK>(p, lo, g + 1);
        if constexpr (SOURCE != kMomentum) {
            if (tid == 0) {
                tc_fence_after();
                uint32_t add = 0;
#pragma unroll
                for (int sum = 2; sum >= 0; --sum)
#pragma unroll
                    for (int ta = 0; ta <= sum; ++ta) {
                        uint64_t ad = sw128_desc(planes + ta * kXPlane);
                        // MN-major: blocks of 64 columns 8192 bytes apart (leading offset)
                        ad = (ad & ~(0x3FFFull << 16)) | (uint64_t(8192 >> 4) << 16);
                        const uint64_t bd = sw128_desc(mplanes + (sum - ta) * kMPlane);
#pragma unroll
                        for (int k = 0; k < 4; ++k) {        // 16 rows of X: 2048 bytes; of M: 32
                            mma_bf16(ty, ad + 128 * k, bd + 2 * k, idesc | (1u << 15), add);
                            add = 1;
                        }
                    }
                mma_commit(&bar_y);
            }
            // this thread's column j of X, rows i0 ..; p is fetched while the product runs
            const int j = q * 32 + lane, i0 = half * 32;
            const int64_t step = a.tall ? 1 : a.n;
            float *pp = a.tall ? a.p + int64_t(j0 + j) * a.r + i0 : a.p + int64_t(i0) * a.n + j0 + j;
            const bool quads = a.tall && a.vec;
            const int rows = j < jn ? a.r - i0 : 0;
            float x[SINK == kParam ? 32 : 1];
            if constexpr (SINK == kParam) {
#pragma unroll
                for (int c = 0; c < 32; c += 4) {
                    float *x4 = x + c;
                    if (quads) {
                        const float4 t = c < rows ? *reinterpret_cast<const float4 *>(pp + c) : make_float4(0.f, 0.f, 0.f, 0.f);
                        x4[0] = t.x; x4[1] = t.y; x4[2] = t.z; x4[3] = t.w;
                    } else {
#pragma unroll
                        for (int d = 0; d < 4; ++d) x4[d] = c + d < rows ? pp[(c + d) * step] : 0.f;
                    }
                }
            }
            ok = mbar_wait(&bar_y, done & 1, p.status, 41u);
            ok = __all_sync(0xffffffffu, ok);                // tensor memory is read by whole warps
            tc_fence_after();
            uint32_t v[32];
            tmem_ld32(ty + (uint32_t(q * 32) << 16) + uint32_t(half * 32), v);
            tmem_wait_ld();
            if constexpr (SINK == kParam) {
                const float decay = a.lr * p.wd, move = a.lr_scale;
                const int moved = ok ? rows : 0;
#pragma unroll
                for (int c = 0; c < 32; ++c) x[c] -= fmaf(move, __uint_as_float(v[c]), __fmul_rn(decay, x[c]));
#pragma unroll
                for (int c = 0; c < 32; c += 4) {
                    if (quads) {
                        if (c < moved) *reinterpret_cast<float4 *>(pp + c) = make_float4(x[c], x[c + 1], x[c + 2], x[c + 3]);
                    } else {
#pragma unroll
                        for (int d = 0; d < 4; ++d)
                            if (c + d < moved) pp[(c + d) * step] = x[c + d];
                    }
                }
            } else {                                         // (workspace only)
#pragma unroll
                for (int c = 0; c < 32; ++c) y[(i0 + c) * kTcJ + j] = __uint_as_float(v[c]);
#pragma unroll
                for (int c = 0; c < 32; ++c) {
                    float x[1] = {__uint_as_float(v[c])};
                    put_terms<1, 1>(planes, kXPlane, i0 + c, j, x);
                }
                fence_proxy_async();
            }
            tc_fence_before();
            if (__syncthreads_or(!ok)) {                     // (kParam: the planes and Y are read by all)
                pending = &bar_y;
                break;
            }
        }
        if constexpr (SINK != kParam) {
            if (tid == 0) {
                tc_fence_after();
                auto gram = [&](uint32_t d, int ta, int tb, uint32_t first) {
#pragma unroll
                    for (int k = 0; k < 8; ++k) {            // 16 columns: 32 bytes, 64 a block
                        const int off = (k >> 2) * (64 * 128);
                        mma_bf16(d, sw128_desc(planes + ta * kXPlane + off) + 2 * (k & 3),
                                 sw128_desc(planes + tb * kXPlane + off) + 2 * (k & 3), idesc, first | uint32_t(k > 0));
                    }
                };
                gram(td1, 1, 1, 0u);
                gram(td1, 0, 0, 1u);
                gram(td2, 0, 2, 0u);
                gram(td2, 0, 1, 1u);
                mma_commit(&bar_g);
            }
            // Every tile's sums go out by themselves: tensor memory cuts a sum after every MMA, and
            // a second tile's 16 onto a whole sum would cost five times the error
            ok = mbar_wait(&bar_g, done & 1, p.status, 42u);
            ok = __all_sync(0xffffffffu, ok);
            tc_fence_after();
            float *s1 = reinterpret_cast<float *>(planes), *s2 = s1 + 64 * 65;    // in the planes' place
            if (q < 2) {
                uint32_t v[32], w[32];
                const uint32_t at = (uint32_t(q * 32) << 16) + uint32_t(half * 32);
                tmem_ld32(td1 + at, v);
                tmem_ld32(td2 + at, w);
                tmem_wait_ld();
#pragma unroll
                for (int c = 0; c < 32; ++c) {
                    s1[(q * 32 + lane) * 65 + half * 32 + c] = __uint_as_float(v[c]);
                    s2[(q * 32 + lane) * 65 + half * 32 + c] = __uint_as_float(w[c]);
                }
            }
            tc_fence_before();
            if (__syncthreads_or(!ok)) {
                pending = &bar_g;
                break;
            }
            float *out = p.ws + a.part + int64_t(t) * T::GSIZE;
            for (int e = tid; e < T::GSIZE; e += NT) {
                int i, k;
                block_place(pairs, e, i, k);
                out[e] = s1[i * 65 + k] + (s2[i * 65 + k] + s2[k * 65 + i]);
            }
            __syncthreads();                                 // the planes are free again
        }
    }
    if (pending != nullptr && tid == 0) mbar_wait(pending, done & 1, nullptr, 0u);
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc(tmem, tc_columns<SOURCE, SINK>());
    }
}

// One matrix a block: G from its partial sums in block order, then M.
template <int RP> constexpr int kPolyThreads = RP == 64 ? 512 : NT;   // 8 of 64 x 64 elements a thread: the products
                                                                    // are bound by latency
template <int RP>
__global__ void __launch_bounds__(kPolyThreads<RP>) muon_poly_kernel(const __grid_constant__ Params p, int done, int steps) {
    using T = Tile<RP>;
    constexpr int LM = T::LM, PT = kPolyThreads<RP>;
    extern __shared__ __align__(16) float sh[];
    float *gm = sh, *sq = gm + RP * LM, *pm = sq + RP * LM, *mm = pm + RP * LM;
    __shared__ float s_inv;
    __shared__ uchar2 pairs[T::PAIRS];
    fill_pairs<RP>(pairs);
    const Mat &a = p.mat[blockIdx.x];
    const float *part = p.ws + a.part;
    const int nb = a.ctas;
    constexpr int OWN = (T::GSIZE + PT - 1) / PT, U = 6;     // U blocks of all own elements in flight
    float g[OWN] = {};
    for (int k = 0; k < nb; k += U) {
        float v[U][OWN];
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int o = 0; o < OWN; ++o) {
                const int e = threadIdx.x + o * PT;
                v[u][o] = k + u < nb && e < T::GSIZE ? part[int64_t(k + u) * T::GSIZE + e] : 0.f;
            }
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int o = 0; o < OWN; ++o) g[o] += v[u][o];
    }
    __syncthreads();
#pragma unroll
    for (int o = 0; o < OWN; ++o) {
        const int e = threadIdx.x + o * PT;
        if (e < T::GSIZE) {
            int i, k;
            if constexpr (RP == 64) block_place(pairs, e, i, k);
            else gram_place<RP>(pairs, e, i, k);
            gm[i * LM + k] = g[o];
            gm[k * LM + i] = g[o];
        }
    }
    __syncthreads();
    const float scale = done == 0 ? normalise<RP, PT>(gm, &s_inv, p.eps) : 1.f;
    polynomial<RP, PT>(gm, sq, pm, mm, steps, (a.r + 7) & ~7, p.a, p.b, p.c, scale);
    float *out = p.ws + p.mpoly + int64_t(blockIdx.x) * RP * RP;
    for (int e = threadIdx.x; e < RP * RP; e += PT) out[e] = mm[(e / RP) * LM + e % RP];
}

// ---------------------------------------------------------------- host side

int rank_class(int64_t r) { return r <= 8 ? 8 : r <= 16 ? 16 : r <= 32 ? 32 : 64; }

// Columns of a pass's tile, and a matrix's tiles.
template <int RP> constexpr int pass_columns() { return RP == 64 ? kTcJ : Tile<RP>::JT; }
template <int RP>
int64_t tiles_of(int64_t n) { return ceil_div(n, pass_columns<RP>()); }

// Column tiles a block takes: one, until that makes more than about 8 blocks an SM (fewer
// partial Gram matrices then), 8 at most.
int tiles_per_block(int64_t tiles) {
    const int64_t want = tiles / (int64_t(num_sms()) * 8);
    return int(std::min<int64_t>(8, std::max<int64_t>(1, want)));
}

// Puts the matrices `idx` into clusters: ctas[k], block0[k] for idx[k], which is sorted by
// block0.  All eight CTAs for a matrix while that leaves SMs free, for the shortest time; else
// as few as its columns fit, for the least work on the r x r products, the largest first, each
// into the first cluster with room.  Returns the CTAs in all.
template <int RP>
int place(const tlb_muon_mat *mats, int *idx, int n, int32_t *ctas, int32_t *block0) {
    auto need = [&](int i) { return int(ceil_div(std::max(mats[i].rows, mats[i].cols), Tile<RP>::JT)); };
    const bool all = int64_t(n) * kCluster <= 2 * num_sms();
    std::sort(idx, idx + n, [&](int x, int y) { return need(x) != need(y) ? need(x) > need(y) : x < y; });
    int used[kMaxMats], clusters = 0, order[kMaxMats];
    int32_t at[kMaxMats], size[kMaxMats];
    for (int k = 0; k < n; ++k) {
        const int c = all ? kCluster : need(idx[k]);
        int j = 0;
        while (j < clusters && used[j] + c > kCluster) ++j;
        if (j == clusters) used[clusters++] = 0;
        at[k] = j * kCluster + used[j];
        size[k] = c;
        used[j] += c;
        order[k] = k;
    }
    std::sort(order, order + n, [&](int x, int y) { return at[x] < at[y]; });
    int sorted[kMaxMats];
    for (int k = 0; k < n; ++k) {
        sorted[k] = idx[order[k]];
        ctas[k] = size[order[k]];
        block0[k] = at[order[k]];
    }
    std::copy(sorted, sorted + n, idx);
    return clusters * kCluster;
}

// Workspace floats of a group of matrices (the passes'): Y, the partial Gram matrices (as many
// as tiles, the most there can be) and the products M.
template <int RP>
size_t group_floats(const tlb_muon_mat *mats, const int *idx, int n) {
    size_t f = 0;
    for (int k = 0; k < n; ++k) {
        const int64_t tiles = tiles_of<RP>(std::max(mats[idx[k]].rows, mats[idx[k]].cols));
        f += size_t(tiles) * (RP * pass_columns<RP>() + Tile<RP>::GSIZE) + size_t(RP) * RP;
    }
    return f;
}

template <int RP, int SOURCE, int SINK>
int pass(const Params &p, unsigned blocks, cudaStream_t st) {
    if constexpr (RP == 64) {
        auto k = muon_tc_pass_kernel<SOURCE, SINK>;
        constexpr int smem = tc_smem<SOURCE, SINK>();
        TLB_CUDA(cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, smem));
        k<<<std::min<int>(p.tiles, tc_ctas<SOURCE, SINK>() * num_sms()), NT, smem, st>>>(p);
        return check_launch("muon_tc_pass");
    } else {
        constexpr int smem = pass_floats<RP>() * 4;
        auto k = muon_pass_kernel<RP, SOURCE, SINK>;
        TLB_CUDA(cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, smem));
        k<<<blocks, NT, smem, st>>>(p);
        return check_launch("muon_pass");
    }
}

template <int RP>
int group(const tlb_muon_mat *mats, int *idx, int n, bool clusters, const tlb_muon_cfg &cfg, float *ws, cudaStream_t st) {
    Params p;
    memset(&p, 0, sizeof(p));
    int64_t tiles = 0, off = 0, blocks = 0;
    for (int k = 0; k < n; ++k) tiles += tiles_of<RP>(std::max(mats[idx[k]].rows, mats[idx[k]].cols));
    int32_t ctas[kMaxMats], block0[kMaxMats];
    if (clusters) blocks = place<RP>(mats, idx, n, ctas, block0);
    p.tiles_per_block = RP == 64 ? 1 : tiles_per_block(tiles);
    p.tiles = int(tiles);
    p.nmat = n;
    p.ws = ws;
    p.status = reinterpret_cast<uint32_t *>(reinterpret_cast<char *>(ws) - kStatusBytes);
    p.mu = float(cfg.momentum);
    p.wd = float(cfg.weight_decay);
    p.nesterov = cfg.nesterov != 0;
    p.a = float(cfg.a);
    p.b = float(cfg.b);
    p.c = float(cfg.c);
    p.eps = float(cfg.eps);
    p.steps = cfg.steps;
    for (int k = 0; k < n; ++k) {
        const tlb_muon_mat &s = mats[idx[k]];
        Mat &a = p.mat[k];
        a.p = s.p;
        a.g = s.g;
        a.m = s.m;
        a.tall = s.rows > s.cols;
        a.r = std::min(s.rows, s.cols);
        a.n = std::max(s.rows, s.cols);
        a.vec = aligned16(s.p) && aligned16(s.g) && aligned16(s.m) && (a.tall ? a.r : a.n) % 4 == 0;
        a.lr = float(cfg.lr * double(s.lr_mult));
        a.lr_scale = float(cfg.lr * double(s.lr_mult) * double(s.scale));
        if (clusters) {
            a.ctas = ctas[k];
            a.block0 = block0[k];
        } else {
            a.ctas = int(ceil_div(tiles_of<RP>(a.n), p.tiles_per_block));
            a.block0 = int(blocks);
            blocks += a.ctas;
        }
        a.y = off;
        off += tiles_of<RP>(a.n) * RP * pass_columns<RP>();
        a.part = off;
        off += tiles_of<RP>(a.n) * Tile<RP>::GSIZE;
    }
    p.mpoly = off;
    if (clusters) {
        constexpr int smem = cluster_floats<RP>() * 4;
        auto k = muon_cluster_kernel<RP>;
        TLB_CUDA(cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, smem));
        cudaLaunchConfig_t lc = {};
        lc.gridDim = dim3(unsigned(blocks));
        lc.blockDim = dim3(NT);
        lc.dynamicSmemBytes = smem;
        lc.stream = st;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = kCluster;
        attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
        lc.attrs = attr;
        lc.numAttrs = 1;
        TLB_CUDA(cudaLaunchKernelEx(&lc, k, p));
        return check_launch("muon_cluster");
    }
    const unsigned grid = unsigned(blocks);
    constexpr int poly_smem = 4 * RP * Tile<RP>::LM * 4;
    TLB_CUDA(cudaFuncSetAttribute(muon_poly_kernel<RP>, cudaFuncAttributeMaxDynamicSharedMemorySize, poly_smem));
    TLB_TRY((pass<RP, kMomentum, kGram>(p, grid, st)));
    for (int done = 0; done < cfg.steps;) {
        const bool first = done == 0;
        const int steps = run_length(done, cfg.steps);
        muon_poly_kernel<RP><<<unsigned(n), kPolyThreads<RP>, poly_smem, st>>>(p, done, steps);
        TLB_TRY(check_launch("muon_poly"));
        done += steps;
        const bool last = done == cfg.steps;
        if (first) TLB_TRY((last ? pass<RP, kUpdate, kParam>(p, grid, st) : pass<RP, kUpdate, kGramY>(p, grid, st)));
        else TLB_TRY((last ? pass<RP, kY, kParam>(p, grid, st) : pass<RP, kY, kGramY>(p, grid, st)));
    }
    return TLB_OK;
}

template <typename F8, typename F16, typename F32, typename F64>
auto by_class(int rp, F8 f8, F16 f16, F32 f32, F64 f64) {
    return rp == 8 ? f8() : rp == 16 ? f16() : rp == 32 ? f32() : f64();
}

// Whether a matrix goes to a cluster: X fits its shared memory.  Every CTA of the cluster forms
// the r x r products for itself, which for r > 32 is as much work as the passes' (3.7 M FMAs a
// CTA), so there only up to a matrix for every eight SMs, where the SMs would be idle.
bool in_cluster(const tlb_muon_mat &s, int rp, int64_t of_class) {
    const int64_t cap = kCluster * (rp == 8 ? Tile<8>::JT : rp == 16 ? Tile<16>::JT : rp == 32 ? Tile<32>::JT : Tile<64>::JT);
    return std::max(s.rows, s.cols) <= cap && (rp <= 32 || of_class * kCluster <= num_sms());
}

// Calls f(class, clusters, indices, count) for groups of at most kMaxMats matrices of one class
// and way.
template <typename F>
int for_groups(const tlb_muon_mat *mats, int32_t n, F f) {
    int idx[kMaxMats];
    for (int rp = 8; rp <= 64; rp *= 2) {
        auto here = [&](int i) {
            return mats[i].rows > 0 && mats[i].cols > 0 && rank_class(std::min(mats[i].rows, mats[i].cols)) == rp;
        };
        int64_t of_class = 0;
        for (int i = 0; i < n; ++i) of_class += here(i);
        for (int way = 0; of_class > 0 && way < 2; ++way) {
            int k = 0;
            for (int i = 0; i < n; ++i) {
                if (!here(i) || in_cluster(mats[i], rp, of_class) != (way == 0)) continue;
                idx[k++] = i;
                if (k == kMaxMats) {
                    TLB_TRY(f(rp, way == 0, idx, k));
                    k = 0;
                }
            }
            if (k > 0) TLB_TRY(f(rp, way == 0, idx, k));
        }
    }
    return TLB_OK;
}

int check_mats(const char *fn, const tlb_muon_mat *mats, int32_t n) {
    TLB_REQUIRE(n >= 0 && (mats != nullptr || n == 0), TLB_EINVAL, "%s: needs n >= 0 matrices", fn);
    for (int i = 0; i < n; ++i) {
        TLB_REQUIRE(mats[i].rows >= 0 && mats[i].cols >= 0, TLB_EINVAL, "%s: matrix %d: negative size", fn, i);
        TLB_REQUIRE(std::min(mats[i].rows, mats[i].cols) <= 64, TLB_EUNSUPPORTED,
                    "%s: matrix %d: the smaller side is at most 64 (the adapters' largest rank)", fn, i);
        TLB_REQUIRE(std::max(mats[i].rows, mats[i].cols) <= (1 << 24), TLB_EUNSUPPORTED,
                    "%s: matrix %d: the larger side is at most 2^24", fn, i);
    }
    return TLB_OK;
}

// The groups run one after another, so they share the workspace.
int ws_floats(const tlb_muon_mat *mats, int32_t n, size_t &most) {
    most = 0;
    return for_groups(mats, n, [&](int rp, bool clusters, const int *idx, int k) {
        (void)clusters;                                      // which need none; the size does not tell
        most = std::max(most, by_class(rp, [&] { return group_floats<8>(mats, idx, k); },
                                       [&] { return group_floats<16>(mats, idx, k); },
                                       [&] { return group_floats<32>(mats, idx, k); },
                                       [&] { return group_floats<64>(mats, idx, k); }));
        return TLB_OK;
    });
}

}  // namespace

}  // namespace tlb

using namespace tlb;

extern "C" {

size_t tlb_muon_workspace_bytes(const tlb_muon_mat *mats, int32_t n) {
    clear_error();
    size_t f = 0;
    if (check_mats("muon_workspace_bytes", mats, n) != TLB_OK || ws_floats(mats, n, f) != TLB_OK) return 0;
    return kStatusBytes + f * 4;
}

int tlb_muon(const tlb_muon_mat *mats, int32_t n, const tlb_muon_cfg *cfg, void *ws, size_t ws_bytes, void *stream) {
    clear_error();
    TLB_REQUIRE(cfg != nullptr, TLB_EINVAL, "muon: null cfg");
    TLB_REQUIRE(cfg->steps >= 1 && cfg->steps <= 100, TLB_EINVAL, "muon: steps must be 1 to 100");
    TLB_REQUIRE(cfg->eps >= 0.0, TLB_EINVAL, "muon: eps must be >= 0");
    TLB_TRY(check_mats("muon", mats, n));
    for (int i = 0; i < n; ++i)
        TLB_REQUIRE(mats[i].rows == 0 || mats[i].cols == 0 || (mats[i].p && mats[i].g && mats[i].m), TLB_EINVAL,
                    "muon: matrix %d: null pointer", i);
    size_t f = 0;
    TLB_TRY(ws_floats(mats, n, f));
    if (f == 0) return TLB_OK;
    TLB_REQUIRE(ws != nullptr && (reinterpret_cast<uintptr_t>(ws) & 255) == 0 && ws_bytes >= kStatusBytes + f * 4, TLB_EINVAL,
                "muon: needs a 256-byte aligned workspace of %zu bytes", kStatusBytes + f * 4);
    float *w = ws_at<float>(ws, kStatusBytes);
    cudaStream_t st = as_stream(stream);
    return for_groups(mats, n, [&](int rp, bool clusters, int *idx, int k) {
        return by_class(rp, [&] { return group<8>(mats, idx, k, clusters, *cfg, w, st); },
                        [&] { return group<16>(mats, idx, k, clusters, *cfg, w, st); },
                        [&] { return group<32>(mats, idx, k, clusters, *cfg, w, st); },
                        [&] { return group<64>(mats, idx, k, clusters, *cfg, w, st); });
    });
}

}  // extern "C"
