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
// Launches for five steps, over all matrices of a rank class together (class: r rounded up to
// 8, 16, 32 or 64):
//   pass   m', u = f(g, m); partial Gram matrices of column chunks
//   poly   sums them in order, |u|_F from the trace, two steps' product M
//   pass   u again from g and m'; Y = M u to the workspace; partial Gram matrices of Y
//   poly   three steps' product M
//   pass   X = M Y; p updated
// Bounds: HBM for r <= 16 (20 bytes an element that must move; g and m' a second time and Y
// come from L2 while they fit it), fp32 FMAs for r = 64 (3 r of them an element and pass pair).
#include <algorithm>
#include <cmath>
#include <cstring>

#include "common.cuh"
#include "kernels.cuh"
#include "tc.cuh"

namespace tlb {

namespace {

constexpr int kMaxMats = 256;            // matrices of one launch (their table is a kernel parameter)
constexpr int kFirstRun = 2, kRun = 3;    // steps from the first and from each later Gram matrix
constexpr int kCluster = 8;              // CTAs that hold one matrix
constexpr int kPassThreads = 128, kPolyThreads = 256, kClusterThreads = 256;

struct Mat {
    float *p, *m;
    const float *g;
    int64_t y, part;                     // offsets in the workspace, in floats: Y tiles, partial Gram matrices
    int32_t r, n;
    int32_t tall;                        // stored [n, r] (else [r, n])
    int32_t vec;                         // 16-byte accesses (aligned; r % 4 == 0 of a tall one, n % 4 == 0 of a wide one)
    int32_t block0;                      // first block of this matrix (multi-pass)
    float lr, lr_scale;                  // lr lr_mult, and times scale
};

struct Params {
    Mat mat[kMaxMats];
    int nmat, tiles_per_block;
    float *ws;
    int64_t mpoly;                       // offset of the products M [nmat][RP * RP]
    float mu, wd;
    int nesterov;
    float a, b, c, eps;                  // Newton-Schulz
    int steps;
};

// What a pass reads, and what it does with X.
enum Source { kMomentum = 0, kUpdate = 1, kY = 2 };   // m' and u; u from g and m'; Y
enum Sink { kGram = 0, kGramY = 1, kParam = 2 };      // Gram matrix; X to Y and its Gram matrix; p

// A tile of up to JT columns of X [r, n], in shared memory as [RP][LD]: 33 KB for r <= 16, 66
// KB above.  LD = JT + 4: the same column of eight neighbouring rows lies in eight different
// groups of four banks.
template <int RP> struct Tile {
    static constexpr int JT = RP == 8 ? 1024 : RP == 64 ? 256 : 512;
    static constexpr int LD = JT + 4, XF = RP * LD;
    static constexpr int LM = RP + 4;                       // row length of an r x r matrix in shared memory
    // Gram blocks of B x B a thread (row k of block b is b + NB k); the upper PAIRS of them
    static constexpr int B = RP == 64 ? 8 : 4, NB = RP / B, PAIRS = NB * (NB + 1) / 2;
    static constexpr int GSIZE = PAIRS * B * B;             // floats of a Gram matrix's upper blocks
};
// NT threads form a Gram matrix in GROUPS groups, each with every GROUPS-th column quad; RG of
// them at a time meet in a buffer of at most 9 KB.
template <int RP, int NT> struct Gram {
    static constexpr int G0 = NT / Tile<RP>::PAIRS, GROUPS = G0 > 32 ? 32 : G0;
    static constexpr int R0 = 9216 / (Tile<RP>::GSIZE * 4), RG = R0 < 1 ? 1 : R0 > GROUPS ? GROUPS : R0;
    static constexpr int RF = RG * Tile<RP>::GSIZE;         // floats of the buffer
    static constexpr int OWN = (Tile<RP>::GSIZE + NT - 1) / NT;
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

// Walks through a tile's elements (columns j0 .. j0 + jn) in pieces of cnt <= 4 that are
// contiguous in memory: f(offset of the first, its place in the tile, places' step, cnt) for U
// pieces at once, so that their loads are in flight together.
template <int RP, int NT, int U, typename F>
__device__ __forceinline__ void visit(const Mat &a, int j0, int jn, F f) {
    constexpr int LD = Tile<RP>::LD;
    int64_t e[U];
    int at[U], cnt[U];
    auto divide = [](uint32_t x, uint32_t magic, int d) { return d > 1 ? int(__umulhi(x, magic)) : int(x); };
    auto magic_of = [](int d) { return 0xFFFFFFFFu / uint32_t(d) + 1u; };           // exact below 2^16
    if (a.tall && a.vec) {
        // a warp takes 8 columns x 16 rows: 64 contiguous bytes a column
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
        const int rq = a.r / 4, rb = (rq + 3) / 4, units = ((jn + 7) / 8) * rb;
        for (int q0 = warp; q0 < units; q0 += U * (NT / 32)) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int q = q0 + u * (NT / 32), jb = q / rb;
                const int j = jb * 8 + (lane >> 2), iq = (q - jb * rb) * 4 + (lane & 3);
                cnt[u] = q < units && j < jn && iq < rq ? 4 : 0;
                e[u] = int64_t(j0 + j) * a.r + iq * 4;
                at[u] = iq * 4 * LD + j;
            }
            f(e, at, LD, cnt);
        }
    } else if (a.tall) {
        const int total = jn * a.r;
        const uint32_t magic = magic_of(a.r);
        for (int q0 = threadIdx.x; q0 < total; q0 += U * NT) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int q = q0 + u * NT, j = divide(uint32_t(q), magic, a.r);
                cnt[u] = q < total ? 1 : 0;
                e[u] = int64_t(j0) * a.r + q;
                at[u] = (q - j * a.r) * LD + j;
            }
            f(e, at, 0, cnt);
        }
    } else {
        const int step = a.vec ? 4 : 1, w = (jn + step - 1) / step, total = w * a.r;   // vec: jn % 4 == 0
        const uint32_t magic = magic_of(w);
        for (int q0 = threadIdx.x; q0 < total; q0 += U * NT) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int q = q0 + u * NT, i = divide(uint32_t(q), magic, w), j = (q - i * w) * step;
                cnt[u] = q < total ? step : 0;
                e[u] = int64_t(i) * a.n + j0 + j;
                at[u] = i * LD + j;
            }
            f(e, at, 1, cnt);
        }
    }
}

__device__ __forceinline__ void load4(const float *p, int64_t e, int cnt, float (&v)[4]) {
    if (cnt == 4) {
        const float4 x = *reinterpret_cast<const float4 *>(p + e);
        v[0] = x.x; v[1] = x.y; v[2] = x.z; v[3] = x.w;
    } else {
        v[0] = cnt > 0 ? p[e] : 0.f;
    }
}
__device__ __forceinline__ void keep4(float *p, int64_t e, int cnt, const float (&v)[4]) {
    if (cnt == 4) *reinterpret_cast<float4 *>(p + e) = make_float4(v[0], v[1], v[2], v[3]);
    else if (cnt > 0) p[e] = v[0];
}

// Rows past r, and columns jn .. up to a whole quad, count as 0.
template <int RP, int NT>
__device__ __forceinline__ void clear_rest(const Mat &a, float *x, int jn) {
    constexpr int LD = Tile<RP>::LD;
    const int j4 = (jn + 3) & ~3;
    for (int k = threadIdx.x; k < (RP - a.r) * j4; k += NT) x[(a.r + k / j4) * LD + k % j4] = 0.f;
    if (j4 > jn)
        for (int k = threadIdx.x; k < a.r * (j4 - jn); k += NT) x[(k / (j4 - jn)) * LD + jn + k % (j4 - jn)] = 0.f;
}

// The tile of u, from g and the momentum, which FIRST brings up to date.
template <int RP, int NT, bool FIRST>
__device__ __forceinline__ void load_update(const Params &p, const Mat &a, float *x, int j0, int jn) {
    constexpr int U = 4;
    clear_rest<RP, NT>(a, x, jn);
    visit<RP, NT, U>(a, j0, jn, [&](const int64_t (&e)[U], const int (&at)[U], int step, const int (&cnt)[U]) {
        float g[U][4], m[U][4];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            load4(a.g, e[u], cnt[u], g[u]);
            load4(a.m, e[u], cnt[u], m[u]);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if constexpr (FIRST) {
#pragma unroll
                for (int c = 0; c < 4; ++c) m[u][c] = fmaf(p.mu, m[u][c], g[u][c]);
                keep4(a.m, e[u], cnt[u], m[u]);
            }
#pragma unroll
            for (int c = 0; c < 4; ++c)
                if (c < cnt[u]) x[at[u] + c * step] = p.nesterov ? fmaf(p.mu, m[u][c], g[u][c]) : m[u][c];
        }
    });
}

// p moved along the tile.
template <int RP, int NT>
__device__ __forceinline__ void move_params(const Params &p, const Mat &a, const float *x, int j0, int jn) {
    constexpr int U = 4;
    visit<RP, NT, U>(a, j0, jn, [&](const int64_t (&e)[U], const int (&at)[U], int step, const int (&cnt)[U]) {
        float v[U][4];
#pragma unroll
        for (int u = 0; u < U; ++u) load4(a.p, e[u], cnt[u], v[u]);
#pragma unroll
        for (int u = 0; u < U; ++u) {
#pragma unroll
            for (int c = 0; c < 4; ++c)
                if (c < cnt[u]) v[u][c] -= a.lr * p.wd * v[u][c] + a.lr_scale * x[at[u] + c * step];
            keep4(a.p, e[u], cnt[u], v[u]);
        }
    });
}

// X <- M X on the shared tile: a thread takes two columns whole into registers, so the product
// goes back in place without a barrier.  mt: M's columns as rows (the same for all threads).
template <int RP, int NT>
__device__ __forceinline__ void apply(float *x, const float *mt, int jn) {
    constexpr int LD = Tile<RP>::LD, LM = Tile<RP>::LM;
#pragma unroll 1
    for (int j = 2 * threadIdx.x; j < jn; j += 2 * NT) {
        float2 v[RP];
#pragma unroll
        for (int k = 0; k < RP; ++k) v[k] = *reinterpret_cast<const float2 *>(x + k * LD + j);
#pragma unroll 1
        for (int i = 0; i < RP; i += 4) {
            float2 y[4];
#pragma unroll
            for (int d = 0; d < 4; ++d) y[d] = make_float2(0.f, 0.f);
#pragma unroll
            for (int k = 0; k < RP; ++k) {
                const float4 w = *reinterpret_cast<const float4 *>(mt + k * LM + i);
                y[0].x = fmaf(w.x, v[k].x, y[0].x); y[0].y = fmaf(w.x, v[k].y, y[0].y);
                y[1].x = fmaf(w.y, v[k].x, y[1].x); y[1].y = fmaf(w.y, v[k].y, y[1].y);
                y[2].x = fmaf(w.z, v[k].x, y[2].x); y[2].y = fmaf(w.z, v[k].y, y[2].y);
                y[3].x = fmaf(w.w, v[k].x, y[3].x); y[3].y = fmaf(w.w, v[k].y, y[3].y);
            }
#pragma unroll
            for (int d = 0; d < 4; ++d) *reinterpret_cast<float2 *>(x + (i + d) * LD + j) = y[d];
        }
    }
}

// This thread's share of the tile's Gram matrix added to acc: block (bi, bk) over the column
// quads grp, grp + GROUPS, ...
template <int RP, int NT>
__device__ __forceinline__ void gram_add(const float *x, int jn, float (&acc)[Tile<RP>::B][Tile<RP>::B]) {
    using T = Tile<RP>;
    constexpr int B = T::B, NB = T::NB, LD = T::LD;
    const int grp = threadIdx.x / T::PAIRS;
    if (grp >= Gram<RP, NT>::GROUPS) return;
    int bi, bk;
    pair_of<NB>(threadIdx.x % T::PAIRS, bi, bk);
    const int quads = (jn + 3) / 4;
#pragma unroll 1
    for (int q = grp; q < quads; q += Gram<RP, NT>::GROUPS) {
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

// The groups' shares added up in group order: out[e] = sum of element e (e < GSIZE, in the
// order [pair][B * B]); red: Gram::RF floats.
template <int RP, int NT>
__device__ __forceinline__ void gram_sum(const float (&acc)[Tile<RP>::B][Tile<RP>::B], float *red, float *out) {
    using T = Tile<RP>;
    using G = Gram<RP, NT>;
    constexpr int B = T::B;
    const int grp = threadIdx.x / T::PAIRS, pair = threadIdx.x % T::PAIRS;
    float s[G::OWN];
#pragma unroll
    for (int o = 0; o < G::OWN; ++o) s[o] = 0.f;
#pragma unroll 1
    for (int g0 = 0; g0 < G::GROUPS; g0 += G::RG) {
        __syncthreads();
        if (grp >= g0 && grp < g0 + G::RG && grp < G::GROUPS) {
#pragma unroll
            for (int k = 0; k < B * B; ++k) red[(grp - g0) * T::GSIZE + k * T::PAIRS + pair] = acc[k / B][k % B];
        }
        __syncthreads();
        const int n = min(G::RG, G::GROUPS - g0);
#pragma unroll
        for (int o = 0; o < G::OWN; ++o) {
            const int e = threadIdx.x + o * NT;
            if (e < T::GSIZE)
                for (int k = 0; k < n; ++k) s[o] += red[k * T::GSIZE + e];
        }
    }
#pragma unroll
    for (int o = 0; o < G::OWN; ++o) {
        const int e = threadIdx.x + o * NT;
        if (e < T::GSIZE) out[e] = s[o];
    }
}

// Element e of [B * B][pair]: its row and column.
template <int RP>
__device__ __forceinline__ void gram_place(int e, int &i, int &k) {
    using T = Tile<RP>;
    int bi, bk;
    pair_of<T::NB>(e % T::PAIRS, bi, bk);
    const int q = e / T::PAIRS;
    i = bi + T::NB * (q / T::B);
    k = bk + T::NB * (q % T::B);
}

// The product of `steps` Newton-Schulz polynomials P of G, times `scale`, in mm.  gm: G
// (symmetric; changed); sq, pm: scratch; all [RP][LM].  G and P are symmetric: a row stands
// for a column.  Called by NT threads, D x D elements each.
template <int RP, int NT>
__device__ __forceinline__ void polynomial(float *gm, float *sq, float *pm, float *mm, int steps, float a, float b, float c,
                                           float scale) {
    constexpr int LM = Tile<RP>::LM;
    constexpr int D = RP == 64 ? 4 : RP == 32 ? 2 : 1, W = RP / D;
    static_assert(W * W <= NT, "threads of a product");
    const int tid = threadIdx.x, r0 = (tid / W) * D, c0 = (tid % W) * D;
    const bool on = tid < W * W;
    // out = f(sum_k x[k][r] y[k][c])
    auto product = [&](const float *x, const float *y, float *out, auto f) {
        float acc[D][D];
#pragma unroll
        for (int s = 0; s < D; ++s)
#pragma unroll
            for (int t = 0; t < D; ++t) acc[s][t] = 0.f;
        if (on) {
#pragma unroll 8
            for (int k = 0; k < RP; ++k) {
                float u[D], v[D];
                if constexpr (D == 4) {
                    const float4 q = *reinterpret_cast<const float4 *>(x + k * LM + r0), w = *reinterpret_cast<const float4 *>(y + k * LM + c0);
                    u[0] = q.x; u[1] = q.y; u[2] = q.z; u[3] = q.w;
                    v[0] = w.x; v[1] = w.y; v[2] = w.z; v[3] = w.w;
                } else if constexpr (D == 2) {
                    const float2 q = *reinterpret_cast<const float2 *>(x + k * LM + r0), w = *reinterpret_cast<const float2 *>(y + k * LM + c0);
                    u[0] = q.x; u[1] = q.y;
                    v[0] = w.x; v[1] = w.y;
                } else {
                    u[0] = x[k * LM + r0];
                    v[0] = y[k * LM + c0];
                }
#pragma unroll
                for (int s = 0; s < D; ++s)
#pragma unroll
                    for (int t = 0; t < D; ++t) acc[s][t] = fmaf(u[s], v[t], acc[s][t]);
            }
        }
        __syncthreads();                                     // out may be x or y
        if (on) {
#pragma unroll
            for (int s = 0; s < D; ++s)
#pragma unroll
                for (int t = 0; t < D; ++t) out[(r0 + s) * LM + c0 + t] = f(acc[s][t], r0 + s, c0 + t);
        }
        __syncthreads();
    };
    auto same = [](float v, int, int) { return v; };
    for (int s = 0; s < steps; ++s) {
        // the first P is the product so far, and carries the scale; P itself is needed without
        // it while G goes on
        product(gm, gm, pm, [&](float v, int i, int k) { return fmaf(c, v, fmaf(b, gm[i * LM + k], i == k ? a : 0.f)); });
        if (s == 0) {
            if (on) {
#pragma unroll
                for (int u = 0; u < D; ++u)
#pragma unroll
                    for (int t = 0; t < D; ++t) mm[(r0 + u) * LM + c0 + t] = pm[(r0 + u) * LM + c0 + t] * scale;
            }
            __syncthreads();
        } else {
            product(pm, mm, mm, same);
        }
        if (s + 1 < steps) {
            // G of the next X: P G P with one factor on either side, made symmetric again
            // (G P P, equal but for rounding, or a G left unsymmetric, cost a digit in X)
            product(gm, pm, sq, same);                       // G P
            product(sq, pm, gm, same);                       // (G P)^T P
            for (int e = tid; e < RP * RP; e += NT) {
                const int i = e / RP, k = e % RP;
                if (i < k) gm[i * LM + k] = gm[k * LM + i] = 0.5f * (gm[i * LM + k] + gm[k * LM + i]);
            }
            __syncthreads();
        }
    }
}

// 1 / (|u|_F + eps) from the Gram matrix of u, which becomes that of X0.  A zero update stays
// zero, also for eps = 0.
template <int RP, int NT>
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
    for (int e = threadIdx.x; e < RP * RP; e += NT) gm[(e / RP) * LM + e % RP] *= inv * inv;
    __syncthreads();
    return inv;
}

__device__ __forceinline__ float ld_cluster(const float *p, int rank) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(cluster_addr(p, uint32_t(rank))) : "memory");
    return v;
}

// ---------------------------------------------------------------- one matrix a cluster

// The whole step of a matrix whose X fits the shared memory of kCluster CTAs: CTA c holds
// columns [c w, (c + 1) w).  X never leaves the SMs: 20 bytes an element cross, as they must.
// Gram matrices are summed over the cluster through distributed shared memory, by every CTA in
// rank order, and every CTA forms the r x r products for itself.
template <int RP> constexpr int cluster_floats() {
    return Tile<RP>::XF + Gram<RP, kClusterThreads>::RF + 2 * Tile<RP>::GSIZE + 4 * RP * Tile<RP>::LM;
}

template <int RP>
__global__ void __launch_bounds__(kClusterThreads) muon_cluster_kernel(const __grid_constant__ Params p) {
    using T = Tile<RP>;
    constexpr int NT = kClusterThreads, LM = T::LM, B = T::B;
    extern __shared__ __align__(16) float sh[];
    float *x = sh, *gm = x + T::XF, *sq = gm + RP * LM, *pm = sq + RP * LM, *mm = pm + RP * LM;
    float *part = mm + RP * LM, *red = part + 2 * T::GSIZE;  // part: two, for alternate runs
    __shared__ float s_inv;
    const Mat &a = p.mat[blockIdx.x / kCluster];
    const int rank = int(cluster_rank());
    const int w = ((a.n + kCluster - 1) / kCluster + 3) & ~3;
    const int j0 = min(a.n, rank * w), jn = min(w, a.n - j0);
    load_update<RP, NT, true>(p, a, x, j0, jn);
    float scale = 1.f;
    for (int done = 0, run = 0; done < p.steps; ++run) {
        __syncthreads();
        float acc[B][B];
#pragma unroll
        for (int k = 0; k < B * B; ++k) acc[k / B][k % B] = 0.f;
        gram_add<RP, NT>(x, jn, acc);
        float *mine = part + (run & 1) * T::GSIZE;
        gram_sum<RP, NT>(acc, red, mine);
        cluster_sync();
        for (int e = threadIdx.x; e < T::GSIZE; e += NT) {
            float v[kCluster], s = 0.f;
#pragma unroll
            for (int c = 0; c < kCluster; ++c) v[c] = ld_cluster(mine + e, c);
#pragma unroll
            for (int c = 0; c < kCluster; ++c) s += v[c];
            int i, k;
            gram_place<RP>(e, i, k);
            gm[i * LM + k] = s;
            gm[k * LM + i] = s;
        }
        __syncthreads();
        if (run == 0) scale = normalise<RP, NT>(gm, &s_inv, p.eps);
        const int steps = min(run == 0 ? kFirstRun : kRun, p.steps - done);
        polynomial<RP, NT>(gm, sq, pm, mm, steps, p.a, p.b, p.c, run == 0 ? scale : 1.f);
        done += steps;
        apply<RP, NT>(x, mm, jn);
    }
    __syncthreads();
    move_params<RP, NT>(p, a, x, j0, jn);
    cluster_sync();                                          // peers have read the last partial sums
}

// ---------------------------------------------------------------- passes over longer matrices

template <int RP> constexpr int pass_floats() {
    return Tile<RP>::XF + Gram<RP, kPassThreads>::RF + RP * Tile<RP>::LM;
}

template <int RP, int SOURCE, int SINK>
__global__ void __launch_bounds__(kPassThreads) muon_pass_kernel(const __grid_constant__ Params p) {
    using T = Tile<RP>;
    constexpr int NT = kPassThreads, JT = T::JT, LD = T::LD, LM = T::LM, B = T::B;
    extern __shared__ __align__(16) float sh[];
    float *x = sh, *mt = x + T::XF, *red = mt + RP * LM;
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
    float acc[B][B];
#pragma unroll
    for (int k = 0; k < B * B; ++k) acc[k / B][k % B] = 0.f;
    for (int t = t0; t < t1; ++t) {
        const int j0 = t * JT, jn = min(JT, a.n - j0);
        float *y = p.ws + a.y + int64_t(t) * RP * JT;       // this tile of Y: [RP][JT]
        __syncthreads();                                    // the last tile is used up (and M is there)
        if constexpr (SOURCE == kY) {
            for (int k = threadIdx.x; k < RP * (JT / 4); k += NT)
                *reinterpret_cast<float4 *>(x + (k / (JT / 4)) * LD + (k % (JT / 4)) * 4) = reinterpret_cast<const float4 *>(y)[k];
        } else {
            load_update<RP, NT, SOURCE == kMomentum>(p, a, x, j0, jn);
        }
        __syncthreads();
        if constexpr (SOURCE != kMomentum) {
            apply<RP, NT>(x, mt, jn);
            __syncthreads();
        }
        if constexpr (SINK == kParam) {
            move_params<RP, NT>(p, a, x, j0, jn);
        } else {
            if constexpr (SINK == kGramY) {
                const int jq = (jn + 3) / 4;
                for (int k = threadIdx.x; k < RP * jq; k += NT)
                    *reinterpret_cast<float4 *>(y + (k / jq) * JT + (k % jq) * 4) =
                        *reinterpret_cast<const float4 *>(x + (k / jq) * LD + (k % jq) * 4);
            }
            gram_add<RP, NT>(x, jn, acc);
        }
    }
    if constexpr (SINK != kParam) gram_sum<RP, NT>(acc, red, p.ws + a.part + int64_t(bl) * T::GSIZE);
}

// One matrix a block: G from its partial sums in block order, then M.
template <int RP>
__global__ void __launch_bounds__(kPolyThreads) muon_poly_kernel(const __grid_constant__ Params p, int done, int steps) {
    using T = Tile<RP>;
    constexpr int LM = T::LM, NT = kPolyThreads;
    extern __shared__ __align__(16) float sh[];
    float *gm = sh, *sq = gm + RP * LM, *pm = sq + RP * LM, *mm = pm + RP * LM;
    __shared__ float s_inv;
    const Mat &a = p.mat[blockIdx.x];
    const float *part = p.ws + a.part;
    const int nb = ((a.n + T::JT - 1) / T::JT + p.tiles_per_block - 1) / p.tiles_per_block;
    for (int e = threadIdx.x; e < T::GSIZE; e += NT) {
        float s = 0.f;
        for (int k = 0; k < nb; k += 8) {
            float v[8];
#pragma unroll
            for (int u = 0; u < 8; ++u) v[u] = k + u < nb ? part[int64_t(k + u) * T::GSIZE + e] : 0.f;
#pragma unroll
            for (int u = 0; u < 8; ++u) s += v[u];
        }
        int i, k;
        gram_place<RP>(e, i, k);
        gm[i * LM + k] = s;
        gm[k * LM + i] = s;
    }
    __syncthreads();
    const float scale = done == 0 ? normalise<RP, NT>(gm, &s_inv, p.eps) : 1.f;
    polynomial<RP, NT>(gm, sq, pm, mm, steps, p.a, p.b, p.c, scale);
    float *out = p.ws + p.mpoly + int64_t(blockIdx.x) * RP * RP;
    for (int e = threadIdx.x; e < RP * RP; e += NT) out[e] = mm[(e / RP) * LM + e % RP];
}

// ---------------------------------------------------------------- host side

int rank_class(int64_t r) { return r <= 8 ? 8 : r <= 16 ? 16 : r <= 32 ? 32 : 64; }

template <int RP>
int64_t tiles_of(int64_t n) { return ceil_div(n, Tile<RP>::JT); }

// Column tiles a block takes: one, until that makes more than about 8 blocks an SM (fewer
// partial Gram matrices then), 8 at most.
int tiles_per_block(int64_t tiles) {
    const int64_t want = tiles / (int64_t(num_sms()) * 8);
    return int(std::min<int64_t>(8, std::max<int64_t>(1, want)));
}

// Workspace floats of a group of matrices (the passes'): Y, the partial Gram matrices (as many
// as tiles, the most there can be) and the products M.
template <int RP>
size_t group_floats(const tlb_muon_mat *mats, const int *idx, int n) {
    size_t f = 0;
    for (int k = 0; k < n; ++k) {
        const int64_t tiles = tiles_of<RP>(std::max(mats[idx[k]].rows, mats[idx[k]].cols));
        f += size_t(tiles) * (RP * Tile<RP>::JT + Tile<RP>::GSIZE) + size_t(RP) * RP;
    }
    return f;
}

template <int RP, int SOURCE, int SINK>
int pass(const Params &p, unsigned blocks, cudaStream_t st) {
    constexpr int smem = pass_floats<RP>() * 4;
    auto k = muon_pass_kernel<RP, SOURCE, SINK>;
    TLB_CUDA(cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, smem));
    k<<<blocks, kPassThreads, smem, st>>>(p);
    return check_launch("muon_pass");
}

template <int RP>
int group(const tlb_muon_mat *mats, const int *idx, int n, bool clusters, const tlb_muon_cfg &cfg, float *ws, cudaStream_t st) {
    Params p;
    memset(&p, 0, sizeof(p));
    int64_t tiles = 0, off = 0, blocks = 0;
    for (int k = 0; k < n; ++k) tiles += tiles_of<RP>(std::max(mats[idx[k]].rows, mats[idx[k]].cols));
    p.tiles_per_block = tiles_per_block(tiles);
    p.nmat = n;
    p.ws = ws;
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
        a.block0 = int(blocks);
        blocks += ceil_div(tiles_of<RP>(a.n), p.tiles_per_block);
        a.y = off;
        off += tiles_of<RP>(a.n) * RP * Tile<RP>::JT;
        a.part = off;
        off += tiles_of<RP>(a.n) * Tile<RP>::GSIZE;
    }
    p.mpoly = off;
    if (clusters) {
        constexpr int smem = cluster_floats<RP>() * 4;
        auto k = muon_cluster_kernel<RP>;
        TLB_CUDA(cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, smem));
        cudaLaunchConfig_t lc = {};
        lc.gridDim = dim3(unsigned(n * kCluster));
        lc.blockDim = dim3(kClusterThreads);
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
        const int steps = std::min(first ? kFirstRun : kRun, cfg.steps - done);
        muon_poly_kernel<RP><<<unsigned(n), kPolyThreads, poly_smem, st>>>(p, done, steps);
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
    return for_groups(mats, n, [&](int rp, bool clusters, const int *idx, int k) {
        return by_class(rp, [&] { return group<8>(mats, idx, k, clusters, *cfg, w, st); },
                        [&] { return group<16>(mats, idx, k, clusters, *cfg, w, st); },
                        [&] { return group<32>(mats, idx, k, clusters, *cfg, w, st); },
                        [&] { return group<64>(mats, idx, k, clusters, *cfg, w, st); });
    });
}

}  // extern "C"
