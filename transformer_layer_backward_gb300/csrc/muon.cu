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

namespace tlb {

namespace {

constexpr int kThreads = 128;
constexpr int kMaxMats = 256;            // matrices of one launch (their table is a kernel parameter)
constexpr int kFirstRun = 2, kRun = 3;    // steps from the first and from each later Gram matrix
constexpr int kPolyThreads = 256;

struct Mat {
    float *p, *m;
    const float *g;
    int64_t y, part;                     // offsets in the workspace, in floats: Y [n][RP], partial Gram matrices
    int32_t r, n;
    int32_t tall;                        // stored [n, r] (else [r, n])
    int32_t vec;                         // 16-byte accesses (aligned; wide: n % 4 == 0)
    int32_t block0;                      // first block of this matrix
    float lr, lr_scale;                  // lr lr_mult, and times scale
};

struct Params {
    Mat mat[kMaxMats];
    int nmat, tiles_per_block;
    float *ws;
    int64_t mpoly;                       // offset of the products M [nmat][RP * RP]
    float mu, wd;
    int nesterov;
};

// What a pass reads, and what it does with X.
enum Source { kMomentum = 0, kUpdate = 1, kY = 2 };   // m' and u; u from g and m'; Y
enum Sink { kGram = 0, kGramY = 1, kParam = 2 };      // Gram matrix; X to Y and its Gram matrix; p

// Column (of the [r, n] form) tile: JT columns, JC a thread.
template <int RP> struct Tile {
    static constexpr int JC = RP >= 32 ? 2 : 4, JT = JC * kThreads;
    static constexpr int LD = RP + 4;                       // floats of a column in shared memory: 16-byte
                                                            // accesses of consecutive columns meet no bank twice
    static constexpr int B = RP >= 32 ? 8 : 4;              // Gram blocks of B x B a thread
    static constexpr int NB = RP / B, PAIRS = NB * (NB + 1) / 2;
    static constexpr int GROUPS = kThreads / PAIRS;         // threads that share a block, each every GROUPS-th column
    static constexpr int GSIZE = PAIRS * B * B;             // floats of one partial Gram matrix (upper blocks)
    static constexpr int HALF = GROUPS > 32 ? 32 : GROUPS > 16 ? 16 : GROUPS > 8 ? 8 : GROUPS > 4 ? 4 : GROUPS > 2 ? 2 : 1;
    static constexpr int XF = JT * LD;                      // X, then the scratch of the groups' sum
    static constexpr int SMEM = (XF > HALF * GSIZE ? XF : HALF * GSIZE) + RP * LD;
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

// Walks through a tile's elements (columns j0 .. j0 + jn) in pieces of up to four that are
// contiguous in memory: f(offset of the first, its local column, its row, step along columns,
// count).  U pieces are handed over together, so that their loads are in flight together.
template <int RP, int U, typename F>
__device__ __forceinline__ void visit(const Mat &a, int j0, int jn, F f) {
    constexpr int JT = Tile<RP>::JT;
    int64_t e[U];
    int j[U], i[U], cnt[U];
    if (a.tall) {
        // rows of r: elements [j0 r, (j0 + jn) r) of the matrix, four at a time
        const int total = jn * a.r, quads = (total + 3) / 4;
        const uint32_t magic = a.r > 1 ? 0xFFFFFFFFu / uint32_t(a.r) + 1u : 0u;
        for (int q0 = threadIdx.x; q0 < quads; q0 += U * kThreads) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int q = q0 + u * kThreads, k = 4 * q;
                cnt[u] = q < quads ? min(4, total - k) : 0;
                j[u] = a.r > 1 ? int(__umulhi(uint32_t(k), magic)) : k;
                i[u] = k - j[u] * a.r;
                e[u] = int64_t(j0) * a.r + k;
            }
            f(e, j, i, cnt);
        }
    } else if (a.vec) {
        // a warp takes 8 rows x 16 columns: 64 contiguous bytes a row
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
        const int cb = (jn + 15) / 16, units = ((a.r + 7) / 8) * cb;
        for (int q0 = warp; q0 < units; q0 += U * (kThreads / 32)) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int q = q0 + u * (kThreads / 32), ib = q / cb;
                i[u] = ib * 8 + (lane >> 2);
                j[u] = (q - ib * cb) * 16 + (lane & 3) * 4;
                cnt[u] = q < units && i[u] < a.r && j[u] < jn ? 4 : 0;     // n % 4 == 0: whole quads
                e[u] = int64_t(i[u]) * a.n + j0 + j[u];
            }
            f(e, j, i, cnt);
        }
    } else {
        for (int q0 = threadIdx.x; q0 < a.r * JT; q0 += U * kThreads) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int q = q0 + u * kThreads;
                i[u] = q / JT;
                j[u] = q % JT;
                cnt[u] = i[u] < a.r && j[u] < jn ? 1 : 0;
                e[u] = int64_t(i[u]) * a.n + j0 + j[u];
            }
            f(e, j, i, cnt);
        }
    }
}

// Element c of a piece: its place in the shared tile.
template <int RP>
__device__ __forceinline__ int place(const Mat &a, int j, int i, int c) {
    if (!a.tall) return (j + c) * Tile<RP>::LD + i;
    i += c;
    while (i >= a.r) {
        i -= a.r;
        ++j;
    }
    return j * Tile<RP>::LD + i;
}

__device__ __forceinline__ void load4(const float *p, int64_t e, int cnt, bool vec, float (&v)[4]) {
    if (vec && cnt == 4) {
        const float4 x = *reinterpret_cast<const float4 *>(p + e);
        v[0] = x.x; v[1] = x.y; v[2] = x.z; v[3] = x.w;
    } else {
#pragma unroll
        for (int c = 0; c < 4; ++c) v[c] = c < cnt ? p[e + c] : 0.f;
    }
}
__device__ __forceinline__ void keep4(float *p, int64_t e, int cnt, bool vec, const float (&v)[4]) {
    if (vec && cnt == 4) {
        *reinterpret_cast<float4 *>(p + e) = make_float4(v[0], v[1], v[2], v[3]);
    } else {
#pragma unroll
        for (int c = 0; c < 4; ++c)
            if (c < cnt) p[e + c] = v[c];
    }
}

// X <- M X on the shared tile: a thread takes its own columns whole into registers, so the
// product goes back in place without a barrier.  M's rows are the same for all threads.
template <int RP>
__device__ __forceinline__ void apply(float *x, const float *mt) {
    constexpr int JC = Tile<RP>::JC, LD = Tile<RP>::LD;
    float v[JC][RP];
#pragma unroll
    for (int c = 0; c < JC; ++c)
#pragma unroll
        for (int k = 0; k < RP; k += 4) {
            const float4 t = *reinterpret_cast<const float4 *>(x + (threadIdx.x + c * kThreads) * LD + k);
            v[c][k] = t.x; v[c][k + 1] = t.y; v[c][k + 2] = t.z; v[c][k + 3] = t.w;
        }
#pragma unroll 1
    for (int i = 0; i < RP; i += 4) {
        float y[JC][4];
#pragma unroll
        for (int c = 0; c < JC; ++c)
#pragma unroll
            for (int d = 0; d < 4; ++d) y[c][d] = 0.f;
#pragma unroll
        for (int k = 0; k < RP; ++k) {
            const float4 w = *reinterpret_cast<const float4 *>(mt + k * LD + i);   // M symmetric: row k, columns i..
#pragma unroll
            for (int c = 0; c < JC; ++c) {
                y[c][0] = fmaf(w.x, v[c][k], y[c][0]);
                y[c][1] = fmaf(w.y, v[c][k], y[c][1]);
                y[c][2] = fmaf(w.z, v[c][k], y[c][2]);
                y[c][3] = fmaf(w.w, v[c][k], y[c][3]);
            }
        }
#pragma unroll
        for (int c = 0; c < JC; ++c)
            *reinterpret_cast<float4 *>(x + (threadIdx.x + c * kThreads) * LD + i) =
                make_float4(y[c][0], y[c][1], y[c][2], y[c][3]);
    }
}

template <int RP, int SOURCE, int SINK>
__global__ void __launch_bounds__(kThreads) muon_pass_kernel(const __grid_constant__ Params p) {
    using T = Tile<RP>;
    constexpr int JT = T::JT, LD = T::LD, B = T::B, U = 4;
    extern __shared__ __align__(16) float sh[];
    float *x = sh, *mt = sh + (T::SMEM - RP * LD);
    int lo = 0, hi = p.nmat - 1;                            // this block's matrix
    while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if (p.mat[mid].block0 <= int(blockIdx.x)) lo = mid;
        else hi = mid - 1;
    }
    const Mat &a = p.mat[lo];
    const int bl = blockIdx.x - a.block0, span = p.tiles_per_block * JT;
    const int jb = bl * span, je = min(a.n, jb + span);
    const bool vec = a.vec != 0;
    if constexpr (SOURCE != kMomentum) {
        const float *src = p.ws + p.mpoly + int64_t(lo) * RP * RP;
        for (int k = threadIdx.x; k < RP * RP; k += kThreads) mt[(k / RP) * LD + k % RP] = src[k];
    }
    float acc[B][B];
#pragma unroll
    for (int s = 0; s < B; ++s)
#pragma unroll
        for (int t = 0; t < B; ++t) acc[s][t] = 0.f;
    int bi = 0, bk = 0;
    const int grp = threadIdx.x / T::PAIRS;
    pair_of<T::NB>(threadIdx.x % T::PAIRS, bi, bk);

    for (int j0 = jb; j0 < je; j0 += JT) {
        const int jn = min(JT, je - j0);
        __syncthreads();                                    // the last tile is used up (and M is there)
        if constexpr (SOURCE == kY) {
            const float4 *y = reinterpret_cast<const float4 *>(p.ws + a.y + int64_t(j0) * RP);
            for (int k = threadIdx.x; k < JT * (RP / 4); k += kThreads) {
                const int j = k / (RP / 4);
                *reinterpret_cast<float4 *>(x + j * LD + (k % (RP / 4)) * 4) = j < jn ? y[k] : make_float4(0.f, 0.f, 0.f, 0.f);
            }
        } else {
            if (jn < JT || a.r < RP) {                      // what lies past the matrix counts as 0
                for (int k = threadIdx.x; k < JT * LD; k += kThreads) x[k] = 0.f;
                __syncthreads();
            }
            visit<RP, U>(a, j0, jn, [&](const int64_t (&e)[U], const int (&j)[U], const int (&i)[U], const int (&cnt)[U]) {
                float g[U][4], m[U][4];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    load4(a.g, e[u], cnt[u], vec, g[u]);
                    load4(a.m, e[u], cnt[u], vec, m[u]);
                }
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    if (cnt[u] == 0) continue;
                    if constexpr (SOURCE == kMomentum) {
#pragma unroll
                        for (int c = 0; c < 4; ++c) m[u][c] = fmaf(p.mu, m[u][c], g[u][c]);
                        keep4(a.m, e[u], cnt[u], vec, m[u]);
                    }
                    float w[4];
#pragma unroll
                    for (int c = 0; c < 4; ++c) w[c] = p.nesterov ? fmaf(p.mu, m[u][c], g[u][c]) : m[u][c];
                    if (a.tall && cnt[u] == 4 && (a.r & 3) == 0) {
                        *reinterpret_cast<float4 *>(x + j[u] * LD + i[u]) = make_float4(w[0], w[1], w[2], w[3]);
                    } else {
#pragma unroll
                        for (int c = 0; c < 4; ++c)
                            if (c < cnt[u]) x[place<RP>(a, j[u], i[u], c)] = w[c];
                    }
                }
            });
        }
        __syncthreads();
        if constexpr (SOURCE != kMomentum) {
            apply<RP>(x, mt);
            __syncthreads();
        }
        if constexpr (SINK == kParam) {
            visit<RP, U>(a, j0, jn, [&](const int64_t (&e)[U], const int (&j)[U], const int (&i)[U], const int (&cnt)[U]) {
                float v[U][4];
#pragma unroll
                for (int u = 0; u < U; ++u) load4(a.p, e[u], cnt[u], vec, v[u]);
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    if (cnt[u] == 0) continue;
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        if (c < cnt[u]) {
                            const float o = x[place<RP>(a, j[u], i[u], c)];
                            v[u][c] -= a.lr * p.wd * v[u][c] + a.lr_scale * o;
                        }
                    keep4(a.p, e[u], cnt[u], vec, v[u]);
                }
            });
        } else {
            if constexpr (SINK == kGramY) {
                float4 *y = reinterpret_cast<float4 *>(p.ws + a.y + int64_t(j0) * RP);
                for (int k = threadIdx.x; k < jn * (RP / 4); k += kThreads)
                    y[k] = *reinterpret_cast<const float4 *>(x + (k / (RP / 4)) * LD + (k % (RP / 4)) * 4);
            }
            if (grp < T::GROUPS) {
#pragma unroll 2
                for (int j = grp; j < jn; j += T::GROUPS) {
                    float s[B], t[B];
#pragma unroll
                    for (int k = 0; k < B; k += 4) {
                        const float4 v = *reinterpret_cast<const float4 *>(x + j * LD + bi * B + k);
                        const float4 w = *reinterpret_cast<const float4 *>(x + j * LD + bk * B + k);
                        s[k] = v.x; s[k + 1] = v.y; s[k + 2] = v.z; s[k + 3] = v.w;
                        t[k] = w.x; t[k + 1] = w.y; t[k + 2] = w.z; t[k + 3] = w.w;
                    }
#pragma unroll
                    for (int k = 0; k < B; ++k)
#pragma unroll
                        for (int l = 0; l < B; ++l) acc[k][l] = fmaf(s[k], t[l], acc[k][l]);
                }
            }
        }
    }
    if constexpr (SINK != kParam) {
        // the groups' sums in a fixed tree, then out: [pair][B * B]
        float *mine = x + (threadIdx.x % T::PAIRS) * B * B;
        for (int h = T::HALF; h > 0; h /= 2) {
            __syncthreads();
            if (grp >= h && grp < 2 * h && grp < T::GROUPS) {
#pragma unroll
                for (int k = 0; k < B * B; ++k) mine[(grp - h) * T::GSIZE + k] = acc[k / B][k % B];
            }
            __syncthreads();
            if (grp < h && grp + h < T::GROUPS) {
#pragma unroll
                for (int k = 0; k < B * B; ++k) acc[k / B][k % B] += mine[grp * T::GSIZE + k];
            }
        }
        if (grp == 0) {
            float *out = p.ws + a.part + int64_t(bl) * T::GSIZE + threadIdx.x * B * B;
#pragma unroll
            for (int k = 0; k < B * B; k += 4)
                *reinterpret_cast<float4 *>(out + k) =
                    make_float4(acc[k / B][k % B], acc[k / B][k % B + 1], acc[k / B][k % B + 2], acc[k / B][k % B + 3]);
        }
    }
}

struct PolyParams {
    int64_t part[kMaxMats];              // offsets of the partial Gram matrices
    int32_t blocks[kMaxMats];            // how many
    float *ws;
    int64_t mpoly;
    float a, b, c, eps;
    int steps, first;                    // first: G is of u, to be normalised
};

// One matrix a block: G from its partial sums in block order, then the product M of `steps`
// Newton-Schulz polynomials P.  G and P are symmetric: a row stands for a column.
template <int RP>
__global__ void __launch_bounds__(kPolyThreads) muon_poly_kernel(const __grid_constant__ PolyParams p) {
    using T = Tile<RP>;
    constexpr int LD = T::LD, B = T::B;
    constexpr int D = RP >= 16 ? RP / 16 : 1, ACTIVE = (RP / D) * (RP / D);   // D x D elements a thread
    extern __shared__ __align__(16) float sh[];
    float *gm = sh, *sq = gm + RP * LD, *pm = sq + RP * LD, *mm = pm + RP * LD;
    __shared__ float s_norm;
    const int tid = threadIdx.x;
    const float *part = p.ws + p.part[blockIdx.x];
    const int nb = p.blocks[blockIdx.x];
    for (int e = tid; e < T::GSIZE; e += kPolyThreads) {
        float s = 0.f;
        for (int k = 0; k < nb; k += 8) {
            float v[8];
#pragma unroll
            for (int u = 0; u < 8; ++u) v[u] = k + u < nb ? part[int64_t(k + u) * T::GSIZE + e] : 0.f;
#pragma unroll
            for (int u = 0; u < 8; ++u) s += v[u];
        }
        int bi, bk;
        pair_of<T::NB>(e / (B * B), bi, bk);
        const int i = bi * B + (e % (B * B)) / B, k = bk * B + e % B;
        gm[i * LD + k] = s;
        gm[k * LD + i] = s;
    }
    __syncthreads();
    float inv = 1.f;
    if (p.first) {
        if (tid < 32) {
            float t = 0.f;
            for (int k = tid; k < RP; k += 32) t += gm[k * LD + k];
            t = warp_sum(t);
            if (tid == 0) s_norm = sqrtf(t);
        }
        __syncthreads();
        // X0 = u inv; a zero update stays zero (0 / eps), also for eps = 0
        const float norm = s_norm + p.eps;
        inv = norm > 0.f ? 1.f / norm : 0.f;
        __syncthreads();
        for (int e = tid; e < RP * RP; e += kPolyThreads) gm[(e / RP) * LD + e % RP] *= inv * inv;
        __syncthreads();
    }
    const int r0 = (tid / (RP / D)) * D, c0 = (tid % (RP / D)) * D;
    const bool on = tid < ACTIVE;
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
#pragma unroll
                for (int s = 0; s < D; ++s) {
                    u[s] = x[k * LD + r0 + s];
                    v[s] = y[k * LD + c0 + s];
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
                for (int t = 0; t < D; ++t) out[(r0 + s) * LD + c0 + t] = f(acc[s][t], r0 + s, c0 + t);
        }
        __syncthreads();
    };
    auto same = [](float v, int, int) { return v; };
    for (int s = 0; s < p.steps; ++s) {
        product(gm, gm, pm, [&](float v, int i, int k) { return fmaf(p.c, v, fmaf(p.b, gm[i * LD + k], i == k ? p.a : 0.f)); });
        if (s == 0) {
            for (int e = tid; e < RP * RP; e += kPolyThreads) mm[(e / RP) * LD + e % RP] = pm[(e / RP) * LD + e % RP];
            __syncthreads();
        } else {
            product(pm, mm, mm, same);
        }
        if (s + 1 < p.steps) {
            // G of the next X: P G P with one factor on either side, made symmetric again
            // (G P P, equal but for rounding, or a G left unsymmetric, cost a digit in X)
            product(gm, pm, sq, same);                       // G P
            product(sq, pm, gm, same);                       // (G P)^T P
            for (int e = tid; e < RP * RP; e += kPolyThreads) {
                const int i = e / RP, k = e % RP;
                if (i < k) gm[i * LD + k] = gm[k * LD + i] = 0.5f * (gm[i * LD + k] + gm[k * LD + i]);
            }
            __syncthreads();
        }
    }
    float *out = p.ws + p.mpoly + int64_t(blockIdx.x) * RP * RP;
    for (int e = tid; e < RP * RP; e += kPolyThreads) out[e] = mm[(e / RP) * LD + e % RP] * inv;
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

// Workspace of a class's group of matrices [first, last) of the list `idx`: Y, the partial
// Gram matrices (as many as tiles, the most there can be) and the products M.
template <int RP>
size_t group_floats(const tlb_muon_mat *mats, const int *idx, int n) {
    size_t f = 0;
    for (int k = 0; k < n; ++k) {
        const int64_t len = std::max(mats[idx[k]].rows, mats[idx[k]].cols);
        f += size_t(len) * RP + size_t(tiles_of<RP>(len)) * Tile<RP>::GSIZE + size_t(RP) * RP;
    }
    return f;
}

template <int RP, int SOURCE, int SINK>
int pass(const Params &p, unsigned blocks, cudaStream_t st) {
    constexpr int smem = Tile<RP>::SMEM * 4;
    auto k = muon_pass_kernel<RP, SOURCE, SINK>;
    TLB_CUDA(cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, smem));
    k<<<blocks, kThreads, smem, st>>>(p);
    return check_launch("muon_pass");
}

template <int RP>
int group(const tlb_muon_mat *mats, const int *idx, int n, const tlb_muon_cfg &cfg, float *ws, cudaStream_t st) {
    Params p;
    PolyParams q;
    memset(&p, 0, sizeof(p));
    memset(&q, 0, sizeof(q));
    int64_t tiles = 0, off = 0;
    for (int k = 0; k < n; ++k) tiles += tiles_of<RP>(std::max(mats[idx[k]].rows, mats[idx[k]].cols));
    p.tiles_per_block = tiles_per_block(tiles);
    p.nmat = n;
    p.ws = q.ws = ws;
    p.mu = float(cfg.momentum);
    p.wd = float(cfg.weight_decay);
    p.nesterov = cfg.nesterov != 0;
    int64_t blocks = 0;
    for (int k = 0; k < n; ++k) {
        const tlb_muon_mat &s = mats[idx[k]];
        Mat &a = p.mat[k];
        a.p = s.p;
        a.g = s.g;
        a.m = s.m;
        a.tall = s.rows > s.cols;
        a.r = std::min(s.rows, s.cols);
        a.n = std::max(s.rows, s.cols);
        a.vec = aligned16(s.p) && aligned16(s.g) && aligned16(s.m) && (a.tall || a.n % 4 == 0);
        a.lr = float(cfg.lr * double(s.lr_mult));
        a.lr_scale = float(cfg.lr * double(s.lr_mult) * double(s.scale));
        a.block0 = int(blocks);
        q.blocks[k] = int(ceil_div(tiles_of<RP>(a.n), p.tiles_per_block));
        blocks += q.blocks[k];
        a.y = off;
        off += int64_t(a.n) * RP;
        a.part = q.part[k] = off;
        off += tiles_of<RP>(a.n) * Tile<RP>::GSIZE;
    }
    p.mpoly = q.mpoly = off;
    q.a = float(cfg.a);
    q.b = float(cfg.b);
    q.c = float(cfg.c);
    q.eps = float(cfg.eps);
    const unsigned grid = unsigned(blocks);
    constexpr int poly_smem = 4 * RP * Tile<RP>::LD * 4;
    TLB_CUDA(cudaFuncSetAttribute(muon_poly_kernel<RP>, cudaFuncAttributeMaxDynamicSharedMemorySize, poly_smem));
    TLB_TRY((pass<RP, kMomentum, kGram>(p, grid, st)));
    for (int done = 0; done < cfg.steps;) {
        q.first = done == 0;
        q.steps = std::min(q.first ? kFirstRun : kRun, cfg.steps - done);
        muon_poly_kernel<RP><<<unsigned(n), kPolyThreads, poly_smem, st>>>(q);
        TLB_TRY(check_launch("muon_poly"));
        done += q.steps;
        const bool last = done == cfg.steps;
        if (q.first) TLB_TRY((last ? pass<RP, kUpdate, kParam>(p, grid, st) : pass<RP, kUpdate, kGramY>(p, grid, st)));
        else TLB_TRY((last ? pass<RP, kY, kParam>(p, grid, st) : pass<RP, kY, kGramY>(p, grid, st)));
    }
    return TLB_OK;
}

template <typename F8, typename F16, typename F32, typename F64>
auto by_class(int rp, F8 f8, F16 f16, F32 f32, F64 f64) {
    return rp == 8 ? f8() : rp == 16 ? f16() : rp == 32 ? f32() : f64();
}

// Calls f(class, indices, count) for groups of at most kMaxMats matrices of one class.
template <typename F>
int for_groups(const tlb_muon_mat *mats, int32_t n, F f) {
    int idx[kMaxMats];
    for (int rp = 8; rp <= 64; rp *= 2) {
        int k = 0;
        for (int i = 0; i < n; ++i) {
            if (mats[i].rows == 0 || mats[i].cols == 0 || rank_class(std::min(mats[i].rows, mats[i].cols)) != rp) continue;
            idx[k++] = i;
            if (k == kMaxMats) {
                TLB_TRY(f(rp, idx, k));
                k = 0;
            }
        }
        if (k > 0) TLB_TRY(f(rp, idx, k));
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
    return for_groups(mats, n, [&](int rp, const int *idx, int k) {
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
    return for_groups(mats, n, [&](int rp, const int *idx, int k) {
        return by_class(rp, [&] { return group<8>(mats, idx, k, *cfg, w, st); },
                        [&] { return group<16>(mats, idx, k, *cfg, w, st); },
                        [&] { return group<32>(mats, idx, k, *cfg, w, st); },
                        [&] { return group<64>(mats, idx, k, *cfg, w, st); });
    });
}

}  // extern "C"
