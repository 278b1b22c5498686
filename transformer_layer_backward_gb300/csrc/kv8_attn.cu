// Attention of single tokens over the 8-bit K/V cache, and its gradient.
//
// Bound by the read of the keys and values (once for up to eight query heads a KV head, four in the gradient; a
// larger group reads and multiplies them again for each tile of as many).  What a CTA (four warps) does for a run of one sequence's keys, one
// KV head and a tile of the query heads that share it, 16 keys a warp at a time:
//   - cp.async brings the keys', values' and scales' bytes to shared memory, a step ahead; keys that
//     are not there come as zeros, so that nothing of what a free slot holds is met;
//   - s = q k and (gradient) dp = d_ctx v are products of mma.sync m16n8k16 with the keys as columns: e4m3 values
//     are halves exactly, and a query is two of them, the second holding what the first leaves times 2^12 (rows g
//     and g + 8 of the operand, which meet in one thread).  The 16 bytes of a row that a lane reads serve as
//     operands as they are, the query's columns being ordered to match;
//   - the sums over keys (p v; p dp k and p k) take the weights x in the same two halves, scaled by a
//     power of two of each row that follows the largest |x| so far (as it counts now: it grows with |x| and falls
//     when the forward's reference rises), and the rows' bytes transposed by byte permutes: 23 bits of each weight,
//     34 below the largest at least.
// The gradient uses d_q = scale (sum p dp k - (sum p dp)(sum p k)), so that one pass does.  Rows of the gradient's
// tile: four heads' s (and p dp) in rows 0..3, their dp (and p) in rows 4..7; of the forward's: eight heads.
// Warps, then the CTAs that share a unit (a second kernel), are joined in a fixed order.
// Of the time of a step (600 instructions for 16 keys in the gradient, a quarter of them conversions to halves)
// half is latency: 16 warps an SM, since a warp's sums take 64 registers a thread.  131072 keys of 8 KV heads and 32 query
// heads of 128: gradient 73.8 us (277 MB, 3.8 TB/s); a batch of 32 sequences up to 16384 keys: forward 34.6 us (116 MB,
// 3.4 TB/s).  65536 keys of 8 KV heads: gradient of 32 heads 47 us, of 64 (two tiles) 75 us.
// Slower: 32 keys a step (82 us: three CTAs an SM), the sums of the step before beside a step's logits (81 us).
#include <cmath>

#include "async.cuh"
#include "kv8.cuh"

namespace tlb {

namespace {

constexpr int kWarps = 4;
constexpr int kStep = 16;                // keys of a warp's step
constexpr int kStages = 2;               // one step ahead: four CTAs an SM keep 70 KB on their way (three stages and three CTAs: slower)
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kLog2eLow = 1.925963033500e-8f;      // log2(e) - float(log2(e))
constexpr float kLow = 4096.f;           // the second half of a value holds what the first leaves, times this

constexpr int tile_heads(bool grad) { return grad ? 4 : 8; }

// Shared memory: the query's operand (and d_ctx's), then each warp's stages of keys, values, scales and a mask.
template <int HD> constexpr int stage_bytes() { return 2 * kStep * HD + 3 * kStep * 4; }
template <int HD, bool GRAD> constexpr int smem_bytes() {
    return (GRAD ? 2 : 1) * (HD / 16) * 32 * 16 + kWarps * kStages * stage_bytes<HD>();
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ void mma_f16(float (&d)[4], const uint4 &a, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1));
}

// bytes < 16 or ok false: zeros
__device__ __forceinline__ void copy16(uint32_t dst, const void *src, bool ok) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(ok ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy4(uint32_t dst, const void *src, bool ok) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(ok ? 4 : 0) : "memory");
}

// Place of the 16-byte piece c of row r of a stage: the pieces are turned by the row so that neither the rows n, n + 1
// that eight lanes read for the logits nor the rows 0, 2, 4, 6 (1, 3, 5, 7) of the sums meet in a bank.
template <int HD>
__device__ __forceinline__ int place(int r, int c) {
    const int turn = HD == 64 ? (r >> 1) & 3 : ((r & 1) << 2) ^ (r & 6);
    return r * HD + ((c ^ turn) << 4);
}

// x = hi + lo / 4096, as a pair of each for two values
__device__ __forceinline__ void halves(float x, float y, uint32_t &hi, uint32_t &lo) {
    const __half2 h = __floats2half2_rn(x, y);
    const float2 f = __half22float2(h);
    const __half2 l = __floats2half2_rn((x - f.x) * kLow, (y - f.y) * kLow);
    hi = *reinterpret_cast<const uint32_t *>(&h);
    lo = *reinterpret_cast<const uint32_t *>(&l);
}

// 2^e, -149 <= e <= 127
__device__ __forceinline__ float pow2(int e) { return e >= -126 ? __uint_as_float(uint32_t(e + 127) << 23) : __uint_as_float(1u << (e + 149)); }

struct AttnParams {
    tlb_kv8 c;
    Kv8Pages pg;
    int64_t n_seq;
    int n_heads, group, tiles, ctas;     // heads a KV head, tiles of them
    float scale;
    const void *q, *d_ctx;
    const float *lse;            // gradient
    void *out;                   // ctx or d_q
    void *d_k, *d_v;             // gradient
    float *out_lse;
    float *part;                 // [ctas][2][8 rows][head_dim]: sums of a CTA's first and last unit, where these are shared
    float2 *sums;                // [ctas][2][8]: forward (max, sum of exp), gradient (sum p dp, -)
    int2 *parts;                 // [n_seq, units]: the first CTA of a unit (times 2, plus its slot) and the last
    float2 *newest;              // [n_seq, n_heads]: p and dp of the newest key
    float *D;                    // [n_seq, n_heads]: sum p dp of a unit that one CTA did
};

// The work is laid out in a line: sequence by sequence, unit by unit (a KV head and a tile of its query heads), a unit
// of S steps of 16 keys weighing kFixed + S, since its start and its end cost as much as some steps.  CTA c of n takes
// [total c / n, total (c + 1) / n) of that line: as many CTAs as are on the GPU at a time, each with the same
// weight whatever the lengths, which only the device knows.  The first kFixed of a unit are no steps.  A batch of 32
// sequences of 64 to 16384 keys (120895 in all), us with kFixed 6 / 12 / 20 / 30:
//   heads of 64 (32 / 8)   bf16 forward 50.0 41.1 40.4 40.6   gradient 64.9 52.5 51.3 51.8
//   heads of 128 (32 / 8)  float32 forward 71.4 59.2 57.5 57.4   gradient 89.9 76.3 74.0 76.5
//   heads of 256 (16 / 4)  float32 forward 76.5 64.0 55.1 55.4   gradient 94.0 79.5 68.6 70.3   bf16 forward 93.4 76.7 63.1 57.8
// kLeast: the weight that is worth a CTA; where it lies in a unit's first kFixed that CTA has nothing to do (1024 keys:
// weight 84, 21 CTAs, 16 of them with steps).  kMostParts: CTAs a unit, on average over the units, since one CTA of the join
// reads all its parts (65536 keys of one KV head: 608 parts 41 us, 128 19.6 us).  Among shorter sequences a long one of
// few KV heads still gets more than that (beside four of 200 keys: 40 us).
constexpr int kFixed = 20, kLeast = 4, kMostParts = 128;

__device__ __forceinline__ int64_t steps_of(int len) { return (len + kStep - 1) / kStep; }
__device__ __forceinline__ int cta_count(int64_t total, int most) { return int(max(int64_t(1), min(int64_t(most), total / kLeast))); }
// a / b for b below 2^31; places of the line seldom need more than 32 bits, whose division is a few times shorter
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
    return uint64_t(a) >> 32 ? a / b : int64_t(uint32_t(a) / uint32_t(b));
}
// total c / n, by parts so that no product overflows
__device__ __forceinline__ int64_t share(int64_t total, int n, int c) {
    const int64_t q = quotient(total, n);
    return q * c + int(total - q * n) * c / n;
}
// What a CTA does next.
struct Segment {
    int64_t pos, end, base;      // places of the line: next, the CTA's last, the sequence's first
    int64_t b;
    int unit, len, s0, s1, slot, run;
};

// Rows of T as the first operand: piece ks of lane (g, t) holds columns 64 (ks / 4) + 16 t + 4 (ks % 4) + {0, 1 | 2, 3} of row
// g's two halves.  f[g]: the power of two that the row was divided by (its largest value becomes 2^14 .. 2^15).
template <typename T, int HD>
__device__ __forceinline__ void stage_rows(const T *rows, int n, int hd, int first, uint4 *to, int *f) {
    // a warp a row; rows first .. first + n - 1 of the operand, the others zero
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int g = warp; g < 8; g += kWarps) {
        const bool there = g >= first && g < first + n;
        const T *p = rows + int64_t(there ? g - first : 0) * hd;
        uint32_t top = 0;
        float x[HD / 32];
#pragma unroll
        for (int i = 0; i < HD / 32; ++i) {
            x[i] = there && lane + 32 * i < hd ? load_float(p + lane + 32 * i) : 0.f;
            top = max(top, magnitude(x[i]));
        }
        top = __reduce_max_sync(0xffffffffu, top);
        // rows below 2^-100 keep that power; of infinities and NaN the halves are NaN whatever it is
        const int e = max(int(top >> 23) - 127, -100) - 14;
        if (lane == 0) f[g] = e;
        const float s = pow2(-e);
#pragma unroll
        for (int i = 0; i < HD / 32; ++i) {
            const int d = lane + 32 * i;
            const float y = x[i] * s;
            const __half hi = __float2half_rn(y);
            const __half lo = __float2half_rn((y - __half2float(hi)) * kLow);
            const int ks = (d >> 6) * 4 + ((d >> 2) & 3), t = (d >> 4) & 3;
            __half *o = reinterpret_cast<__half *>(&to[ks * 32 + g * 4 + t]);   // a0, a1, a2, a3 as pairs
            o[((d >> 1) & 1) * 4 + (d & 1)] = hi;
            o[((d >> 1) & 1) * 4 + 2 + (d & 1)] = lo;
        }
    }
}

template <typename T, int HD, bool GRAD>
__global__ void __launch_bounds__(kWarps * 32, HD <= 128 ? 4 : 2) kv8_attn_kernel(const __grid_constant__ AttnParams p) {
    constexpr int HT = tile_heads(GRAD), KS = HD / 16, NT = HD / 8;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ int s_f[2][8];
    __shared__ float s_m[kWarps][8], s_l[kWarps][8];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    __shared__ Segment sg;
    __shared__ int64_t s_scan[kWarps];
    const int nkv = p.c.n_kv_heads, hd = p.c.head_dim, units = nkv * p.tiles;

    // ---- this CTA's part of the line: a scan of the sequences' weights, a run of them a thread
    {
        const int64_t per = (p.n_seq + kWarps * 32 - 1) / (kWarps * 32), b0 = min(p.n_seq, threadIdx.x * per), b1 = min(p.n_seq, b0 + per);
        int64_t mine = 0;
        for (int64_t i = b0; i < b1; ++i) mine += kFixed + steps_of(kv8_length(p.pg, i));
        int64_t upto = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t v = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += v;
        }
        if (lane == 31) s_scan[warp] = upto;
        __syncthreads();
        int64_t total = 0;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            if (w < warp) upto += s_scan[w];
            total += s_scan[w];
        }
        int64_t base = upto - mine;
        total *= units;
        const int n = cta_count(total, p.ctas);
        if (int(blockIdx.x) >= n) return;
        const int64_t lo = share(total, n, int(blockIdx.x));
        if (lo >= base * units && lo < upto * units) {
            for (int64_t i = b0; i < b1; ++i) {
                const int len = kv8_length(p.pg, i);
                const int64_t next = base + kFixed + steps_of(len);
                if (lo < next * units) {
                    sg.pos = lo;
                    sg.end = share(total, n, int(blockIdx.x) + 1);
                    sg.base = base * units;
                    sg.b = i;
                    sg.len = len;
                    sg.slot = 0;
                    break;
                }
                base = next;
            }
        }
        __syncthreads();
    }
  for (;;) {
    if (threadIdx.x == 0) {
        // the next segment that has something to do: steps [s0, s1) of a unit
        sg.run = 0;
        while (!sg.run && sg.pos < sg.end) {
            const int64_t S = steps_of(sg.len), weight = kFixed + S, unit = quotient(sg.pos - sg.base, weight);
            const int64_t from = sg.base + unit * weight, to = min(sg.end, from + weight);
            sg.unit = int(unit);
            sg.s0 = int(max(sg.pos - from - kFixed, int64_t(0)));
            sg.s1 = int(max(to - from - kFixed, int64_t(0)));
            if (sg.s1 > sg.s0 || (S == 0 && to == from + weight)) {
                sg.run = 1;
                break;
            }
            sg.slot = 1;
            sg.pos = to;
            if (to == from + weight && unit == units - 1) {
                sg.base = to;
                if (sg.pos < sg.end) sg.len = kv8_length(p.pg, ++sg.b);
            }
        }
    }
    __syncthreads();
    if (!sg.run) break;
    const int64_t b = sg.b;
    const int kvh = sg.unit / p.tiles, tile = sg.unit % p.tiles, len = sg.len;
    const int k0 = sg.s0 * kStep, k1 = min(len, sg.s1 * kStep), steps = sg.s1 - sg.s0;
    const bool whole = sg.s0 == 0 && sg.s1 == steps_of(len);
    const int64_t head0 = b * p.n_heads + kvh * p.group + tile * HT;   // first row of q
    const int heads = min(HT, p.group - tile * HT);

    // ---- copies: step i of this warp is keys k0 + 16 (warp + kWarps i) ..
    const uint32_t ring = smem_u32(smem) + (GRAD ? 2 : 1) * KS * 512 + warp * kStages * stage_bytes<HD>();
    const int mine = steps > warp ? (steps - warp + kWarps - 1) / kWarps : 0;
    auto slot_of = [&](int i) {          // lane's key of step i (its lower four bits), -1 where there is none
        const int j = k0 + kStep * (warp + kWarps * i) + (lane & 15);
        return i < mine && j < k1 ? int(kv8_slot(p.pg, p.c.n_slots, b, j)) : -1;
    };
    int slot = slot_of(0);
    // this lane's piece of a row, and the rows r0, r0 + 512 / HD, .. of a step
    constexpr int PER = HD / 16;
    const int ch = lane % PER, r0 = lane / PER;
    const bool in_row = ch * 16 < hd;
    const int64_t first = int64_t(kvh) * hd + (in_row ? ch * 16 : 0);
    const uint8_t *kb = p.c.k + first, *vb = p.c.v + first;
    const int row_stride = nkv * hd;
    const float *sb = (lane < 16 ? p.c.k_scale : p.c.v_scale) + int64_t(kvh) * p.c.n_slots;
    auto issue = [&](int i) {
        if (i < mine) {
            const uint32_t st = ring + (i % kStages) * stage_bytes<HD>();
            const int mask = int(__ballot_sync(0xffffffffu, slot >= 0));
#pragma unroll
            for (int c = 0; c < kStep * PER / 32; ++c) {
                const int r = c * (32 / PER) + r0, sl = __shfl_sync(0xffffffffu, slot, r);
                const bool ok = sl >= 0 && in_row;
                const int64_t at = int64_t(max(sl, 0)) * row_stride;
                copy16(st + place<HD>(r, ch), kb + at, ok);
                copy16(st + kStep * HD + place<HD>(r, ch), vb + at, ok);
            }
            copy4(st + 2 * kStep * HD + lane * 4, sb + max(slot, 0), slot >= 0);
            if (lane == 0)
                asm volatile("st.shared.u32 [%0], %1;" ::"r"(st + 2 * kStep * HD + 128), "r"(mask) : "memory");
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        slot = slot_of(i + 1);
    };
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) issue(i);

    // ---- the queries
    uint4 *qf = reinterpret_cast<uint4 *>(smem);
    stage_rows<T, HD>(static_cast<const T *>(p.q) + head0 * hd, heads, hd, 0, qf, s_f[0]);
    if (GRAD) stage_rows<T, HD>(static_cast<const T *>(p.d_ctx) + head0 * hd, heads, hd, 4, qf + KS * 32, s_f[1]);
    __syncthreads();
    // this lane's row: the factor of its logits (in powers of two, gradient rows 4..7: of dp)
    const bool is_dp = GRAD && g >= 4;
    const float factor = is_dp ? pow2(s_f[1][g]) : p.scale * kLog2e * pow2(s_f[0][g]);
    const int my_head = is_dp ? g - 4 : g;
    // p = 2^(x - lse), x and lse over ln 2.  Of an lse between 0 and 100 the whole part goes into a factor, so that the
    // difference is of x's size and keeps x's bits; the rest keeps the product's rounding
    float norm = 0.f, p_scale = 1.f;
    if (GRAD && my_head < heads) {
        const float lse = __ldg(p.lse + head0 + my_head), hi = lse * kLog2e;
        const float part = hi > 0.f && hi < 100.f ? rintf(hi) : 0.f;
        const float lo = fmaf(lse, kLog2e, -hi) + lse * kLog2eLow;
        norm = (hi - part) + (isfinite(lo) ? lo : 0.f);
        p_scale = pow2(-int(part));
    }

    float acc[NT][4];
#pragma unroll
    for (int i = 0; i < NT; ++i) acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.f;
    float m = -INFINITY, l = 0.f;        // forward: the row's largest logit, sum of exp; gradient: l = sum p dp (rows 0..3)
    int ex = -120;                       // the sums are of x / 2^ex
    for (int i = 0; i < mine; ++i) {
        issue(i + kStages - 1);
        asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
        __syncwarp();
        const uint8_t *st = smem + (GRAD ? 2 : 1) * KS * 512 + (warp * kStages + i % kStages) * stage_bytes<HD>();
        const uint8_t *sk_rows = st, *sv_rows = st + kStep * HD;
        const float *scales = reinterpret_cast<const float *>(st + 2 * kStep * HD);
        const uint32_t mask = *reinterpret_cast<const uint32_t *>(st + 2 * kStep * HD + 128);

        // ---- logits (and dp): columns are keys.  The gradient's rows of q and of d_ctx have sums of their own: 0 times a
        // value that is NaN is NaN, and the logits do not depend on the values
        float cf[2][4], part[2][2][4] = {};                    // [chain][tile of 8 keys]: two chains of products at least
#pragma unroll
        for (int c = 0; c < HD / 64; ++c)
#pragma unroll
            for (int w = 0; w < (GRAD ? 2 : 1); ++w) {
                uint4 kq[2];
#pragma unroll
                for (int nt = 0; nt < 2; ++nt)
                    kq[nt] = *reinterpret_cast<const uint4 *>((w == 0 ? sk_rows : sv_rows) + place<HD>(nt * 8 + g, c * 4 + t));
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const uint4 a = qf[(w * KS + c * 4 + u) * 32 + lane];
#pragma unroll
                    for (int nt = 0; nt < 2; ++nt) {
                        uint32_t b0, b1;
                        e4m3x4_to_half2(u == 0 ? kq[nt].x : u == 1 ? kq[nt].y : u == 2 ? kq[nt].z : kq[nt].w, b0, b1);
                        mma_f16(part[GRAD ? w : u & 1][nt], a, b0, b1);
                    }
                }
            }
#pragma unroll
        for (int nt = 0; nt < 2; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                cf[nt][e] = GRAD ? (is_dp ? part[1][nt][e] : part[0][nt][e]) : part[0][nt][e] + part[1][nt][e];
        // ---- the weights x of this lane's row for keys 2 t, 2 t + 1, 2 t + 8, 2 t + 9
        float x[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int key = (e >> 1) * 8 + 2 * t + (e & 1);
            const float raw = fmaf(cf[e >> 1][2 + (e & 1)], 1.f / kLow, cf[e >> 1][e & 1]) * factor;
            x[e] = raw * scales[is_dp ? 16 + key : key];
        }
        auto there = [&](int e) { return (mask >> ((e >> 1) * 8 + 2 * t + (e & 1))) & 1u; };
        int fall = 0;                    // powers of two that the reference rose by, and the sums fell by
        if (!GRAD) {
            float top = m;
#pragma unroll
            for (int e = 0; e < 4; ++e) top = there(e) ? fmaxf(top, x[e]) : top;
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
            // the reference, a whole number, follows the largest logit when that is 2^8 beyond it: until then weights are
            // up to 2^8.  The sums' power falls by as much as the reference rises: weights of now are held to the
            // bits of what counts now, however large the values of keys were that have lost their weight
            if (top > m + 8.f || (m == -INFINITY && top > m)) {
                const float to = floorf(top);
                l *= ex2(m - to);
                fall = int(fminf(to - m, 4096.f));
                m = to;
            }
            const float ref = m == -INFINITY ? 0.f : m;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int key = (e >> 1) * 8 + 2 * t + (e & 1);
                const float w = there(e) ? ex2(x[e] - ref) : 0.f;
                l += w;
                x[e] = there(e) ? w * scales[16 + key] : 0.f;
            }
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int key = (e >> 1) * 8 + 2 * t + (e & 1);
                const float own = is_dp ? x[e] : ex2(x[e] - norm) * p_scale;
                const float other = __shfl_xor_sync(0xffffffffu, own, 16);   // dp for the rows of p and the other way round
                const float w = there(e) ? (is_dp ? other : own * other) : 0.f;
                if (!is_dp) {
                    l += w;
                    if (k0 + kStep * (warp + kWarps * i) + key == len - 1 && my_head < heads)
                        p.newest[head0 + my_head] = there(e) ? make_float2(own, other) : make_float2(0.f, 0.f);
                }
                x[e] = there(e) ? w * scales[key] : 0.f;
            }
        }
        uint32_t top = max(max(magnitude(x[0]), magnitude(x[1])), max(magnitude(x[2]), magnitude(x[3])));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        // with room for weights of eight times the size, so that the sums are seldom turned to a new power (2^127 holds
        // every float; of weights that are not finite the sums are NaN whatever it is)
        const int low = max(ex - fall, -120), grown = int(top >> 23) - 127 > low ? min(int(top >> 23) - 124, 127) : low;
        const int turn = ex - fall - grown;
        ex = grown;
        if (__any_sync(0xffffffffu, turn != 0)) {
            const float alpha = pow2(max(turn, -149));
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                acc[n][0] *= alpha; acc[n][1] *= alpha; acc[n][2] *= alpha; acc[n][3] *= alpha;
            }
        }
        const float down = pow2(-ex);
        uint4 a;
        halves(x[0] * down, x[1] * down, a.x, a.y);
        halves(x[2] * down, x[3] * down, a.z, a.w);

        // ---- sums over keys: the rows' bytes transposed, columns are dimensions
        const uint8_t *rows = GRAD ? sk_rows : sv_rows;
#pragma unroll
        for (int c = 0; c < (HD > 128 ? 2 : 1); ++c) {
            constexpr int W = HD == 64 ? 2 : 4;                // words a lane takes of a row: dimensions 4 W n ..
            uint32_t v[4][W];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int r = (e >> 1) * 8 + 2 * t + (e & 1);
                if (HD == 64) {
                    const uint2 y = *reinterpret_cast<const uint2 *>(rows + place<HD>(r, g >> 1) + (g & 1) * 8);
                    v[e][0] = y.x;
                    v[e][1] = y.y;
                } else {
                    const uint4 y = *reinterpret_cast<const uint4 *>(rows + place<HD>(r, c * 8 + g));
                    v[e][0] = y.x;
                    v[e][1] = y.y;
                    v[e][W - 2] = y.z;
                    v[e][W - 1] = y.w;
                }
            }
#pragma unroll
            for (int w = 0; w < W; ++w)
#pragma unroll
                for (int h = 0; h < 2; ++h) {                  // bytes 2 h, 2 h + 1 of the word
                    const uint32_t b0 = __byte_perm(v[0][w], v[1][w], h ? 0x7362 : 0x5140);
                    const uint32_t b1 = __byte_perm(v[2][w], v[3][w], h ? 0x7362 : 0x5140);
                    const int n = c * 16 + w * 4 + h * 2;
                    uint32_t lo0, hi0, lo1, hi1;
                    e4m3x4_to_half2(b0, lo0, hi0);
                    e4m3x4_to_half2(b1, lo1, hi1);
                    mma_f16(acc[n], a, lo0, lo1);
                    mma_f16(acc[n + 1], a, hi0, hi1);
                }
        }
        __syncwarp();                                          // before this stage is copied over
    }
    asm volatile("cp.async.wait_all;" ::: "memory");

    // ---- the warps' sums join in shared memory: [warp][row][hd]
    l += __shfl_xor_sync(0xffffffffu, l, 1);
    l += __shfl_xor_sync(0xffffffffu, l, 2);
    __syncthreads();
    if (t == 0) {
        s_m[warp][g] = m;
        s_l[warp][g] = l;
    }
    float *all = reinterpret_cast<float *>(smem);
    const float up = pow2(ex);
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            // column 2 t + e of tile n: the byte that lane group 2 t + e took
            const int d = HD == 64 ? (2 * t + e) * 8 + n : (n >> 4) * 128 + (2 * t + e) * 16 + (n & 15);
            all[(warp * 8 + g) * HD + d] = fmaf(acc[n][2 + e], 1.f / kLow, acc[n][e]) * up;
        }
    __syncthreads();
    const int64_t row0 = (int64_t(blockIdx.x) * 2 + sg.slot) * 8;      // where a part of a unit goes
    for (int e = threadIdx.x; e < 8 * HD; e += kWarps * 32) {
        const int r = e / HD, d = e % HD;
        const int h = GRAD ? r & 3 : r;
        if (h >= heads || d >= hd) continue;
        float y = 0.f;
        if (!GRAD) {
            float top = -INFINITY;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) top = fmaxf(top, s_m[w][r]);
            const float ref = top == -INFINITY ? 0.f : top;
            float total = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float f = ex2(s_m[w][r] - ref);
                y = fmaf(all[(w * 8 + r) * HD + d], f, y);
                total = fmaf(s_l[w][r], f, total);
            }
            if (whole) {
                store_float(static_cast<T *>(p.out) + (head0 + h) * hd + d, total == 0.f ? 0.f : y / total);
                if (d == 0) p.out_lse[head0 + h] = total == 0.f ? -INFINITY : fmaf(log2f(total), kLn2, top * kLn2);
            } else {
                p.part[(row0 + r) * hd + d] = y;
                if (d == 0) p.sums[row0 + r] = make_float2(top, total);
            }
        } else {
            float D = 0.f, z = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                y += all[(w * 8 + r) * HD + d];
                D += s_l[w][h];
            }
            if (!whole) {
                p.part[(row0 + r) * hd + d] = y;
                if (d == 0 && r < 4) p.sums[row0 + r] = make_float2(D, 0.f);
            } else if (r < 4) {
#pragma unroll
                for (int w = 0; w < kWarps; ++w) z += all[(w * 8 + r + 4) * HD + d];
                // (of one key there is no gradient, whatever its weight came to)
                store_float(static_cast<T *>(p.out) + (head0 + h) * hd + d, len == 1 ? 0.f : p.scale * fmaf(-D, z, y));
                if (d == 0) p.D[head0 + h] = D;
            }
        }
    }
    __syncthreads();                                           // before the next segment's queries and keys
    if (threadIdx.x == 0) {
        int2 *parts = p.parts + b * units + sg.unit;           // for the join
        if (sg.s0 == 0) parts->x = int(blockIdx.x) * 2 + sg.slot;
        if (sg.s1 == steps_of(len)) parts->y = int(blockIdx.x);
        const int64_t weight = kFixed + steps_of(len), from = sg.base + sg.unit * weight, to = min(sg.end, from + weight);
        sg.slot = 1;
        sg.pos = to;
        if (to == from + weight && sg.unit == units - 1) {
            sg.base = to;
            if (sg.pos < sg.end) sg.len = kv8_length(p.pg, ++sg.b);
        }
    }
  }
}

// Where the parts of a unit are: CTAs c0 .. c1, in their slot 0 but for c0's.
struct Parts {
    int c0, c1, slot0;
    __device__ __forceinline__ Parts(const AttnParams &p, int64_t b, int unit) {
        const int2 v = __ldcg(p.parts + b * p.c.n_kv_heads * p.tiles + unit);
        c0 = v.x >> 1;
        slot0 = v.x & 1;
        c1 = v.y;
    }
    __device__ __forceinline__ bool whole() const { return c0 == c1; }
    __device__ __forceinline__ int64_t row(int c, int r) const { return (int64_t(c) * 2 + (c == c0 ? slot0 : 0)) * 8 + r; }
};

constexpr int kJoinThreads = 256, kJoinWarps = kJoinThreads / 32;

// Gradients of the newest key and value of one (sequence, KV head) from what the pass left of it.
template <typename T>
__device__ __forceinline__ void newest_rows(const AttnParams &p, int64_t unit) {
    const int hd = p.c.head_dim, nkv = p.c.n_kv_heads, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int d = threadIdx.x;                                // head_dim <= 256
    const int64_t b = unit / nkv;
    const int kvh = int(unit - b * nkv);
    const int64_t row0 = b * p.n_heads + int64_t(kvh) * p.group;
    const int len = kv8_length(p.pg, b);
    const bool any = len > 0;
    __shared__ float2 s_w[kJoinWarps];                        // ds and p of a warp's head
    float dk = 0.f, dv = 0.f;
    for (int e0 = 0; e0 < p.group && any; e0 += kJoinWarps) {
        const int e = e0 + warp;
        if (e < p.group) {
            const Parts at(p, b, kvh * p.tiles + e / tile_heads(true));
            float D = 0.f;
            if (at.whole()) {
                D = __ldcg(p.D + row0 + e);
            } else {
                for (int c = at.c0 + lane; c <= at.c1; c += 32) D += __ldcg(&p.sums[at.row(c, e % tile_heads(true))].x);
                D = warp_sum(D);
            }
            const float2 w = __ldcg(p.newest + row0 + e);
            if (lane == 0) s_w[warp] = make_float2(len == 1 ? 0.f : w.x * (w.y - D) * p.scale, w.x);
        }
        __syncthreads();
        for (int i = 0; i < kJoinWarps && e0 + i < p.group && d < hd; ++i) {
            const int64_t at = (row0 + e0 + i) * hd + d;
            // a weight of 0 adds nothing (a newest key that is not there)
            if (s_w[i].x != 0.f) dk = fmaf(s_w[i].x, load_float(static_cast<const T *>(p.q) + at), dk);
            if (s_w[i].y != 0.f) dv = fmaf(s_w[i].y, load_float(static_cast<const T *>(p.d_ctx) + at), dv);
        }
        __syncthreads();
    }
    if (d < hd) {
        store_float(static_cast<T *>(p.d_k) + unit * hd + d, dk);
        store_float(static_cast<T *>(p.d_v) + unit * hd + d, dv);
    }
}

// Joins the parts of one query head, where its unit has more than one, in a fixed order: warps take every eighth, a
// lane four dimensions (and four from 128 on).  The gradient's last CTAs do the newest keys.
template <typename T, bool GRAD>
__global__ void __launch_bounds__(kJoinThreads) kv8_attn_join_kernel(const __grid_constant__ AttnParams p) {
    __shared__ float4 sum[GRAD ? 2 : 1][kJoinWarps][64];
    pdl_wait();
    const int64_t row = blockIdx.x;
    if (GRAD && row >= p.n_seq * p.n_heads) {
        newest_rows<T>(p, row - p.n_seq * p.n_heads);
        return;
    }
    const int hd = p.c.head_dim, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t b = row / p.n_heads;
    const int h = int(row - b * p.n_heads), kvh = h / p.group, e = h - kvh * p.group;
    constexpr int HT = tile_heads(GRAD);
    const Parts at(p, b, kvh * p.tiles + e / HT);
    if (at.whole()) return;
    const int r = e % HT;
    // the largest logit and the sum (gradient: D) of all parts, the same in every warp
    float top = -INFINITY, total = 0.f;
    if (!GRAD) {
        for (int c = at.c0 + lane; c <= at.c1; c += 32) top = fmaxf(top, __ldcg(&p.sums[at.row(c, r)].x));
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    }
    const float ref = top == -INFINITY ? 0.f : top;
    for (int c = at.c0 + lane; c <= at.c1; c += 32) {
        const float2 v = __ldcg(p.sums + at.row(c, r));
        total += GRAD ? v.x : v.y * ex2(v.x - ref);
    }
    total = warp_sum(total);
    for (int d = lane * 4, k = 0; k < 2; d += 128, ++k) {
        if (d >= hd) break;
        float4 y = make_float4(0.f, 0.f, 0.f, 0.f), z = y;
#pragma unroll 8
        for (int c = at.c0 + warp; c <= at.c1; c += kJoinWarps) {
            const int64_t from = at.row(c, r);
            const float4 v = __ldcg(reinterpret_cast<const float4 *>(p.part + from * hd + d));
            if (GRAD) {
                const float4 w = __ldcg(reinterpret_cast<const float4 *>(p.part + (from + 4) * hd + d));
                y.x += v.x; y.y += v.y; y.z += v.z; y.w += v.w;
                z.x += w.x; z.y += w.y; z.z += w.z; z.w += w.w;
            } else {
                const float f = ex2(__ldcg(&p.sums[from].x) - ref);
                y.x = fmaf(v.x, f, y.x); y.y = fmaf(v.y, f, y.y); y.z = fmaf(v.z, f, y.z); y.w = fmaf(v.w, f, y.w);
            }
        }
        sum[0][warp][k * 32 + lane] = y;
        if (GRAD) sum[GRAD ? 1 : 0][warp][k * 32 + lane] = z;
    }
    __syncthreads();
    for (int d = threadIdx.x; d < hd; d += kJoinThreads) {
        float a = 0.f, c = 0.f;
#pragma unroll
        for (int w = 0; w < kJoinWarps; ++w) {
            a += reinterpret_cast<const float *>(sum[0][w])[d];
            if (GRAD) c += reinterpret_cast<const float *>(sum[GRAD ? 1 : 0][w])[d];
        }
        store_float(static_cast<T *>(p.out) + row * hd + d,
                    GRAD ? p.scale * fmaf(-total, c, a) : total == 0.f ? 0.f : a / total);
    }
    if (!GRAD && threadIdx.x == 0) p.out_lse[row] = total == 0.f ? -INFINITY : fmaf(log2f(total), kLn2, top * kLn2);
}

bool sizes_ok(const tlb_kv8 *c, int64_t n_seq, int32_t n_heads, int64_t max_len) {
    return c != nullptr && n_seq >= 0 && max_len >= 0 && max_len <= (int64_t(1) << 30) && n_heads >= 1 && c->n_kv_heads >= 1 &&
           n_heads % c->n_kv_heads == 0 && n_heads <= 65535 && n_seq <= (int64_t(1) << 30) / n_heads && c->head_dim >= 1 &&
           c->head_dim % 16 == 0 && c->head_dim <= 256 && c->n_slots < (int64_t(1) << 31);
}

struct Layout {
    size_t part, sums, parts, newest, D, bytes;
};

// CTAs at a time: four an SM (two with heads of more than 128 values).
int cta_most(const tlb_kv8 &c) { return num_sms() * (c.head_dim <= 128 ? 4 : 2); }

Layout layout_of(const tlb_kv8 &c, int64_t n_seq, int n_heads, bool grad) {
    WsPlan p;
    Layout l{};
    const size_t rows = size_t(n_seq) * n_heads, parts = size_t(cta_most(c)) * 2 * 8;
    l.part = p.take(parts * c.head_dim * sizeof(float));
    l.sums = p.take(parts * sizeof(float2));
    l.parts = p.take(size_t(n_seq) * c.n_kv_heads * size_t(ceil_div(n_heads / c.n_kv_heads, tile_heads(grad))) * sizeof(int2));
    if (grad) {
        l.newest = p.take(rows * sizeof(float2));
        l.D = p.take(rows * sizeof(float));
    }
    l.bytes = p.off;
    return l;
}

size_t ws_bytes_of(const tlb_kv8 *c, int64_t n_seq, int32_t n_heads, int64_t max_len, bool grad) {
    if (!sizes_ok(c, n_seq, n_heads, max_len)) return 0;
    const size_t fwd = layout_of(*c, n_seq, n_heads, false).bytes, bwd = layout_of(*c, n_seq, n_heads, true).bytes;
    return grad && bwd > fwd ? bwd : fwd;
}

template <typename T, int HD, bool GRAD>
int attn_launch(const AttnParams &p, cudaStream_t st) {
    auto kernel = kv8_attn_kernel<T, HD, GRAD>;
    constexpr int smem = smem_bytes<HD, GRAD>();
    static_assert(smem >= kWarps * 8 * HD * 4, "the warps' sums fit where the stages were");
    if (smem > 48 * 1024) TLB_CUDA(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem));
    kernel<<<unsigned(p.ctas), kWarps * 32, smem, st>>>(p);
    TLB_TRY(check_launch(GRAD ? "kv8_attn_backward" : "kv8_attn_forward"));
    const int64_t rows = p.n_seq * p.n_heads + (GRAD ? p.n_seq * p.c.n_kv_heads : 0);
    TLB_CUDA(launch_dependent(kv8_attn_join_kernel<T, GRAD>, dim3(unsigned(rows)), dim3(kJoinThreads), 0, st, p));
    return check_launch("kv8_attn_join");
}

template <typename T, bool GRAD>
int attn_run(const AttnParams &p, cudaStream_t st) {
    return p.c.head_dim <= 64 ? attn_launch<T, 64, GRAD>(p, st)
           : p.c.head_dim <= 128 ? attn_launch<T, 128, GRAD>(p, st)
                                 : attn_launch<T, 256, GRAD>(p, st);
}

AttnParams params_of(const tlb_kv8 &c, const Kv8Pages &pg, int64_t n_seq, int n_heads, bool grad, float scale, const void *q,
                     void *ws) {
    const Layout l = layout_of(c, n_seq, n_heads, grad);
    AttnParams p{};
    p.c = c;
    p.pg = pg;
    p.n_seq = n_seq;
    p.n_heads = n_heads;
    p.group = n_heads / c.n_kv_heads;
    p.tiles = int(ceil_div(p.group, tile_heads(grad)));
    // no more than the longest sequences could fill (max_len bounds them)
    const int64_t units = n_seq * c.n_kv_heads * p.tiles, full = units * (kFixed + ceil_div(pg.max_len, kStep)) / kLeast;
    const int64_t parts = units * kMostParts, most = full < parts ? full : parts;
    p.ctas = int(most < cta_most(c) ? (most > 1 ? most : 1) : cta_most(c));
    p.scale = scale;
    p.q = q;
    p.part = ws_at<float>(ws, l.part);
    p.sums = ws_at<float2>(ws, l.sums);
    p.parts = ws_at<int2>(ws, l.parts);
    p.newest = ws_at<float2>(ws, l.newest);
    p.D = ws_at<float>(ws, l.D);
    return p;
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
    TLB_REQUIRE(aligned_to(pages, 4) && aligned_to(lengths, 4), TLB_EINVAL, "%s: pages and lengths must be aligned", what);
    const size_t need = ws_bytes_of(cache, n_seq, n_heads, max_len, grad);
    TLB_REQUIRE(ws != nullptr && ws_bytes >= need, TLB_EINVAL, "%s: workspace of %zu bytes is smaller than the %zu bytes needed",
                what, ws_bytes, need);
    TLB_REQUIRE((reinterpret_cast<uintptr_t>(ws) & 255) == 0, TLB_EINVAL, "%s: workspace must be 256-byte aligned", what);
    int64_t most = max_len;
    if (max_pages < (int64_t(1) << 31)) most = most < max_pages * page ? most : max_pages * page;
    if (cache->n_slots == 0) most = 0;                        // no key is there, and no address is made of the null pointers
    int shift = -1;
    if ((page & (page - 1)) == 0)
        for (shift = 0; (1 << shift) < page;) ++shift;
    pg = Kv8Pages{pages, lengths, max_pages, page, int32_t(most), shift};
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
    TLB_REQUIRE(aligned16(ctx) && aligned_to(lse, 4), TLB_EINVAL, "kv8_attn_forward: ctx must be 16-byte aligned, lse to its elements");
    AttnParams p = params_of(*cache, pg, n_seq, n_heads, false, scale, q, ws);
    p.out = ctx;
    p.out_lse = lse;
    return type == TLB_W_F32 ? attn_run<float, false>(p, as_stream(stream)) : attn_run<__nv_bfloat16, false>(p, as_stream(stream));
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
    TLB_REQUIRE(aligned16(d_ctx) && aligned16(d_q) && aligned16(d_k) && aligned16(d_v) && aligned_to(lse, 4), TLB_EINVAL,
                "kv8_attn_backward: d_ctx, d_q, d_k and d_v must be 16-byte aligned, lse to its elements");
    AttnParams p = params_of(*cache, pg, n_seq, n_heads, true, scale, q, ws);
    p.lse = lse;
    p.d_ctx = d_ctx;
    p.out = d_q;
    p.d_k = d_k;
    p.d_v = d_v;
    return type == TLB_W_F32 ? attn_run<float, true>(p, as_stream(stream)) : attn_run<__nv_bfloat16, true>(p, as_stream(stream));
}

}  // extern "C"
