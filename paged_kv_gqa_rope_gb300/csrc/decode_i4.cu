// Single-token GQA decode against the 4-bit pool (include/pa.h,
// pa_cache_i4_t): out = softmax(scale q K^T) V with K and V standing for
// m + s c.
//
// Work decomposition.  The blocks of all (sequence, KV head) pairs, each pair
// followed by kPairCost units for its fixed cost, laid end to end, form one
// line of W units, cut into equal ranges, one per WARP of a persistent grid
// (one CTA of 12 warps per SM).  A warp streams its range by itself into its
// own ring of shared memory (K and V of one block and KV head are 20 d
// contiguous bytes, which its lanes bring by 16-byte asynchronous copies), so
// no warp waits for another until the end.  A pair that lies within one range
// is finished by its warp; the pieces of a pair cut between warps are joined by
// the CTA once all its warps are done, and a pair cut between CTAs by the CTA
// whose record of it arrives last.  Every join sums in the order of the line,
// so the result does not depend on who arrives when.
//
// Bound: HBM on paper (1.25 d bytes per token and KV head); measured, the
// latency of dependent instructions at three warps a scheduler, which issue half
// the slots (2.0 of 4 an SM; of the waits a fixed latency is the longest, then
// the tensor and integer pipes): about 285 warp instructions and 22 MMAs a block,
// 5.4 TB/s on 32 x 32 heads of 2049 keys (62.3 us, 81 % of the copy peak; the same
// loads without the arithmetic take 53).  On short launches the edges, about 7 us
// to the first tiles and 5 to the joins (32 x 8 heads of 4097 keys: 40.1 us,
// 63 %).  Time grows in proportion from 12 warps an SM to 10, and 16 warps of
// 128 registers spill what they gain.
//
// Arithmetic, on warp-level MMAs (scores S^T = K Q^T and O^T = V^T P^T, the g
// heads that share the KV head being the N = 8 columns of both, so each code
// is unpacked once for the whole group):
//   - A code is used as the fp16 whose low bits it is: c 2^-24 (or 16 c 2^-24
//     for every other one, taken out of the other operand), exact, for one
//     logic operation per two codes.
//   - q k = sum over groups of  s (q . c) + m (sum of q): per group of 32 the
//     product of fp16 q and codes, scaled in fp32 by s; the second term one
//     MMA more, with the sums of q as the sum of two fp16.  q enters scaled by
//     a power of two to [2^9, 2^10), so nothing of it underflows.
//   - p v = sum over keys of  (p s)(c - 8) + p (m + 8 s): p s is rounded to
//     fp16 once, and so are p and the centre m + 8 s for their product (the
//     roundings of this kernel that show, as P's in the fp16 kernel); c - 8
//     rather than c, and the centre rather than the least value, keep both
//     terms as small as the values themselves, so the rounding is not magnified
//     by their cancelling.  c - 8 is the product with c and, from the same
//     rounded operand, 8 times its sum (one MMA a group; making c - 8 itself,
//     one packed add for each two codes, was slower: 77.9 against 75.4 us on
//     32 x 32 heads of 2049 keys).
//     Every other block enters as -(p s)(15 - c) and 7 times the sum instead:
//     the tensor core truncates its sums, and with c alone they grow to many
//     times the result (a warp's 575 blocks of even weights: 4.6e-3 off).  For
//     the same reason the sums of p s and of the centres are added up outside.
//   - Both roundings keep fp16's 11 bits over a wide range.  p is taken 2^13 times
//     as large (the maximum kept lies 13 below the scores', in log2; where steps
//     pass 1, by so much less that p s fits fp16).  Steps that stay at or below
//     2^-5 are multiplied by the power of two that brings the largest to
//     (1/2, 1].  So p s is normal down to 2^-22 of that of the largest score and
//     step, and below it off by at most 2^-33 of that, whatever the size of V; a
//     larger step scales the sums down as a larger score does.  (As they come,
//     beside one key with most of the weight the others' p s is subnormal or
//     nothing: 32768 keys with V of std 0.1, and a value of zero that had 0.9 of
//     the weight, came out with a relative error of 0.33.)  The small steps'
//     products are under a branch: 32 x 8 heads of 4097 keys take 39.9 us without
//     and 40.3 with them, 40.5 where they are always made.
//   - The running maximum is raised only when a score passes it by kLazy
//     (in log2), so P <= 2^(13 + kLazy) and O is rarely rescaled.
#include <mutex>

#include "common.cuh"
#include "internal.h"
#include "kv_int4.cuh"

namespace pa {
namespace {

constexpr int kMaxSeqs = 4096;
constexpr int kGroupPad = 8;  // Q heads per KV head, padded
constexpr int kWarps = 12;
constexpr int kThreads = kWarps * 32;
constexpr int kMaxGrid = 152;  // CTAs the workspace has records for
// Units of the line for a pair's fixed cost, in blocks: 64 histories of 16 to 16384
// tokens took 49.0, 46.4, 46.6, 46.8 and 47.0 us with 2, 3, 4, 6 and 8, so that 3 to
// 8 serve alike; equal histories do not care.  (One history of 32768 over 8 heads
// took 20.3, 20.2, 18.8, 19.9 and 19.8: with 4 its 8 (2048 + 4) units happen to be 9
// for each of the 1824 warps.)
constexpr int kPairCost = 4;
constexpr int kMinUnits = 4;   // least units of a warp's range
constexpr int kSeqStep = 4;    // sequences per entry of the prefix table
constexpr float kLazy = 2.f;
constexpr int kShift = 13;        // the maximum kept lies at most this far below the scores'
constexpr float kNoMax = -1e30f;  // running maximum before the first score

template <int D>
constexpr int kStages = D == 128 ? 3 : 6;  // stages of a warp's ring, two blocks each

struct DecodeI4Args {
    const __half *q;              // [B][H][D]
    const uint8_t *tiles;         // tile pairs of the layer
    const int32_t *block_tables;  // [B][maxb]
    const int32_t *context_lens;  // [B]
    __half *out;                  // [B][H][D]
    int32_t *counters;            // [B][H] arrivals (zero between calls)
    float *rec;                   // [grid][2][8][D + 4] O, then max, sum
    float *lead;                  // [grid][kWarps][8][D] O of a warp's first piece
    int32_t *status;
    float scale_log2;             // scale * log2(e)
    int B, H, Hk, g, maxb, num_blocks;
};

__device__ __forceinline__ int blocks_of(int ctx, int maxb) {
    return ctx >= 1 && ctx <= maxb * kBlockSize ? (ctx + kBlockSize - 1) / kBlockSize : 0;
}

__device__ __forceinline__ int64_t divide(int64_t a, int64_t b) {  // both >= 0, b > 0
    if (((a | b) >> 32) == 0) return (uint32_t)a / (uint32_t)b;
    return a / b;
}

// A pair on the line: its blocks are the units [start, start + nblk).
struct Pair {
    int64_t start;
    int s, kvh, nblk, ctx;

    __device__ __forceinline__ void load(const DecodeI4Args &a) {
        ctx = __ldg(a.context_lens + s);
        nblk = blocks_of(ctx, a.maxb);
    }
    // The pair that holds unit pos: `first`, at most kSeqStep sequences, starts
    // at unit `from` <= pos and holds it.
    __device__ __forceinline__ void find(int64_t pos, int first, int64_t from,
                                         const DecodeI4Args &a) {
        start = from;
        s = first;
        while (true) {
            load(a);
            const int64_t n = nblk ? (int64_t)(nblk + kPairCost) * a.Hk : 0;
            if (pos < start + n) break;
            start += n;
            ++s;
        }
        kvh = (int)divide(pos - start, nblk + kPairCost);
        start += (int64_t)kvh * (nblk + kPairCost);
    }
    // The next pair; only called while it starts before W.
    __device__ __forceinline__ void next(const DecodeI4Args &a) {
        start += nblk + kPairCost;
        if (++kvh < a.Hk) return;
        kvh = 0;
        do {
            ++s;
            load(a);
        } while (nblk == 0);
    }
};

// The line cut into A ranges of `per` units, the first `more` of them one longer.
struct Cuts {
    int64_t per, more;
    __device__ __forceinline__ Cuts(int64_t W, int A) {
        per = divide(W, A);
        more = W - per * A;
    }
    __device__ __forceinline__ int64_t start(int w) const { return per * w + min((int64_t)w, more); }
    __device__ __forceinline__ int range_of(int64_t unit) const {
        const int64_t longer = more * (per + 1);
        return (int)(unit < longer ? divide(unit, per + 1) : more + divide(unit - longer, per));
    }
};

// 16-byte asynchronous copy global -> shared through L2 only.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, uint64_t pol) {
    asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2;" ::"r"(dst),
                 "l"(src), "l"(pol)
                 : "memory");
}

// D(16x8, f32) = A(16x8, f16, row) * B(8x8, f16, col)
__device__ __forceinline__ void mma_1688_zero(float (&d)[4], uint32_t a0, uint32_t a1,
                                              uint32_t b0) {
    asm("mma.sync.aligned.m16n8k8.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5}, {%6},"
        " {%7, %7, %7, %7};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(b0), "f"(0.f));
}
// (mma_16816 without volatile: the compiler may move it among the others)
__device__ __forceinline__ void mma_add(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                        uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7},"
        " {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// D(16x8, f32) = A(16x16, f16, row) * B(16x8, f16, col)
__device__ __forceinline__ void mma_16816_zero(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                               uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7},"
        " {%8, %9}, {%10, %10, %10, %10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}

__device__ __forceinline__ void cp_async_commit() {
    asm volatile("cp.async.commit_group;" ::: "memory");
}
// (hi + lo) s of two fp16 pairs, or its negative, rounded to fp16 (lo s, far
// below it, before).
template <bool kNegative>
__device__ __forceinline__ uint32_t times(uint32_t hi, uint32_t lo, uint32_t s) {
    __half2 x = as_half2(s);
    if (kNegative) x = __hneg2(x);
    return as_u32(__hfma2(as_half2(hi), x, __hmul2(as_half2(lo), x)));
}
// Two outputs as fp16, saturated (a value m + 15 s may lie past 65504, and the
// roundings may carry a mean of values at the edge past it); a NaN stays one.
__device__ __forceinline__ uint32_t pack_out(float lo, float hi) {
    const __half2 top = __float2half2_rn(65504.f);
    return as_u32(__hmax2_nan(__hmin2_nan(__floats2half2_rn(lo, hi), top), __hneg2(top)));
}
// (movmatrix_trans without volatile)
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

// G consecutive words (G = 4 or 2) of shared memory, 4 G-byte aligned.
template <int G>
__device__ __forceinline__ void ld_words(uint32_t (&w)[G], const uint8_t *p) {
    if constexpr (G == 4) {
        const uint4 x = *reinterpret_cast<const uint4 *>(p);
        w[0] = x.x, w[1] = x.y, w[2] = x.z, w[3] = x.w;
    } else {
        const uint2 x = *reinterpret_cast<const uint2 *>(p);
        w[0] = x.x, w[1] = x.y;
    }
}

// One warp's state of the softmax over the keys it has seen of one pair.
// Lane = 4 r + t (r = 0..7, t = 0..3).  Head r: the Q fragments; heads 2 t, 2 t + 1:
// the scores of keys r and r + 8 of a block, m, l (this lane's keys only) and the
// accumulators of O^T, rows (values of V) 32 grp + 4 r + n:
//   o[2 grp][0..1] n = 0, [2..3] n = 1; o[2 grp + 1][0..1] n = 2, [2..3] n = 3,
// in units of 2^-24 (n even) and 2^-20 (n odd); row grp of z: the sum of p times
// the centre of group grp; e[grp]: -8 (or 7) times the sum of its p s.  m lies
// room - kLazy below the maximum; lim is the power of two (as two fp16) that no
// step so far passes, 1 for 2^-4 to 1; where it is below 1, o and e are sums of
// p s / lim.
template <int D>
struct State {
    static constexpr int G = D / 32;
    static constexpr uint32_t kLeastLim = 0x04000400u, kOneLim = 0x3c003c00u;  // 2^-14, 1
    uint32_t qb[G][4];  // B fragments of Q^T: a group's codes of weight 1, then of weight 16
    uint32_t qsum;      // B fragment of the groups' sums of q, high and low parts
    float qs[2];        // scores -> log2 units
    float m[2], l[2];
    float o[2 * G][4];
    uint64_t z, e[G];
    uint32_t lim;
    float room;

    __device__ __forceinline__ void begin(const DecodeI4Args &a, const Pair &p, int lane) {
        const int r = lane >> 2, t = lane & 3;
        uint4 x[G];
        const uint4 *row = reinterpret_cast<const uint4 *>(
            a.q + ((int64_t)p.s * a.H + p.kvh * a.g + (r < a.g ? r : 0)) * D);
        __half2 big = __float2half2_rn(0.f);
#pragma unroll
        for (int i = 0; i < G; ++i) {
            x[i] = r < a.g ? row[4 * i + t] : make_uint4(0, 0, 0, 0);
            const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
            for (int k = 0; k < 4; ++k)
                big = __hmax2(big, __habs2(*reinterpret_cast<const __half2 *>(&w[k])));
        }
        float amax = fmaxf(__low2float(big), __high2float(big));
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
        // 2^(9 - floor(log2 amax)) and its inverse
        const int ex = __float_as_int(amax) >> 23;
        const bool fine = amax > 0.f && amax <= 65504.f;
        const float up = fine ? __int_as_float((263 - ex) << 23) : 1.f;
        const float down = a.scale_log2 * 0x1p24f * (fine ? __int_as_float((ex - 9) << 23) : 1.f);
        qs[0] = __shfl_sync(0xffffffffu, down, 8 * t);
        qs[1] = __shfl_sync(0xffffffffu, down, 8 * t + 4);
        float sum[G];
#pragma unroll
        for (int i = 0; i < G; ++i) {
            const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
            float f[8];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float2 y = __half22float2(*reinterpret_cast<const __half2 *>(&w[k]));
                f[2 * k] = y.x * up;
                f[2 * k + 1] = y.y * up;
            }
            // codes 0, 4 | 2, 6 at weight 1; codes 1, 5 | 3, 7 at weight 16
            qb[i][0] = pack_half2(f[0], f[4]);
            qb[i][1] = pack_half2(f[2], f[6]);
            qb[i][2] = pack_half2(f[1] * 0.0625f, f[5] * 0.0625f);
            qb[i][3] = pack_half2(f[3] * 0.0625f, f[7] * 0.0625f);
            sum[i] = ((f[0] + f[1]) + (f[2] + f[3])) + ((f[4] + f[5]) + (f[6] + f[7]));
            sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], 1);
            sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], 2);
        }
        // k = 0 .. G - 1 the high parts, G .. 2 G - 1 the low parts
        qsum = 0;
#pragma unroll
        for (int i = 0; i < G; i += 2) {
            const __half h0 = __float2half_rn(sum[i]), h1 = __float2half_rn(sum[i + 1]);
            const __half2 hi = __halves2half2(h0, h1);
            if (t == i / 2) qsum = *reinterpret_cast<const uint32_t *>(&hi);
            if (t == (G + i) / 2)
                qsum = pack_half2(sum[i] - __half2float(h0), sum[i + 1] - __half2float(h1));
        }
        m[0] = m[1] = kNoMax;
        l[0] = l[1] = 0.f;
#pragma unroll
        for (int i = 0; i < 2 * G; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
        z = f2_pack(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < G; ++i) e[i] = f2_pack(0.f, 0.f);
        lim = kLeastLim;
        room = kShift + kLazy;
    }

    // One block, its tile pair at `kt` in shared memory.  With kTail, only its
    // first `valid` tokens count; kFlip: V's codes enter as 15 - c.
    template <bool kTail, bool kFlip>
    __device__ __forceinline__ void block(const uint8_t *kt, int valid, int lane) {
        const int r = lane >> 2, t = lane & 3;
        using T = I4Tile<D>;
        // scores of keys r (y[0..1]: heads 2 t, 2 t + 1) and r + 8 (y[2..3])
        float y[4];
        uint32_t w[2][G];
#pragma unroll
        for (int h = 0; h < 2; ++h) ld_words<G>(w[h], kt + (8 * h + r) * (D / 2) + t * (4 * G));
        {
            const uint8_t *par = kt + T::kCodes + 2 * (16 * G + G * r) + (G == 4 ? (t & 1) * 4 : 0);
            float d[4];
            mma_1688_zero(d, *reinterpret_cast<const uint32_t *>(par),
                          *reinterpret_cast<const uint32_t *>(par + 16 * G), qsum);
#pragma unroll
            for (int k = 0; k < 4; ++k) y[k] = d[k] * 0x1p-24f;
        }
#pragma unroll
        for (int gr = 0; gr < G; ++gr) {
            const uint32_t v0 = w[0][gr], v1 = w[1][gr], u0 = v0 >> 8, u1 = v1 >> 8;
            const uint32_t a0[4] = {v0 & 0x000f000fu, v1 & 0x000f000fu, u0 & 0x000f000fu,
                                    u1 & 0x000f000fu};
            const uint32_t a1[4] = {v0 & 0x00f000f0u, v1 & 0x00f000f0u, u0 & 0x00f000f0u,
                                    u1 & 0x00f000f0u};
            float d[4];
            mma_16816_zero(d, a0, qb[gr][0], qb[gr][1]);
            mma_add(d, a1, qb[gr][2], qb[gr][3]);
            const __half *st = reinterpret_cast<const __half *>(
                kt + T::kCodes + 8 * (G * (r >> 1) + gr) + 2 * (r & 1));
            const float s0 = __half2float(st[0]), s1 = __half2float(st[2]);
            y[0] = fmaf(d[0], s0, y[0]);
            y[1] = fmaf(d[1], s0, y[1]);
            y[2] = fmaf(d[2], s1, y[2]);
            y[3] = fmaf(d[3], s1, y[3]);
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            y[k] *= qs[k & 1];
            if (kTail && r + 8 * (k >> 1) >= valid) y[k] = -INFINITY;
        }
        float top[2] = {fmaxf(y[0], y[2]), fmaxf(y[1], y[3])};
        const uint8_t *vt = kt + T::kBytes, *par = vt + T::kCodes;
        // V's steps of keys 2 t, + 1, + 8, + 9 and group r % G
        const int row = 8 * (G * t + (r & (G - 1)));
        uint2 ss = *reinterpret_cast<const uint2 *>(par + row);
        uint32_t k0 = 0, k1 = 0;
        if (kTail) {
            // parameters of tokens that do not count may be anything, NaN included
            k0 = (2 * t < valid ? 0x0000ffffu : 0u) | (2 * t + 1 < valid ? 0xffff0000u : 0u);
            k1 = (2 * t + 8 < valid ? 0x0000ffffu : 0u) | (2 * t + 9 < valid ? 0xffff0000u : 0u);
            ss.x &= k0;
            ss.y &= k1;
        }
        const uint32_t big = as_u32(__hmax2(as_half2(ss.x), as_half2(ss.y)));
        if (__any_sync(0xffffffffu, top[0] > __fadd_rd(m[0], room) ||
                                        top[1] > __fadd_rd(m[1], room) ||
                                        !__hble2(as_half2(big), as_half2(lim)))) {
            // the limits' exponents, 15 for 1
            const int was = (int)((lim >> 10) & 31u);
            const uint32_t most = __reduce_max_sync(0xffffffffu, max(big & 0xffffu, big >> 16));
            int now = max(was, min(29, (int)((most + 0x3ffu) >> 10)));
            if (now > 10 && now < 15) now = 15;
            lim = (uint32_t)now * 0x04000400u;
            const float scaled = __int_as_float((127 + min(was, 15) - min(now, 15)) << 23);
            const float shift = (float)max(0, kShift - max(0, now - 15));
            const float less = room - kLazy - shift;  // what the maxima kept come nearer by
            room = shift + kLazy;
#pragma unroll
            for (int k = 0; k < 2; ++k) {
#pragma unroll
                for (int f = 4; f < 32; f <<= 1)
                    top[k] = fmaxf(top[k], __shfl_xor_sync(0xffffffffu, top[k], f));
                // (rounded so that top - n <= room, however large the scores)
                float n = __fadd_ru(m[k], less);
                if (top[k] > __fadd_rd(n, room)) n = __fsub_ru(top[k], shift);
                const float f = ex2(m[k] - n);
                m[k] = n;
                l[k] *= f;
                top[k] = f;
            }
            z = f2_mul(z, f2_pack(top[0], top[1]));
            top[0] *= scaled;
            top[1] *= scaled;
#pragma unroll
            for (int k = 0; k < 2 * G; ++k) {
                o[k][0] *= top[0];
                o[k][1] *= top[1];
                o[k][2] *= top[0];
                o[k][3] *= top[1];
            }
            const uint64_t both = f2_pack(top[0], top[1]);
#pragma unroll
            for (int k = 0; k < G; ++k) e[k] = f2_mul(e[k], both);
        }
        // p as the sum of two fp16 (so that its product with a step is rounded
        // once), transposed to head r, keys 2 t, + 1 ([0]), + 8, + 9 ([1])
        uint32_t hi[2], lo[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const float p0 = ex2(y[2 * k] - m[0]), p1 = ex2(y[2 * k + 1] - m[1]);
            l[0] += p0;
            l[1] += p1;
            const uint32_t x = pack_half2(p0, p1);
            const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&x));
            hi[k] = transpose8(x);
            lo[k] = transpose8(pack_half2(p0 - f.x, p1 - f.y));
        }
        uint32_t st[2][G];
        ld_words<G>(st[0], par + t * (8 * G));
        ld_words<G>(st[1], par + t * (8 * G) + 4 * G);
        // row r % G of the centre's operand: m + 8 s of keys 2 t, + 1, + 8, + 9
        const uint2 ls = *reinterpret_cast<const uint2 *>(par + 32 * G + row);
        const __half2 eight = __float2half2_rn(8.f);
        uint32_t za[2] = {as_u32(__hfma2(as_half2(ss.x), eight, as_half2(ls.x))),
                          as_u32(__hfma2(as_half2(ss.y), eight, as_half2(ls.y)))};
        uint32_t w0[G], w1[G];  // word grp: keys 2 t (low half), 2 t + 1; then + 8
        ld_words<G>(w0, vt + lane * (4 * G));
        ld_words<G>(w1, vt + lane * (4 * G) + 4 * D);
        if (lim < kOneLim) {
            const __half2 sc = as_half2(2 * kOneLim - lim);  // 1 / lim
#pragma unroll
            for (int k = 0; k < G; ++k) {
                st[0][k] = as_u32(__hmul2(as_half2(st[0][k]), sc));
                st[1][k] = as_u32(__hmul2(as_half2(st[1][k]), sc));
            }
        }
        if (kTail) {
#pragma unroll
            for (int k = 0; k < G; ++k) {
                st[0][k] &= (k & 1) ? k1 : k0;
                st[1][k] &= (k & 1) ? k1 : k0;
            }
            za[0] &= k0;
            za[1] &= k1;
        }
        {  // (rows 8-15 of the operand and the product are not used)
            const uint32_t a4[4] = {za[0], za[0], za[1], za[1]};
            float d[4];
            mma_16816_zero(d, a4, hi[0], hi[1]);
            z = f2_add(z, f2_pack(d[0], d[1]));
        }
        // -8, or -7 beside the negated p s
        constexpr uint32_t kOff = kFlip ? 0xc700c700u : 0xc800c800u;
        const uint32_t off[4] = {kOff, kOff, kOff, kOff};
#pragma unroll
        for (int gr = 0; gr < G; ++gr) {
            const uint32_t *sw = &st[gr / (G / 2)][2 * (gr % (G / 2))];
            const uint32_t b0 = times<kFlip>(hi[0], lo[0], sw[0]);
            const uint32_t b1 = times<kFlip>(hi[1], lo[1], sw[1]);
            const uint32_t v0 = kFlip ? ~w0[gr] : w0[gr], v1 = kFlip ? ~w1[gr] : w1[gr];
            const uint32_t u0 = v0 >> 8, u1 = v1 >> 8;
            const uint32_t a0[4] = {v0 & 0x000f000fu, v0 & 0x00f000f0u, v1 & 0x000f000fu,
                                    v1 & 0x00f000f0u};
            const uint32_t a1[4] = {u0 & 0x000f000fu, u0 & 0x00f000f0u, u1 & 0x000f000fu,
                                    u1 & 0x00f000f0u};
            mma_add(o[2 * gr], a0, b0, b1);
            mma_add(o[2 * gr + 1], a1, b0, b1);
            float d[4];
            mma_16816_zero(d, off, b0, b1);
            e[gr] = f2_add(e[gr], f2_pack(d[0], d[1]));
        }
    }

    // l over all keys; O of heads 2 t + (0, 1): v[grp][head][n], values 32 grp + 4 r + n.
    __device__ __forceinline__ void end(float (&v)[G][2][4], int lane) {
        const int t = lane & 3;
        const float unit = __int_as_float((127 - 15 + min(15, (int)((lim >> 10) & 31u))) << 23);
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int f = 4; f < 32; f <<= 1) l[k] += __shfl_xor_sync(0xffffffffu, l[k], f);
#pragma unroll
        for (int gr = 0; gr < G; ++gr) {
            float es[2], zs[2];
            f2_unpack(e[gr], es[0], es[1]);
            f2_unpack(z, zs[0], zs[1]);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const float zz = fmaf(es[h], unit, __shfl_sync(0xffffffffu, zs[h], 4 * gr + t));
                v[gr][h][0] = fmaf(o[2 * gr][h], 0x1p24f * unit, zz);
                v[gr][h][1] = fmaf(o[2 * gr][2 + h], 0x1p20f * unit, zz);
                v[gr][h][2] = fmaf(o[2 * gr + 1][h], 0x1p24f * unit, zz);
                v[gr][h][3] = fmaf(o[2 * gr + 1][2 + h], 0x1p20f * unit, zz);
            }
        }
    }
};

// What a warp leaves of a pair that it does not finish by itself.
struct Piece {
    int64_t start;  // the pair's first unit; negative (its own for each piece): none
    int row;        // the pair's first row of the output
    int first, n;   // the CTAs that hold the pair, if there are several (n = 0: only this one)
    int pad;
};

template <int D>
struct Smem {
    alignas(128) uint8_t ring[kWarps][kStages<D>][2 * 20 * D];
    float m[2 * kWarps][kGroupPad], l[2 * kWarps][kGroupPad];
    Piece piece[2 * kWarps];  // 2 w: the warp's first, begun by another; 2 w + 1: its last
    int64_t prefix[kMaxSeqs / kSeqStep + 1];
};

// A row (one head) of partial results: D / 32 columns a lane, from column lane D / 32.
template <int D>
struct Row {
    static constexpr int N = D / 32;
    float o[N], m, l;

    __device__ __forceinline__ void add(float f, const float (&v)[N]) {
#pragma unroll
        for (int i = 0; i < N; ++i) o[i] = __fmaf_rn(f, v[i], o[i]);
    }
    __device__ __forceinline__ void store_out(__half *row, int lane) const {
        const float inv = l != 0.f ? 1.f / l : 0.f;
        if constexpr (N == 4)
            *reinterpret_cast<uint2 *>(row + lane * 4) =
                make_uint2(pack_out(o[0] * inv, o[1] * inv), pack_out(o[2] * inv, o[3] * inv));
        else
            *reinterpret_cast<uint32_t *>(row + lane * 2) = pack_out(o[0] * inv, o[1] * inv);
    }
};
// N consecutive floats that another CTA or warp may have written.
template <int N>
__device__ __forceinline__ void load_cols(float (&v)[N], const float *p) {
    if constexpr (N == 4) {
        const float4 x = __ldcg(reinterpret_cast<const float4 *>(p));
        v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w;
    } else {
        const float2 x = __ldcg(reinterpret_cast<const float2 *>(p));
        v[0] = x.x, v[1] = x.y;
    }
}
template <int N>
__device__ __forceinline__ void store_cols(float *p, const float (&v)[N]) {
    if constexpr (N == 4)
        *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
    else
        *reinterpret_cast<float2 *>(p) = make_float2(v[0], v[1]);
}
__device__ __forceinline__ float warp_max(float x) {
#pragma unroll
    for (int f = 16; f; f >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, f));
    return x;
}
__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
    for (int f = 16; f; f >>= 1) x += __shfl_xor_sync(0xffffffffu, x, f);
    return x;
}

// One head's row of a pair cut between CTAs first .. first + n - 1, from their
// records; the row of CTA first + own (none if own < 0) is `mine` instead.
template <int D>
__device__ __forceinline__ Row<D> join_records(const DecodeI4Args &a, int first, int n, int h,
                                               int own, const Row<D> &mine, int lane) {
    constexpr int N = Row<D>::N;
    // the first CTA holds the pair as its last (slot 1), the others as their first
    auto rec = [&](int k) {
        return a.rec + (((int64_t)(first + k) * 2 + (k == 0)) * kGroupPad + h) * (D + 4);
    };
    // Up to 32 records, a lane for each: their (max, sum) and the O of the first
    // eight are asked for together, so that a short join waits once.
    constexpr int kBatch = 8;
    Row<D> r;
    r.m = kNoMax;
    r.l = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) r.o[i] = 0.f;
    for (int k0 = 0; k0 < n; k0 += 32) {
        const int c = min(32, n - k0);
        float m = kNoMax, l = 0.f;
        if (lane < c) {
            m = __ldcg(rec(k0 + lane) + D);  // (own record: in bounds, not used)
            l = __ldcg(rec(k0 + lane) + D + 1);
        }
        float v[kBatch][N];
        auto ask = [&](int j) {
#pragma unroll
            for (int i = 0; i < kBatch; ++i)
                load_cols<N>(v[i], rec(k0 + min(j + i, c - 1)) + lane * N);
        };
        ask(0);
        if (k0 + lane == own) {
            m = mine.m;
            l = mine.l;
        }
        const float M = fmaxf(r.m, warp_max(m)), old = ex2(r.m - M);
        const float f = lane < c ? ex2(m - M) : 0.f;
        r.m = M;
        r.l = r.l * old + warp_sum(f * l);
#pragma unroll
        for (int i = 0; i < N; ++i) r.o[i] *= old;
        for (int j = 0; j < c; j += kBatch) {
            if (j) ask(j);
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                if (j + i >= c) break;
                if (k0 + j + i == own)
#pragma unroll
                    for (int d = 0; d < N; ++d) v[i][d] = mine.o[d];
                r.add(__shfl_sync(0xffffffffu, f, j + i), v[i]);
            }
        }
    }
    return r;
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1) decode_i4_kernel(const DecodeI4Args a) {
    extern __shared__ __align__(128) uint8_t smem_raw[];
    Smem<D> &sm = *reinterpret_cast<Smem<D> *>(smem_raw);
    constexpr int R = kStages<D>, G = D / 32, kPairBytes = 20 * D;
    static_assert(sizeof(sm.ring[0]) >= kGroupPad * D * sizeof(float), "a piece's O fits the ring");
    static_assert(2 * kWarps <= 32, "a lane for each piece");
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int cta = blockIdx.x;

    // The work before this kernel may still be writing the context lengths; were
    // CTAs to read different ones, their cuts would not match.  (Reading them
    // ahead of this wait would save 0.5 to 0.7 us a call.)
    griddep_wait();

    // -------- units of every kSeqStep sequences and their prefix sums
    const int entries = (a.B + kSeqStep - 1) / kSeqStep;
    for (int i = tid; i < entries; i += kThreads) {
        int64_t n = 0;
#pragma unroll
        for (int k = 0; k < kSeqStep; ++k) {
            const int s = i * kSeqStep + k;
            if (s >= a.B) break;
            const int nblk = blocks_of(__ldg(a.context_lens + s), a.maxb);
            if (nblk)
                n += nblk + kPairCost;
            else if (cta == 0)
                report(a.status, PA_DEV_BAD_LENGTH);
        }
        sm.prefix[i + 1] = n * a.Hk;
    }
    if (lane == 0) {  // (by the lane that may overwrite them)
        sm.piece[2 * warp].start = -1 - 2 * warp;
        sm.piece[2 * warp + 1].start = -2 - 2 * warp;
    }
    if (tid == 0) sm.prefix[0] = 0;
    __syncthreads();
    if (warp == 0) prefix_sums(sm.prefix, entries, lane);
    __syncthreads();
    const int64_t W = sm.prefix[entries];
    griddep_launch_dependents();
    if (W == 0) return;
    const int A = (int)min((int64_t)gridDim.x * kWarps, (W + kMinUnits - 1) / kMinUnits);
    if (cta * kWarps >= A) return;
    const int me = cta * kWarps + warp;
    const Cuts cuts(W, A);
    const int c0 = cta * kWarps;
    const int64_t cta_begin = cuts.start(c0), cta_end = cuts.start(min(A, c0 + kWarps));

    if (me < A) {
        const int64_t begin = cuts.start(me), end = cuts.start(me + 1);
        const uint64_t pol = [] {
            uint64_t p;
            asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(p));
            return p;
        }();
        Pair cur;  // the pair being attended to
        {
            int lo = 0, hi = entries - 1;  // largest entry at or before `begin`
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (sm.prefix[mid] <= begin)
                    lo = mid;
                else
                    hi = mid - 1;
            }
            cur.find(begin, lo * kSeqStep, sm.prefix[lo], a);
        }
        Pair nxt = cur;  // the pair being loaded
        int ib, ie;      // its next block to load, and the end of those in the range
        int chunk;       // block of lane 0's entry
        int entry, entry2;  // block ids of blocks chunk + lane, chunk + 32 + lane
        const uint32_t block_stride = (uint32_t)a.Hk * kPairBytes;
        const uint8_t *tiles;  // of nxt's KV head, this lane's first 16 bytes

        auto open = [&](int64_t pos) {  // blocks of nxt in [pos, end)
            ib = (int)min((int64_t)nxt.nblk, pos - nxt.start);
            ie = (int)min((int64_t)nxt.nblk, end - nxt.start);
            chunk = ib;
            const int32_t *row = a.block_tables + (int64_t)nxt.s * a.maxb;
            entry = ib + lane < ie ? __ldg(row + ib + lane) : 0;
            entry2 = ib + 32 + lane < ie ? __ldg(row + ib + 32 + lane) : 0;
            tiles = a.tiles + nxt.kvh * kPairBytes + lane * 16;
        };
        // A stage takes the next two blocks of the range, or a pair's last one
        // (a block that cannot be loaded is left out and marked); each is one group
        // of copies, so that of the R stages in flight the oldest has landed
        // when at most R - 1 groups are outstanding.
        uint32_t bad = 0;  // bit 2 stage + block
        auto copy = [&](uint8_t *dst, int blk) {
            const uint8_t *src = tiles + (uint64_t)(uint32_t)blk * block_stride;
            const uint32_t to = smem_u32(dst) + lane * 16;
#pragma unroll
            for (int k = 0; k < kPairBytes; k += 512)
                if (k + 512 <= kPairBytes || lane * 16 < kPairBytes - k)
                    cp_async16(to + k, src + k, pol);
        };
        auto issue = [&](uint8_t *dst, int stage) {
            if (ib + 2 > min(ie, chunk + 32)) {
                while (ib >= ie) {
                    const int64_t pos = nxt.start + nxt.nblk + kPairCost;
                    if (pos >= end) {
                        cp_async_commit();
                        return;
                    }
                    nxt.next(a);
                    open(pos);
                }
                if (ib == chunk + 32) {  // (chunks and stages both begin at the pair's first block)
                    chunk = ib;
                    entry = entry2;
                    entry2 = ib + 32 + lane < ie
                                 ? __ldg(a.block_tables + (int64_t)nxt.s * a.maxb + ib + 32 + lane)
                                 : 0;
                }
            }
            const int blk0 = __shfl_sync(0xffffffffu, entry, ib - chunk);
            const int blk1 = __shfl_sync(0xffffffffu, entry, (ib - chunk + 1) & 31);
            if (ib + 1 < ie && max((unsigned)blk0, (unsigned)blk1) < (unsigned)a.num_blocks) {
                copy(dst, blk0);
                copy(dst + kPairBytes, blk1);
            } else {
                for (int i = 0; i < 2 && ib + i < ie; ++i) {
                    const int blk = i ? blk1 : blk0;
                    if ((unsigned)blk < (unsigned)a.num_blocks) {
                        copy(dst + i * kPairBytes, blk);
                    } else {
                        if (lane == 0) report(a.status, PA_DEV_BAD_BLOCK);
                        bad |= 1u << (2 * stage + i);
                    }
                }
            }
            cp_async_commit();
            ib += 2;
        };

        open(begin);
        // The first stage alone before Q is asked for, so that every warp's first
        // blocks arrive ahead of the later stages' (28 MB over all warps).
        issue(sm.ring[warp][0], 0);
        int get = 0;
        bool primed = false;
        State<D> st;
        for (int64_t pos = begin; pos < end;) {
            const int b0 = (int)min((int64_t)cur.nblk, pos - cur.start);
            const int b1 = (int)min((int64_t)cur.nblk, end - cur.start);
            if (b0 < b1) {
                st.begin(a, cur, lane);
                if (!primed) {
                    for (int i = 1; i < R; ++i) issue(sm.ring[warp][i], i);
                    primed = true;
                }
                // blocks whose tokens all count
                const int full_end = min(b1, cur.ctx / kBlockSize);
                for (int b = b0; b < b1; b += 2) {
                    asm volatile("cp.async.wait_group %0;" ::"n"(R - 1) : "memory");
                    __syncwarp();  // every lane's copies of the stage have landed
                    uint8_t *at = sm.ring[warp][get];
                    if (b + 2 <= full_end && bad == 0) {
                        st.template block<false, false>(at, kBlockSize, lane);
                        st.template block<false, true>(at + kPairBytes, kBlockSize, lane);
                    } else {
                        for (int i = 0; i < 2 && b + i < b1; ++i) {
                            const uint32_t bit = 1u << (2 * get + i);
                            st.template block<true, false>(
                                at + i * kPairBytes,
                                (bad & bit) ? 0 : min(kBlockSize, cur.ctx - (b + i) * kBlockSize),
                                lane);
                            bad &= ~bit;
                        }
                    }
                    __syncwarp();  // every lane has read the stage
                    issue(at, get);
                    get = get + 1 == R ? 0 : get + 1;
                }
                float v[G][2][4];
                st.end(v, lane);
                const int r = lane >> 2, t = lane & 3;
                if (b0 == 0 && b1 == cur.nblk) {  // the whole pair
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const float inv = st.l[h] != 0.f ? 1.f / st.l[h] : 0.f;
                        if (2 * t + h < a.g) {
                            __half *row = a.out + ((int64_t)cur.s * a.H + cur.kvh * a.g + 2 * t + h) * D;
#pragma unroll
                            for (int gr = 0; gr < G; ++gr)
                                *reinterpret_cast<uint2 *>(row + 32 * gr + 4 * r) =
                                    make_uint2(pack_out(v[gr][h][0] * inv, v[gr][h][1] * inv),
                                               pack_out(v[gr][h][2] * inv, v[gr][h][3] * inv));
                        }
                    }
                } else {
                    // A pair that ends in this range leaves its O in the
                    // workspace (the ring still streams); one that goes on, the
                    // warp's last, in the ring, which is empty by then.
                    const int k = b1 == cur.nblk ? 0 : 1;
                    float *dst = k == 0 ? a.lead + (int64_t)me * kGroupPad * D
                                        : reinterpret_cast<float *>(sm.ring[warp]);
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        if (2 * t + h < a.g)
#pragma unroll
                            for (int gr = 0; gr < G; ++gr)
                                *reinterpret_cast<float4 *>(dst + (2 * t + h) * D + 32 * gr + 4 * r) =
                                    make_float4(v[gr][h][0], v[gr][h][1], v[gr][h][2], v[gr][h][3]);
                    if (r == 0) {
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            sm.m[2 * warp + k][2 * t + h] = st.m[h];
                            sm.l[2 * warp + k][2 * t + h] = st.l[h];
                        }
                    }
                    if (lane == 0) {
                        Piece p;
                        p.start = cur.start;
                        p.row = cur.s * a.H + cur.kvh * a.g;
                        p.first = p.n = p.pad = 0;
                        if (cur.start < cta_begin || cur.start + cur.nblk > cta_end) {
                            p.first = cuts.range_of(cur.start) / kWarps;
                            p.n = cuts.range_of(cur.start + cur.nblk - 1) / kWarps - p.first + 1;
                        }
                        sm.piece[2 * warp + k] = p;
                    }
                }
            }
            pos = cur.start + cur.nblk + kPairCost;
            if (pos < end) cur.next(a);
        }
    }
    __syncthreads();

    // -------- pairs cut between warps.  In every warp, lane k speaks for piece
    // k (in the order of the line) and knows the pieces of the same pair.
    Piece p;
    p.start = -1 - lane;
    p.row = p.first = p.n = 0;
    if (lane < 2 * kWarps) p = sm.piece[lane];
    const uint32_t same = __match_any_sync(0xffffffffu, (unsigned long long)p.start);
    const uint32_t heads = __ballot_sync(0xffffffffu, p.start >= 0 && lane == __ffs(same) - 1);
    constexpr int N = Row<D>::N;
    const int rows = __popc(heads) * a.g;
    for (int x = warp; x < rows; x += kWarps) {  // a row (one head) per warp
        // the last pair's rows, then the others': those cut between CTAs, the
        // last pair and the first, are the ones that another CTA may wait for
        const int h = x % a.g;
        int which = x / a.g - 1;
        if (which < 0) which = __popc(heads) - 1;
        uint32_t rest = heads;
        for (int k = which; k > 0; --k) rest &= rest - 1;
        const int lead = __ffs(rest) - 1;
        const uint32_t members = __shfl_sync(0xffffffffu, same, lead);
        const int qrow = __shfl_sync(0xffffffffu, p.row, lead) + h;
        // A row cut between CTAs: each leaves a record of it (slot 1 the pair's
        // first CTA, whose last pair it is, slot 0 the others) and arrives on the
        // row's counter; the last joins the records.  If the others' have all
        // arrived already, this CTA needs neither record nor arrival of its own.
        const int first = __shfl_sync(0xffffffffu, p.first, lead);
        const int n = __shfl_sync(0xffffffffu, p.n, lead);
        // A piece in the workspace (the members' last, if any) is asked for first.
        const int tail = 31 - __clz(members);
        float v[N];
        if (!(tail & 1))
            load_cols<N>(v, a.lead + ((int64_t)(c0 + (tail >> 1)) * kGroupPad + h) * D + lane * N);
        int seen = 0;
        if (n && lane == 0)
            asm volatile("ld.relaxed.gpu.global.s32 %0, [%1];"
                         : "=r"(seen)
                         : "l"(a.counters + qrow)
                         : "memory");
        const bool in = members >> lane & 1;
        const float pm = in ? sm.m[lane][h] : kNoMax;
        Row<D> r;
        r.m = warp_max(pm);
        const float f = in ? ex2(pm - r.m) : 0.f;
        r.l = warp_sum(in ? f * sm.l[lane][h] : 0.f);
#pragma unroll
        for (int i = 0; i < N; ++i) r.o[i] = 0.f;
        for (uint32_t left = members & 0xaaaaaaaau; left; left &= left - 1) {
            const int k = __ffs(left) - 1;
            const float *o = reinterpret_cast<const float *>(sm.ring[k >> 1]);
            float w[N];
#pragma unroll
            for (int i = 0; i < N; ++i) w[i] = o[h * D + lane * N + i];
            r.add(__shfl_sync(0xffffffffu, f, k), w);
        }
        if (!(tail & 1)) r.add(__shfl_sync(0xffffffffu, f, tail), v);
        if (n) {
            int own = cta - first;
            if (__shfl_sync(0xffffffffu, seen, 0) != n - 1) {
                float *rec =
                    a.rec + (((int64_t)cta * 2 + (own == 0)) * kGroupPad + h) * (D + 4);
                store_cols<N>(rec + lane * N, r.o);
                if (lane == 0) {
                    rec[D] = r.m;
                    rec[D + 1] = r.l;
                }
                __syncwarp();
                if (lane == 0) {
                    asm volatile("fence.acq_rel.gpu;" ::: "memory");
                    seen = atomicAdd(a.counters + qrow, 1);
                    asm volatile("fence.acq_rel.gpu;" ::: "memory");
                }
                if (__shfl_sync(0xffffffffu, seen, 0) != n - 1) continue;
                own = -1;
            } else {
                asm volatile("fence.acq_rel.gpu;" ::: "memory");
            }
            __syncwarp();
            r = join_records<D>(a, first, n, h, own, r, lane);
            if (lane == 0) a.counters[qrow] = 0;
        }
        r.store_out(a.out + (int64_t)qrow * D, lane);
    }
}

// The workspace: records, first pieces, counters.  The counters must stay zero
// between calls of any shape, so they lie behind areas whose sizes no shape
// changes (head_dim 128's).
constexpr size_t kRecBytes = (size_t)kMaxGrid * 2 * kGroupPad * (128 + 4) * sizeof(float);
constexpr size_t kLeadBytes = (size_t)kMaxGrid * kWarps * kGroupPad * 128 * sizeof(float);
static_assert(kRecBytes % 256 == 0 && kLeadBytes % 256 == 0, "");

template <int D>
int launch_decode_i4(const DecodeI4Args &a, cudaStream_t st) {
    constexpr size_t smem = sizeof(Smem<D>);
    static std::mutex mu;
    static bool attr_set[64] = {false};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return PA_ERR_CUDA;
    {
        std::lock_guard<std::mutex> lock(mu);
        if (!attr_set[dev]) {
            if (cudaFuncSetAttribute(decode_i4_kernel<D>,
                                     cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     (int)smem) != cudaSuccess) {
                cudaGetLastError();
                return PA_ERR_CUDA;
            }
            attr_set[dev] = true;
        }
    }
    // One CTA per SM, fewer when the tables' width bounds the work below that.
    const int64_t most = (int64_t)a.B * a.Hk * ((int64_t)a.maxb + kPairCost);
    const int64_t ctas = (most + kMinUnits * kWarps - 1) / (kMinUnits * kWarps);
    int grid = sm_count();
    if (grid > kMaxGrid) grid = kMaxGrid;
    if (grid > ctas) grid = (int)ctas;
    if (grid < 1) return PA_ERR_CUDA;
    launch_dependent(decode_i4_kernel<D>, dim3(grid), dim3(kThreads), smem, st, a);
    return launch_status();
}

}  // namespace
}  // namespace pa

using namespace pa;

extern "C" size_t pa_decode_i4_workspace_bytes(int num_seqs, int n_heads, int n_kv_heads,
                                               int head_dim) {
    if (num_seqs <= 0 || n_heads <= 0 || n_kv_heads <= 0 || head_dim <= 0) return 0;
    return kRecBytes + kLeadBytes + (size_t)num_seqs * n_heads * sizeof(int32_t);
}

extern "C" int pa_decode_i4(const void *q, const pa_cache_i4_t *cache, int layer,
                            const int32_t *block_tables, int max_blocks_per_seq,
                            const int32_t *context_lens, int num_seqs, int n_heads,
                            int n_kv_heads, int head_dim, float scale, void *workspace,
                            size_t workspace_bytes, void *out, int32_t *dev_status,
                            pa_stream_t stream) {
    if (num_seqs < 0 || n_heads <= 0 || n_kv_heads <= 0 || n_heads % n_kv_heads != 0 ||
        max_blocks_per_seq <= 0 || max_blocks_per_seq > kMaxBlocksPerSeq || !(scale >= 0.f))
        return PA_ERR_INVALID;
    if (head_dim != 64 && head_dim != 128) return PA_ERR_UNSUPPORTED;
    if (n_heads / n_kv_heads > kGroupPad || num_seqs > kMaxSeqs) return PA_ERR_UNSUPPORTED;
    if ((int64_t)n_kv_heads * head_dim * 20 > INT32_MAX) return PA_ERR_UNSUPPORTED;  // a block's bytes
    if (!cache_i4_ok(cache, layer, n_kv_heads, head_dim)) return PA_ERR_INVALID;
    if (num_seqs == 0) return PA_OK;
    if (!q || !block_tables || !context_lens || !out || !workspace) return PA_ERR_INVALID;
    if (!aligned16(q) || !aligned16(out) || (reinterpret_cast<uintptr_t>(workspace) & 255u))
        return PA_ERR_INVALID;
    if (workspace_bytes < pa_decode_i4_workspace_bytes(num_seqs, n_heads, n_kv_heads, head_dim))
        return PA_ERR_WORKSPACE;
    if (scale == 0.f) scale = 1.0f / sqrtf((float)head_dim);
    DecodeI4Args a;
    a.q = static_cast<const __half *>(q);
    a.tiles = cache_i4_layer(cache, layer);
    a.block_tables = block_tables;
    a.context_lens = context_lens;
    a.out = static_cast<__half *>(out);
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    a.rec = reinterpret_cast<float *>(ws);
    a.lead = reinterpret_cast<float *>(ws + kRecBytes);
    a.counters = reinterpret_cast<int32_t *>(ws + kRecBytes + kLeadBytes);
    a.status = dev_status;
    a.scale_log2 = scale * 1.4426950408889634f;
    a.B = num_seqs;
    a.H = n_heads;
    a.Hk = n_kv_heads;
    a.g = n_heads / n_kv_heads;
    a.maxb = max_blocks_per_seq;
    a.num_blocks = cache->num_blocks;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    return head_dim == 128 ? launch_decode_i4<128>(a, st) : launch_decode_i4<64>(a, st);
}
