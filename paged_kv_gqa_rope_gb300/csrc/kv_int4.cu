// The 4-bit KV pool ("Meta Llama source deep-dive", 8.4: a quantised KV
// cache; the scheme is this library's, see include/pa.h): allocation, the
// RoPE + append kernel that quantises each appended K/V row, and the kernel
// that reads rows back as fp16.
#include <string.h>

#include <algorithm>

#include "common.cuh"
#include "internal.h"
#include "kv_int4.cuh"

namespace pa {
namespace {

struct RopeI4Args {
    const __half *q;
    __half *q_out;
    const __half *k;
    const __half *v;
    const int32_t *positions;
    const int32_t *slots;
    const float2 *table;  // [max_pos][d/2] {cos, sin}
    uint8_t *tiles;       // tile pairs of the layer
    int64_t num_slots;
    int32_t *status;
    int num_tokens, n_heads, n_kv_heads, max_pos, rounds_per_cta;
};

// One group's 8 values held by this lane, its other 24 by the lanes of the
// same aligned quad: the group's step and least value and this lane's codes,
// value i in nibble i.  Every lane of the warp takes part.
__device__ __forceinline__ uint32_t quantise8(const uint4 x, __half &step, __half &least) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    // (min, -max) as a pair, reduced together; a NaN stays one
    const __half2 mn = __hmin2_nan(__hmin2_nan(as_half2(w[0]), as_half2(w[1])),
                                   __hmin2_nan(as_half2(w[2]), as_half2(w[3])));
    const __half2 mx = __hneg2(__hmax2_nan(__hmax2_nan(as_half2(w[0]), as_half2(w[1])),
                                           __hmax2_nan(as_half2(w[2]), as_half2(w[3]))));
    __half2 r = __hmin2_nan(__lows2half2(mn, mx), __highs2half2(mn, mx));
#pragma unroll
    for (int o = 1; o < 4; o <<= 1)
        r = __hmin2_nan(r, as_half2(__shfl_xor_sync(0xffffffffu, as_u32(r), o)));
    const float lo = __low2float(r) + 0.f;  // (-0 becomes +0)
    const float range = __fsub_rn(-__high2float(r), lo);
    // The range's fifteenth rounded up to fp16: the nearest fp16 of a product
    // that is within 2^-22 of it, or the next one if 15 times that (exact) falls
    // short of the range.
    __half s16 = __float2half_rn(range * (1.f / 15.f));
    if (15.f * __half2float(s16) < range) s16 = __ushort_as_half(__half_as_ushort(s16) + 1);
    step = s16;
    least = __float2half_rn(lo);
    if (!(range <= 131008.f)) {  // a NaN or an infinity among them
        step = __ushort_as_half(0);
        least = __ushort_as_half(0x7fff);
    }
    const float s = __half2float(step);
    if (!(s > 0.f)) return 0u;
    // rint((v - lo) / s): the quotient by an approximate reciprocal, which is
    // within 2^-16 of the divided one, unless that leaves the rounding open
    // (then by division).  Adding 1.5 2^23 rounds to an integer, ties to even;
    // the quotient is at most 15 (1 + 2^-21), since 15 s is not below the range.
    constexpr float kRint = 12582912.f;
    float inv;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(s));
    const uint64_t lo2 = f2_pack(-lo, -lo), inv2 = f2_pack(inv, inv);
    const uint64_t rint2 = f2_pack(kRint, kRint), back2 = f2_pack(-kRint, -kRint);
    float c[8], off = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 v = __half22float2(as_half2(w[i]));
        const uint64_t q = f2_mul(f2_add(f2_pack(v.x, v.y), lo2), inv2);
        const uint64_t n = f2_add(f2_add(q, rint2), back2);
        f2_unpack(n, c[2 * i], c[2 * i + 1]);
        float q0, q1;
        f2_unpack(q, q0, q1);
        off = fmaxf(off, fmaxf(fabsf(q0 - c[2 * i]), fabsf(q1 - c[2 * i + 1])));
    }
    if (off > 0.4999f) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const __half2 h = as_half2(w[i >> 1]);
            c[i] = rintf(__fdiv_rn(
                __fsub_rn((i & 1) ? __high2float(h) : __low2float(h), lo), s));
        }
    }
    // four codes as one integer below 2^16 (exact), twice
    const float a = fmaf(fmaf(fmaf(c[3], 16.f, c[2]), 16.f, c[1]), 16.f, c[0]);
    const float b = fmaf(fmaf(fmaf(c[7], 16.f, c[6]), 16.f, c[5]), 16.f, c[4]);
    return __byte_perm(__float_as_uint(a + 8388608.f), __float_as_uint(b + 8388608.f), 0x5410);
}

// A CTA takes tokens blockIdx.x, + gridDim.x, ..., of each the rounds of rows of
// its blockIdx.y: first the Q rows, kAhead rounds of loads together (and the
// first round of K and V rows with them), then the K and V rows.  A thread
// keeps to one 16-byte piece (8 values) of the rows, so that it needs one set
// of cosines and sines a token.  The four threads of a group of 32 (an aligned
// quad of lanes) find its least and greatest value with shuffles.  Bound by
// HBM (Q, K and V in, Q and the codes out) with the K and V rows' arithmetic and
// narrow stores close behind: 8116 tokens of 64 + 16 heads, 310 MB, take 53.5 us
// (5.8 TB/s; 63.7 with Q, K and V rows in one loop and a division a code).  Two
// tokens a CTA, so that V's codes leave in whole words, and loads a token ahead
// took as long.
constexpr int kAhead = 4;
constexpr int kWriteCtas = 4;  // per SM

template <int D>
__global__ void __launch_bounds__(kTokenThreads, kWriteCtas)
    rope_kv_write_i4_kernel(const RopeI4Args a) {
    // Launched as a dependent; what follows may be launched once all work before
    // this kernel is done (so pa_decode's set-up, which reads the context lengths
    // ahead of its own wait, never runs beside the work that writes them).
    griddep_wait();
    griddep_launch_dependents();
    using T = I4Tile<D>;
    constexpr int kPieces = D / 8, kRows = kTokenThreads / kPieces;  // rows of a round
    const int H = a.n_heads, Hk = a.n_kv_heads;
    const int piece = threadIdx.x % kPieces, sub = threadIdx.x / kPieces;
    const int g = piece >> 2, t8 = piece & 3;
    // this CTA's rounds: Q rows q0, + kRows, ... < q1; K and V rows (K first) k0 ... < k1
    const int q_rounds = (H + kRows - 1) / kRows;
    const int r0 = (int)blockIdx.y * a.rounds_per_cta, r1 = r0 + a.rounds_per_cta;
    const int q0 = r0 * kRows + sub, q1 = min(H, r1 * kRows);
    const int k0 = max(0, r0 - q_rounds) * kRows + sub;
    const int k1 = min(2 * Hk, (r1 - q_rounds) * kRows);  // <= 0: none
    int pos = 0, slot = 0, next_pos = __ldg(a.positions + blockIdx.x),
        next_slot = __ldg(a.slots + blockIdx.x);
    for (int t = (int)blockIdx.x; t < a.num_tokens; t += (int)gridDim.x) {
        pos = next_pos;
        slot = next_slot;
        if (t + (int)gridDim.x < a.num_tokens) {
            next_pos = __ldg(a.positions + t + gridDim.x);
            next_slot = __ldg(a.slots + t + gridDim.x);
        }
        const bool pos_ok = pos >= 0 && pos < a.max_pos;
        if (threadIdx.x == 0 && blockIdx.y == 0) {
            if (!pos_ok)
                report(a.status, PA_DEV_BAD_POSITION);
            else if (slot >= a.num_slots)
                report(a.status, PA_DEV_BAD_SLOT);
        }
        if (!pos_ok) continue;
        const bool write_cache = slot >= 0 && slot < a.num_slots;
        const float4 *cs =
            reinterpret_cast<const float4 *>(a.table + (int64_t)pos * (D / 2) + piece * 4);
        const float4 cs0 = __ldg(cs), cs1 = __ldg(cs + 1);
        const uint4 *k = reinterpret_cast<const uint4 *>(a.k + (int64_t)t * Hk * D) + piece;
        const uint4 *v = reinterpret_cast<const uint4 *>(a.v + (int64_t)t * Hk * D) + piece;
        auto load_kv = [&](int row) {
            return row >= k1   ? make_uint4(0, 0, 0, 0)
                   : row < Hk ? __ldg(k + row * kPieces)
                              : __ldg(v + (row - Hk) * kPieces);
        };
        uint4 y = load_kv(k0);
        if (q0 - sub < q1) {
            const uint4 *q = reinterpret_cast<const uint4 *>(a.q + (int64_t)t * H * D) + piece;
            uint4 *q_out = reinterpret_cast<uint4 *>(a.q_out + (int64_t)t * H * D) + piece;
            for (int base = q0; base - sub < q1; base += kRows * kAhead) {
                uint4 x[kAhead];
#pragma unroll
                for (int u = 0; u < kAhead; ++u)  // (ordinary loads: q_out may be q)
                    if (base + u * kRows < q1) x[u] = q[(base + u * kRows) * kPieces];
#pragma unroll
                for (int u = 0; u < kAhead; ++u)
                    if (base + u * kRows < q1)
                        q_out[(base + u * kRows) * kPieces] = rope_rotate8(x[u], cs0, cs1);
            }
        }
        if (!write_cache) continue;
        uint8_t *tiles = a.tiles + (int64_t)(slot / kBlockSize) * Hk * T::kPair;
        const int j = slot % kBlockSize;
        for (int row = k0; row - sub < k1; row += kRows) {
            const uint4 next = load_kv(row + kRows);
            const bool is_k = row < Hk;
            if (is_k) y = rope_rotate8(y, cs0, cs1);
            __half step, least;
            const uint32_t codes = quantise8(y, step, least);  // every lane: rows past k1 are 0
            if (row < k1) {
                uint8_t *tile = tiles + (int64_t)(is_k ? row : row - Hk) * T::kPair;
                if (is_k) {
                    *reinterpret_cast<uint32_t *>(tile + T::k_word(j, g, t8)) = codes;
                } else {
                    tile += T::kBytes;
                    *reinterpret_cast<uint16_t *>(tile + T::v_half(j, g, 2 * t8)) = (uint16_t)codes;
                    *reinterpret_cast<uint16_t *>(tile + T::v_half(j, g, 2 * t8 + 1)) =
                        (uint16_t)(codes >> 16);
                }
                if (t8 == 0)
                    *reinterpret_cast<__half *>(tile + T::step(j, g)) = step;
                else if (t8 == 1)
                    *reinterpret_cast<__half *>(
                        tile + (is_k ? T::least_k(j, g) : T::least_v(j, g))) = least;
            }
            y = next;
        }
    }
}

// ---------------------------------------------------------------- read back

// A warp takes one block of one KV head (a K and a V tile) at a time, its lanes
// the words of codes in the order they are stored, so that every load is a
// whole line; the 8 values of a word leave as one 16-byte store, four lanes
// side by side for 64 bytes of a row.  Bound by HBM: 1.25 d bytes read and 4 d
// written per (token, KV head).
constexpr int kReadThreads = 256;
constexpr int kReadCtas = 8;  // per SM; four fit at a time (4 of them: 66.6 us on 32 histories of
                              // 1000 to 5000 tokens and 8 heads, 8: 64.3)
constexpr int kMaxReadSeqs = 4096;
constexpr int kMaxPrefillSeqs = 2048;  // pa_prefill_varlen's limit

struct ReadI4Args {
    const uint8_t *tiles;  // tile pairs of the layer
    const int32_t *block_tables;
    const int32_t *lengths;  // rows mode: [B]; scratch mode: cu_seqlens_k [B + 1]
    const int32_t *first;    // rows mode: [B] or null
    const int32_t *rows;     // rows mode: [B]
    const int32_t *cu_q;     // scratch mode: cu_seqlens_q [B + 1]
    __half *k_out;
    __half *v_out;
    int32_t *scratch_table;  // scratch mode: [B][maxb]
    int64_t total_rows;
    int32_t *status;
    int B, Hk, maxb, num_blocks, total_q;
};

// 8 codes (nibble i = value i) with their step and least value (each twice) ->
// 8 fp16, m + s c rounded once.  The codes are the low mantissa bits of 1024
// (of every other one 16 times as large); the fused multiply-add rounds once.
__device__ __forceinline__ uint4 dequantise8(uint32_t codes, uint32_t s, uint32_t m) {
    const __half2 top = __float2half2_rn(65504.f);
    auto value = [&](uint32_t w, bool high) {
        const uint32_t x = (w & (high ? 0x00f000f0u : 0x000f000fu)) | 0x64006400u;
        const __half2 c = high ? __hfma2(as_half2(x), __float2half2_rn(0.0625f),
                                         __float2half2_rn(-64.f))
                               : __hadd2(as_half2(x), __float2half2_rn(-1024.f));
        return as_u32(__hmin2_nan(__hfma2(as_half2(s), c, as_half2(m)), top));
    };
    const uint32_t a = value(codes, false), b = value(codes, true);  // 0, 4 | 1, 5
    const uint32_t c = value(codes >> 8, false), d = value(codes >> 8, true);  // 2, 6 | 3, 7
    return make_uint4(__byte_perm(a, b, 0x5410), __byte_perm(c, d, 0x5410),
                      __byte_perm(a, b, 0x7632), __byte_perm(c, d, 0x7632));
}

// G words of 32 bits, 4 G-byte aligned, read once.
template <int G>
__device__ __forceinline__ void read_words(uint32_t (&w)[G], const uint8_t *p) {
    if constexpr (G == 4) {
        const uint4 x = __ldcs(reinterpret_cast<const uint4 *>(p));
        w[0] = x.x, w[1] = x.y, w[2] = x.z, w[3] = x.w;
    } else {
        const uint2 x = __ldcs(reinterpret_cast<const uint2 *>(p));
        w[0] = x.x, w[1] = x.y;
    }
}

// 8 values of an output row; kKeep: the next kernel reads them, so they stay in L2.
template <bool kKeep>
__device__ __forceinline__ void store_row(__half *p, const uint4 &x) {
    if constexpr (kKeep)
        *reinterpret_cast<uint4 *>(p) = x;
    else
        __stcs(reinterpret_cast<uint4 *>(p), x);
}

// One K tile: rows j0 .. j1 - 1 to `out` (row 0 of the block), rows `stride` halves apart.
template <int D, bool kKeep>
__device__ __forceinline__ void read_k(const uint8_t *tile, __half *out, int64_t stride, int j0,
                                       int j1, int lane) {
    using T = I4Tile<D>;
    constexpr int G = T::kGroups;
    const int r = lane >> 2, t = lane & 3;
    uint32_t w[2][G], st[2][G], ls[2][G / 2];  // rows r and r + 8
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        read_words<G>(w[h], tile + T::k_word(r + 8 * h, 0, t));
        // steps of rows 2 (r / 2) + (0, 1, 8, 9), group after group
        read_words<G>(st[h], tile + T::step(r & 6, 0) + 4 * G * h);
        if constexpr (G == 4) {
            const uint2 x = *reinterpret_cast<const uint2 *>(tile + T::least_k(r + 8 * h, 0));
            ls[h][0] = x.x, ls[h][1] = x.y;
        } else {
            ls[h][0] = *reinterpret_cast<const uint32_t *>(tile + T::least_k(r + 8 * h, 0));
        }
    }
    const uint32_t pick = (r & 1) ? 0x3232u : 0x1010u;
#pragma unroll
    for (int g = 0; g < G; ++g)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int j = r + 8 * h;
            const uint32_t s = __byte_perm(st[g / (G / 2)][2 * (g % (G / 2)) + h], 0u, pick);
            const uint32_t m = __byte_perm(ls[h][g / 2], 0u, (g & 1) ? 0x3232u : 0x1010u);
            if (j >= j0 && j < j1)
                store_row<kKeep>(out + j * stride + 32 * g + 8 * t, dequantise8(w[h][g], s, m));
        }
}

// One V tile, likewise.  Lane = (half h of the rows, t, i): rows 8 h + 2 t and + 1,
// values 32 g + 8 i .. + 7.
template <int D, bool kKeep>
__device__ __forceinline__ void read_v(const uint8_t *tile, __half *out, int64_t stride, int j0,
                                       int j1, int lane) {
    using T = I4Tile<D>;
    constexpr int G = T::kGroups;
    const int i = lane & 3, t = (lane >> 2) & 3, h = lane >> 4;
    const int j = 8 * h + 2 * t;
    uint32_t w0[G], w1[G], st[2][G], ls[2][G];
    read_words<G>(w0, tile + T::v_half(j, 0, 2 * i));
    read_words<G>(w1, tile + T::v_half(j, 0, 2 * i + 1));
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        read_words<G>(st[k], tile + T::step(2 * t, 0) + 4 * G * k);
        read_words<G>(ls[k], tile + T::least_v(2 * t, 0) + 4 * G * k);
    }
#pragma unroll
    for (int g = 0; g < G; ++g) {
        // words 2 g + h: rows j and j + 1
        const uint32_t *sp = &st[g / (G / 2)][2 * (g % (G / 2))];
        const uint32_t *mp = &ls[g / (G / 2)][2 * (g % (G / 2))];
        const uint32_t sw = h ? sp[1] : sp[0], mw = h ? mp[1] : mp[0];
#pragma unroll
        for (int k = 0; k < 2; ++k)
            if (j + k >= j0 && j + k < j1)
                store_row<kKeep>(out + (j + k) * stride + 32 * g + 8 * i,
                                 dequantise8(__byte_perm(w0[g], w1[g], k ? 0x7632 : 0x5410),
                                             __byte_perm(sw, 0u, k ? 0x3232 : 0x1010),
                                             __byte_perm(mw, 0u, k ? 0x3232 : 0x1010)));
    }
}

// kScratch false: rows of sequences to the caller's row positions.
// kScratch true: the whole context of every sequence that the prefill kernel
// attends to (the others may be long, and have tables of another call) into
// consecutive blocks of a scratch fp16 pool, with its block table.
template <int D, bool kScratch>
__global__ void __launch_bounds__(kReadThreads) kv_read_i4_kernel(const ReadI4Args a) {
    using T = I4Tile<D>;
    griddep_wait();  // as in rope_kv_write_i4_kernel
    griddep_launch_dependents();
    extern __shared__ int64_t prefix[];  // [B + 1] blocks of the sequences before
    const int tid = threadIdx.x, lane = tid & 31;
    for (int s = tid; s < a.B; s += kReadThreads) {
        int64_t n = 0;
        const int64_t len = kScratch
                                ? (int64_t)__ldg(a.lengths + s + 1) - __ldg(a.lengths + s)
                                : (int64_t)__ldg(a.lengths + s);
        const int64_t f = !kScratch && a.first ? __ldg(a.first + s) : 0;
        const int64_t r = kScratch ? 0 : __ldg(a.rows + s);
        bool ok = len >= 0 && f >= 0 && f + len <= (int64_t)a.maxb * kBlockSize && r >= 0 &&
                  (kScratch || r + len <= a.total_rows);
        if constexpr (kScratch) {
            const int64_t q0 = __ldg(a.cu_q + s), q1 = __ldg(a.cu_q + s + 1);
            ok = ok && q0 >= 0 && q0 < q1 && q1 <= a.total_q && q1 - q0 <= len;
        }
        if (len == 0) {
            // nothing to read, whatever the rest says (a padded batch)
        } else if (!ok) {
            // (the prefill kernel reports a bad length of its own)
            if (!kScratch && blockIdx.x == 0) report(a.status, PA_DEV_BAD_LENGTH);
        } else {
            n = (f % kBlockSize + len + kBlockSize - 1) / kBlockSize;
        }
        prefix[s + 1] = n;
    }
    if (tid == 0) prefix[0] = 0;
    __syncthreads();
    if (tid < 32) prefix_sums(prefix, a.B, lane);
    __syncthreads();
    const int64_t units = prefix[a.B];
    // warps take (block, head) pairs, the heads of a block side by side
    const int64_t items = units * a.Hk;
    const int64_t warps = (int64_t)gridDim.x * (kReadThreads / 32);
    const int64_t stride = (int64_t)a.Hk * D;
    for (int64_t x = (int64_t)blockIdx.x * (kReadThreads / 32) + (tid >> 5); x < items; x += warps) {
        const int64_t u = (x >> 32) == 0 ? (int64_t)((uint32_t)x / (uint32_t)a.Hk) : x / a.Hk;
        const int h = (int)(x - u * a.Hk);
        int lo = 0, hi = a.B - 1;  // largest s with prefix[s] <= u
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (prefix[mid] <= u)
                lo = mid;
            else
                hi = mid - 1;
        }
        const int s = lo;
        const int64_t f = !kScratch && a.first ? __ldg(a.first + s) : 0;
        const int64_t len = kScratch
                                ? (int64_t)__ldg(a.lengths + s + 1) - __ldg(a.lengths + s)
                                : (int64_t)__ldg(a.lengths + s);
        const int64_t b = f / kBlockSize + (u - prefix[s]);  // logical block
        const int blk = __ldg(a.block_tables + (int64_t)s * a.maxb + b);
        const bool blk_ok = blk >= 0 && blk < a.num_blocks;
        // output row of the block's token 0 (it may lie before the first row)
        int64_t row0;
        if constexpr (kScratch) {
            row0 = u * kBlockSize;
            const bool fits = row0 + kBlockSize <= a.total_rows;
            if (h == 0 && lane == 0) {
                a.scratch_table[(int64_t)s * a.maxb + b] = blk_ok && fits ? (int32_t)u : -1;
                if (!fits) report(a.status, PA_DEV_WORKSPACE);
            }
            if (!fits) continue;
        } else {
            row0 = (int64_t)__ldg(a.rows + s) + b * kBlockSize - f;
        }
        if (!blk_ok) {
            if (h == 0 && lane == 0) report(a.status, PA_DEV_BAD_BLOCK);
            continue;
        }
        const int j0 = (int)max((int64_t)0, f - b * kBlockSize);
        const int j1 = (int)min((int64_t)kBlockSize, f + len - b * kBlockSize);
        const uint8_t *tile = a.tiles + ((int64_t)blk * a.Hk + h) * T::kPair;
        const int64_t at = row0 * stride + (int64_t)h * D;
        if (a.k_out) read_k<D, kScratch>(tile, a.k_out + at, stride, j0, j1, lane);
        if (a.v_out) read_v<D, kScratch>(tile + T::kBytes, a.v_out + at, stride, j0, j1, lane);
    }
}

template <int D, bool kScratch>
int launch_read(const ReadI4Args &a, cudaStream_t st) {
    const int sms = sm_count();
    if (sms < 1) return PA_ERR_CUDA;
    const size_t smem = (size_t)(a.B + 1) * sizeof(int64_t);
    launch_dependent(kv_read_i4_kernel<D, kScratch>, dim3(sms * kReadCtas), dim3(kReadThreads), smem,
                     st, a);
    return launch_status();
}

}  // namespace
}  // namespace pa

using namespace pa;

extern "C" size_t pa_cache_i4_bytes(int layers, int num_blocks, int block_size, int n_kv_heads,
                                    int head_dim) {
    if (layers <= 0 || num_blocks <= 0 || block_size <= 0 || n_kv_heads <= 0 || head_dim <= 0)
        return 0;
    // 5 bits a value, K and V; 0 if that passes a size_t
    size_t values = (size_t)layers * num_blocks;
    if (__builtin_mul_overflow(values, (size_t)block_size * n_kv_heads, &values) ||
        __builtin_mul_overflow(values, (size_t)head_dim, &values) || values > SIZE_MAX / 5 * 4)
        return 0;
    return values / 4 * 5;
}

extern "C" int pa_alloc_cache_i4(pa_cache_i4_t *out, int layers, int num_blocks, int block_size,
                                 int n_kv_heads, int head_dim, void *device_base) {
    if (!out) return PA_ERR_INVALID;
    memset(out, 0, sizeof(*out));
    const size_t bytes = pa_cache_i4_bytes(layers, num_blocks, block_size, n_kv_heads, head_dim);
    if (bytes == 0) return PA_ERR_INVALID;
    if ((int64_t)num_blocks * block_size > INT32_MAX) return PA_ERR_INVALID;
    if (block_size != kBlockSize || (head_dim != 64 && head_dim != 128)) return PA_ERR_UNSUPPORTED;
    if ((int64_t)n_kv_heads * head_dim * 20 > INT32_MAX) return PA_ERR_UNSUPPORTED;
    if (device_base && (reinterpret_cast<uintptr_t>(device_base) & 255u)) return PA_ERR_INVALID;
    void *base = device_base;
    if (!base) {
        if (cudaMalloc(&base, bytes) != cudaSuccess) {
            cudaGetLastError();
            return PA_ERR_CUDA;
        }
        out->owns = 1;
    }
    out->base = static_cast<uint8_t *>(base);
    out->layers = layers;
    out->num_blocks = num_blocks;
    out->block_size = block_size;
    out->n_kv_heads = n_kv_heads;
    out->head_dim = head_dim;
    return PA_OK;
}

extern "C" int pa_free_cache_i4(pa_cache_i4_t *cache) {
    if (!cache) return PA_ERR_INVALID;
    int rc = PA_OK;
    if (cache->owns && cache->base && cudaFree(cache->base) != cudaSuccess) rc = PA_ERR_CUDA;
    memset(cache, 0, sizeof(*cache));
    return rc;
}

extern "C" int pa_rope_kv_write_i4(const void *q, void *q_out, const void *k, const void *v,
                                   const int32_t *positions, const int32_t *slot_mapping,
                                   int num_tokens, int n_heads, int n_kv_heads, int head_dim,
                                   const void *rope_table, int max_positions,
                                   const pa_cache_i4_t *cache, int layer, int32_t *dev_status,
                                   pa_stream_t stream) {
    if (num_tokens < 0 || n_heads <= 0 || n_kv_heads <= 0 || n_heads % n_kv_heads != 0 ||
        max_positions <= 0)
        return PA_ERR_INVALID;
    if (head_dim != 64 && head_dim != 128) return PA_ERR_UNSUPPORTED;
    if (!cache_i4_ok(cache, layer, n_kv_heads, head_dim)) return PA_ERR_INVALID;
    if (num_tokens == 0) return PA_OK;
    if (!q || !q_out || !k || !v || !positions || !slot_mapping || !rope_table)
        return PA_ERR_INVALID;
    if (!aligned16(q) || !aligned16(q_out) || !aligned16(k) || !aligned16(v) ||
        !aligned16(rope_table))
        return PA_ERR_INVALID;
    if (num_tokens > ((int64_t)1 << 40) / (((int64_t)n_heads + 2 * (int64_t)n_kv_heads) *
                                           (head_dim / 8)))
        return PA_ERR_INVALID;
    if ((int64_t)n_heads * head_dim * 2 > INT32_MAX) return PA_ERR_UNSUPPORTED;  // a token's Q
    // q_out is q or lies apart from every input
    const int64_t qb = (int64_t)num_tokens * n_heads * head_dim * 2;
    const int64_t kb = (int64_t)num_tokens * n_kv_heads * head_dim * 2;
    const uintptr_t o = reinterpret_cast<uintptr_t>(q_out);
    auto apart = [&](const void *p, int64_t n) {
        const uintptr_t x = reinterpret_cast<uintptr_t>(p);
        return x + (uintptr_t)n <= o || o + (uintptr_t)qb <= x;
    };
    if ((q_out != q && !apart(q, qb)) || !apart(k, kb) || !apart(v, kb)) return PA_ERR_INVALID;

    RopeI4Args a;
    a.q = static_cast<const __half *>(q);
    a.q_out = static_cast<__half *>(q_out);
    a.k = static_cast<const __half *>(k);
    a.v = static_cast<const __half *>(v);
    a.positions = positions;
    a.slots = slot_mapping;
    a.table = static_cast<const float2 *>(rope_table);
    a.tiles = cache_i4_layer(cache, layer);
    a.num_slots = (int64_t)cache->num_blocks * kBlockSize;
    a.status = dev_status;
    a.num_tokens = num_tokens;
    a.n_heads = n_heads;
    a.n_kv_heads = n_kv_heads;
    a.max_pos = max_positions;
    // Four CTAs per SM.  A token's rows are spread over several CTAs, down to one
    // round of rows each, while that leaves two per SM: 1 token of 64 + 16 heads
    // takes 1.75 us spread and 2.27 not, 16 tokens 2.16 and 2.58, but 256 tokens
    // 3.39 (in two) and 3.14.
    const int sms = sm_count();
    if (sms < 1) return PA_ERR_CUDA;
    const int round = kTokenThreads / (head_dim / 8);
    const int rounds = (n_heads + round - 1) / round + (2 * n_kv_heads + round - 1) / round;
    const int split = std::max(1, std::min(rounds, sms * 2 / num_tokens));
    a.rounds_per_cta = (rounds + split - 1) / split;
    const dim3 grid(std::min(num_tokens, sms * kWriteCtas),
                    (rounds + a.rounds_per_cta - 1) / a.rounds_per_cta);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (head_dim == 128)
        launch_dependent(rope_kv_write_i4_kernel<128>, grid, dim3(kTokenThreads), 0, st, a);
    else
        launch_dependent(rope_kv_write_i4_kernel<64>, grid, dim3(kTokenThreads), 0, st, a);
    return launch_status();
}

extern "C" int pa_kv_read_i4(const pa_cache_i4_t *cache, int layer, const int32_t *block_tables,
                             int max_blocks_per_seq, const int32_t *lengths,
                             const int32_t *first_tokens, const int32_t *row_starts, int num_seqs,
                             int total_rows, int n_kv_heads, int head_dim, void *k_out,
                             void *v_out, int32_t *dev_status, pa_stream_t stream) {
    if (num_seqs < 0 || total_rows < 0 || n_kv_heads <= 0 || max_blocks_per_seq <= 0 ||
        max_blocks_per_seq > kMaxBlocksPerSeq)
        return PA_ERR_INVALID;
    if (head_dim != 64 && head_dim != 128) return PA_ERR_UNSUPPORTED;
    if (num_seqs > kMaxReadSeqs) return PA_ERR_UNSUPPORTED;
    if (!cache_i4_ok(cache, layer, n_kv_heads, head_dim)) return PA_ERR_INVALID;
    if (num_seqs == 0) return PA_OK;
    if (!block_tables || !lengths || !row_starts) return PA_ERR_INVALID;
    if (!aligned16(k_out) || !aligned16(v_out)) return PA_ERR_INVALID;
    if (!k_out && !v_out) return PA_OK;

    ReadI4Args a = {};
    a.tiles = cache_i4_layer(cache, layer);
    a.block_tables = block_tables;
    a.lengths = lengths;
    a.first = first_tokens;
    a.rows = row_starts;
    a.k_out = static_cast<__half *>(k_out);
    a.v_out = static_cast<__half *>(v_out);
    a.total_rows = total_rows;
    a.status = dev_status;
    a.B = num_seqs;
    a.Hk = n_kv_heads;
    a.maxb = max_blocks_per_seq;
    a.num_blocks = cache->num_blocks;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    return head_dim == 128 ? launch_read<128, false>(a, st) : launch_read<64, false>(a, st);
}

// ---------------------------------------------------------------- prefill

namespace pa {
namespace {

size_t scratch_table_bytes(int num_seqs, int maxb) {
    return ((size_t)num_seqs * maxb * sizeof(int32_t) + 255) & ~(size_t)255;
}
size_t scratch_block_bytes(int Hk, int d) { return (size_t)kBlockSize * Hk * d * 2 * 2; }

}  // namespace
}  // namespace pa

extern "C" size_t pa_prefill_i4_workspace_bytes(int scratch_blocks, int num_seqs,
                                                int max_blocks_per_seq, int n_kv_heads,
                                                int head_dim) {
    if (scratch_blocks <= 0 || num_seqs <= 0 || max_blocks_per_seq <= 0 || n_kv_heads <= 0 ||
        head_dim <= 0)
        return 0;
    // (the table's bytes and one row of a block fit a size_t; 0 if the sum does not)
    size_t bytes;
    if (__builtin_mul_overflow((size_t)n_kv_heads * head_dim, (size_t)kBlockSize * 4, &bytes) ||
        __builtin_mul_overflow(bytes, (size_t)scratch_blocks, &bytes) ||
        __builtin_add_overflow(bytes, scratch_table_bytes(num_seqs, max_blocks_per_seq), &bytes))
        return 0;
    return bytes;
}

extern "C" int pa_prefill_varlen_i4(const void *q, int total_q, const pa_cache_i4_t *cache,
                                    int layer, const int32_t *cu_seqlens_q,
                                    const int32_t *cu_seqlens_k, const int32_t *block_tables,
                                    int max_blocks_per_seq, int num_seqs, int max_seqlen_q,
                                    int n_heads, int n_kv_heads, int head_dim, float scale,
                                    void *workspace, size_t workspace_bytes, void *out,
                                    int32_t *dev_status, pa_stream_t stream) {
    if (n_heads <= 0 || n_kv_heads <= 0 || n_heads % n_kv_heads != 0 || num_seqs < 0 ||
        total_q < 0 || max_seqlen_q < 0 || max_blocks_per_seq <= 0 ||
        max_blocks_per_seq > kMaxBlocksPerSeq || !(scale >= 0.f))
        return PA_ERR_INVALID;
    if (head_dim != 64 && head_dim != 128) return PA_ERR_UNSUPPORTED;
    if (num_seqs > kMaxPrefillSeqs) return PA_ERR_UNSUPPORTED;
    if (!cache_i4_ok(cache, layer, n_kv_heads, head_dim)) return PA_ERR_INVALID;
    if (num_seqs == 0 || max_seqlen_q == 0 || total_q == 0) return PA_OK;
    if (!q || !out || !cu_seqlens_q || !cu_seqlens_k || !block_tables || !workspace)
        return PA_ERR_INVALID;
    if (!aligned16(q) || !aligned16(out) || (reinterpret_cast<uintptr_t>(workspace) & 255u))
        return PA_ERR_INVALID;
    const size_t tab = scratch_table_bytes(num_seqs, max_blocks_per_seq);
    const size_t per_block = scratch_block_bytes(n_kv_heads, head_dim);
    if (workspace_bytes < tab + per_block) return PA_ERR_WORKSPACE;
    size_t blocks = (workspace_bytes - tab) / per_block;
    if (blocks > (size_t)(INT32_MAX / kBlockSize)) blocks = INT32_MAX / kBlockSize;

    uint8_t *ws = static_cast<uint8_t *>(workspace);
    pa_cache_t pool;
    int rc = pa_alloc_cache(&pool, 1, (int)blocks, kBlockSize, n_kv_heads, head_dim, ws + tab);
    if (rc != PA_OK) return rc;
    ReadI4Args a = {};
    a.tiles = cache_i4_layer(cache, layer);
    a.block_tables = block_tables;
    a.lengths = cu_seqlens_k;
    a.cu_q = cu_seqlens_q;
    a.total_q = total_q;
    a.k_out = cache_plane(&pool, 0, 0);
    a.v_out = cache_plane(&pool, 1, 0);
    a.scratch_table = reinterpret_cast<int32_t *>(ws);
    a.total_rows = (int64_t)blocks * kBlockSize;
    a.status = dev_status;
    a.B = num_seqs;
    a.Hk = n_kv_heads;
    a.maxb = max_blocks_per_seq;
    a.num_blocks = cache->num_blocks;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    rc = head_dim == 128 ? launch_read<128, true>(a, st) : launch_read<64, true>(a, st);
    if (rc != PA_OK) return rc;
    return pa_prefill_varlen(q, total_q, &pool, 0, cu_seqlens_q, cu_seqlens_k,
                             a.scratch_table, max_blocks_per_seq, num_seqs, max_seqlen_q, n_heads,
                             n_kv_heads, head_dim, scale, out, dev_status, stream);
}
