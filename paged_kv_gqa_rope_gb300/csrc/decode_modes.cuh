// What pa_decode_weights and pa_decode_shared have in common with decode.cu:
// the decode kernel's other results, and the groups of sequences that share a
// prefix as every kernel of a call reads them.
#pragma once

#include "common.cuh"
#include "internal.h"

namespace pa {

// Sequences starts[r] .. starts[r + 1] - 1 name the same first blocks[r] blocks.
struct Groups {
    const int32_t *starts;
    const int32_t *blocks;
    int n, maxb, seqs;
};

// A group whose prefix is read once.  The prefixes' work lies on a line: group
// after group, KV head after KV head, unit after unit (2 * (128 / g) sequences:
// two tiles of 128 query rows), 128-key tile after tile and kUnitCost places for a
// unit's fixed cost (its Q, the ring's start, its record: about 3.5 us, without which
// CTAs with several short units end last).  A tile has `weight` places: two
// (1.15 us) against one tile of query rows, three (1.7 us) against two.  G CTAs take
// equal ranges of the line; a tile belongs to the range of its first place.
struct PlanGroup {
    int tiles;    // key tiles of a unit
    int blocks;   // blocks shared
    int s0;       // first sequence
    int members;
    int lead;     // sequence whose block table is read
    int units;    // units of a KV head
    int weight;
    __device__ __forceinline__ int span() const;  // places of a unit
};
// Where a CTA's range begins: at place t0 of unit `unit` (all KV heads counted) of
// group `group`, and how many places it has.
struct PlanCut {
    PlanGroup p;
    int group, unit, t0;
    int64_t places;
};
// What the other two kernels need of a sequence, and of the call.
struct alignas(16) SeqPlan {
    int tail;        // tokens behind the shared blocks, 0 for a sequence left out
    int skip;        // shared blocks
    int state;
    int local;       // row of its first Q head (of a KV head) in its unit
    int64_t start;   // line: first place of the unit, of KV head 0
    int64_t stride;  // places from a KV head's unit to the next head's
    int last;        // first place of the unit's last tile, from the unit's first
    int pad[3];
};
enum : int { kInGroup = 0, kAlone = -1, kLeftOut = -2 };  // SeqPlan::state
struct alignas(16) PlanHead {
    int64_t total;  // places of the line
    int ctas;       // CTAs with a range of it
    int tail_ctas;  // CTAs of the tails' kernel
};

// Records of rows, with four columns of all of them side by side ([D / 4][rows][4],
// then {m, l}[rows]): neither the threads that write them, one a row, nor those that
// read them leave a line half used.
struct Record {
    float *base;
    int64_t rows, row;
    __device__ __forceinline__ float4 *cols(int i) const {  // columns 4 i .. 4 i + 3
        return reinterpret_cast<float4 *>(base) + i * rows + row;
    }
    __device__ __forceinline__ float2 *stat(int d) const {
        return reinterpret_cast<float2 *>(base + d * rows) + row;
    }
};

// What the decode kernel's other modes leave for the kernel after it: a row's
// unnormalised O, m and l.  A pair (sequence, KV head) that the CTAs' ranges cut stays in
// its pieces: the first in its place in rec, the others in their CTAs' records.  (Merged
// by the last piece to arrive, a piece took 3.7 us against a whole pair's 1.5, and the
// last CTAs of a launch were done 4 us later; four sequences of 16384 tokens and one KV
// head, 76 pieces each, took 57 us and take 24.)
struct Pieces {
    float *rec;    // rows (KV head, sequence, Q head of the KV head), as Record has them
    int32_t *cut;  // [B][Hk]: CTA of the second piece | pieces but the first << 16
};

// A sequence in pa_decode_weights: its first block in the scores (-1: none kept, -2: left
// out), and its tokens, as the decode kernel has checked and counted them.
struct alignas(16) SeqScores {
    int64_t first;
    int32_t len, pad;
};

// pa_decode_weights: scores and row statistics besides the output.  Of a pair left in
// pieces (of no other) there are no statistics and no output.
struct DecodeScores {
    Pieces pieces;
    float *scores;     // [blocks of all KV heads][16 tokens][g]: log2 units
    float2 *stats;     // [B][H]: {m, 1 / l}, a weight being 2^(score - m) / l
    SeqScores *seqs;   // [B]
    int64_t capacity;  // blocks of all KV heads that scores holds
    int max_len;       // longest context that the rows of weights hold
};

// Units of a pair's fixed cost on the tails' line (a block: 1).  With 64/8, 32/32 and
// 32/8 heads 8 took 26.2, 33.7 and 44.4 us, 6 27.4, 33.7 and 44.1.
constexpr int kTailCost = 8;
// pa_decode_shared: records in the place of the output, over the tokens behind the
// shared blocks.  A sequence with no shared blocks gets its output, but for the pairs
// left in pieces.
struct DecodeTails {
    Pieces pieces;
    // by the prefix kernel, ahead of its launch_dependents
    const PlanHead *head;
    const SeqPlan *seqs;  // [B]
};

constexpr int kPrefixTile = 128;  // keys of a tile, and query rows
constexpr int kTileBlocks = kPrefixTile / kBlockSize;

constexpr int kUnitCost = 6, kTileWeight = 2, kPairWeight = 3;
__device__ __forceinline__ int PlanGroup::span() const { return tiles * weight + kUnitCost; }

// CTAs with a range: each of kPairWeight places at least, so that it has a tile of
// every unit that goes on through it and a unit's pieces are those of neighbouring
// CTAs.
__device__ __forceinline__ int plan_ctas(int64_t total, int sms) {
    return (int)min(total / kPairWeight, (int64_t)sms);
}

// First place of CTA c's range, and the CTA whose range holds place t.  (32-bit
// divisions for all but absurd lines: G < 1024, so their operands fit.)
constexpr int kShortLine = INT32_MAX / 1024;
__device__ __forceinline__ int64_t plan_cut(int64_t total, int c, int G) {
    if (total < kShortLine) return (uint32_t)total * (uint32_t)c / (uint32_t)G;
    return total * c / G;
}
__device__ __forceinline__ int plan_cta(int64_t t, int64_t total, int G) {
    if (total < kShortLine)
        return (int)((((uint32_t)t + 1) * (uint32_t)G + (uint32_t)total - 1) / (uint32_t)total) - 1;
    return (int)(((t + 1) * G + total - 1) / total) - 1;
}

// The output's rounding.  An average of values at the end of fp16's range, its two
// sums each a fp32 chain of one step a tile or block, can come out past it where the
// context is long: finite ones are saturated.
__device__ __forceinline__ float saturate16(float x) {
    return fabsf(x) < INFINITY ? fminf(fmaxf(x, -65504.f), 65504.f) : x;
}

// A decode call as its entry point has checked it.
struct DecodeCall {
    const void *q;
    const pa_cache_t *cache;
    int layer;
    const int32_t *block_tables;
    int max_blocks_per_seq;
    const int32_t *context_lens;
    int num_seqs, n_heads, n_kv_heads, head_dim;
    float scale;
    void *out;
    int32_t *dev_status;
    cudaStream_t stream;
};

// pa_decode's checks of everything but the workspace (PA_OK with num_seqs 0:
// nothing to do).
int check_decode_args(const void *q, const pa_cache_t *cache, int layer,
                      const int32_t *block_tables, int max_blocks_per_seq,
                      const int32_t *context_lens, int num_seqs, int n_heads, int n_kv_heads,
                      int head_dim, float scale, const void *out);

// The decode kernel in its other modes.  The CTAs' records stand at the start of the
// workspace, which so serves calls of several shapes.
constexpr int kModeCtas = 608;          // with two records each
size_t mode_workspace_bytes(int head_dim);
constexpr int kModeRows = 8;             // of D + 4 floats each
float *mode_records(void *workspace);    // [2 * CTA + slot]
int launch_decode_scores(const DecodeCall &c, void *workspace, const DecodeScores &sc);
int launch_decode_tails(const DecodeCall &c, void *workspace, const DecodeTails &tl);

// The pieces of a pair behind its first, `more` of them, each a CTA's first record.
// (What a call that gave up has not written may be anything.)
struct Cut {
    int cta, more;
};
__device__ __forceinline__ Cut cut_of(int32_t x) {
    Cut c = {x & 0xffff, x >> 16};
    if (c.more < 0 || c.cta + c.more > kModeCtas) c.more = 0;
    return c;
}
__device__ __forceinline__ Record piece_of(float *records, int cta, int d, int head) {
    return {records + (int64_t)cta * 2 * kModeRows * (d + 4), kModeRows, head};
}

// A prefix is read once for its group if that saves at least this many blocks
// of a KV head, else by each sequence with the rest of its context (a single
// sequence has nothing to share).  Eight sequences over 128 shared tokens, 56
// blocks: 9.9 us shared and 14.5 not with 4/2 heads of 64, 13.7 and 17.1 with 32/32
// of 128; two over 256, 16 blocks, 64/8 of 128: 11.1 and 22.6.  It holds for few groups
// and large ones.  Of many small ones the fixed cost of a unit a group and KV head, which
// the rule does not weigh, is more than they save: 64 sequences with up to 512 tokens of
// their own, 32/8 heads of 128, in 32 groups over 128 tokens 30.2 us shared and 25.6 not,
// over 256 30.6 and 27.1, over 1024 46.5 and 50.7; in 16 groups over 128 26.0 and 25.1,
// over 256 27.2 and 28.5.
constexpr int kMinSavedBlocks = 8;

__device__ __forceinline__ int shared_of(int blocks, int members) {
    return (int64_t)blocks * (members - 1) >= kMinSavedBlocks ? blocks : 0;
}

// For every sequence, by all `threads` threads of the CTA: skip[s], the shared
// blocks to leave to the group (-1 for a sequence that is left out: its length
// is out of range or shorter than the blocks it shares, its group's blocks are
// out of range, or the groups do not partition the sequences), and lens[s], the
// tokens behind them.  Every CTA of a call comes to the same result.  Returns, to
// every thread, 0, 1 if anything was out of range, 2 for groups that are no
// partition.
__device__ __forceinline__ int read_groups(const Groups &g, const int32_t *context_lens, int B,
                                            int32_t *skip, int32_t *lens, int tid, int threads) {
    int bad = 0;
    for (int r = tid; r < g.n; r += threads)
        bad |= __ldg(g.starts + r) > __ldg(g.starts + r + 1);
    if (tid == 0) bad |= __ldg(g.starts) != 0 || __ldg(g.starts + g.n) != B;
    const bool broken = __syncthreads_or(bad);
    if (broken) {
        for (int s = tid; s < B; s += threads) {
            skip[s] = -1;
            lens[s] = 0;
        }
        __syncthreads();
        return 2;
    }
    // Rising from 0 to B, so every start is in range.  A warp takes 32 groups.
    const int lane = tid & 31;
    for (int r0 = (tid >> 5) * 32; r0 < g.n; r0 += threads) {
        int start = 0, end = 0, blocks = 0;
        if (r0 + lane < g.n) {
            start = __ldg(g.starts + r0 + lane);
            end = __ldg(g.starts + r0 + lane + 1);
            blocks = __ldg(g.blocks + r0 + lane);
        }
        for (int i = 0; i < min(32, g.n - r0); ++i) {
            const int s0 = __shfl_sync(0xffffffffu, start, i), s1 = __shfl_sync(0xffffffffu, end, i);
            const int named = __shfl_sync(0xffffffffu, blocks, i);
            const bool ok = named >= 0 && named <= g.maxb;
            const int kept = shared_of(named, s1 - s0);
            for (int s = s0 + lane; s < s1; s += 32) {
                const int ctx = __ldg(context_lens + s);
                const bool fine = ok && ctx >= 1 && ctx <= g.maxb * kBlockSize &&
                                  ctx >= named * kBlockSize;
                skip[s] = fine ? kept : -1;
                lens[s] = fine ? ctx - kept * kBlockSize : 0;
                bad |= !fine;
            }
        }
    }
    return __syncthreads_or(bad) != 0 ? 1 : 0;
}

// Group r's share of the line (tiles 0: none), from global memory.  (Whoever asks has
// seen that the groups are a partition; a group that by now is none of the sequences'
// has no share, so that no read leaves the arrays.)
__device__ __forceinline__ PlanGroup load_group(const Groups &g, const int32_t *context_lens, int r,
                                                int per_unit) {
    PlanGroup p;
    p.s0 = __ldg(g.starts + r);
    p.members = __ldg(g.starts + r + 1) - p.s0;
    const int named = __ldg(g.blocks + r);
    const bool in_range = named >= 0 && named <= g.maxb && p.s0 >= 0 && p.members >= 0 &&
                          p.members <= g.seqs - p.s0;
    p.blocks = in_range ? shared_of(named, p.members) : 0;
    p.lead = p.s0;
    if (p.blocks > 0) {
        // the first sequence in order (as read_groups has it)
        for (int ctx; p.lead < p.s0 + p.members; ++p.lead) {
            ctx = __ldg(context_lens + p.lead);
            if (ctx <= g.maxb * kBlockSize && ctx >= named * kBlockSize) break;
        }
        if (p.lead == p.s0 + p.members) p.blocks = 0;
    }
    p.tiles = (p.blocks + kTileBlocks - 1) / kTileBlocks;
    p.units = (p.members + per_unit - 1) / per_unit;
    p.weight = p.members > per_unit / 2 ? kPairWeight : kTileWeight;
    return p;
}

// How the SMs are divided between the prefixes and the tails, which run side by
// side: in proportion to what each would take of one SM, in units of a tail's
// block (8 KB at d = 128, about 0.14 us with two decode CTAs an SM).
constexpr int kTileCost = 8;  // of kTileWeight places

__device__ __forceinline__ int divide_sms(unsigned long long places, unsigned long long tail,
                                          int active, int64_t units, int sms) {
    if (places == 0) return 0;
    int n = sms, most = sms;
    if (tail > 0) {
        most = sms - 1;
        const float cost = (float)places * ((float)kTileCost / kTileWeight);
        n = max(1, min(most, (int)((float)sms * cost / (cost + (float)tail) + 0.5f)));
    }
    // Of one group every unit is alike: a multiple of them cuts none but at its ends.
    if (active == 1 && units <= most) {
        const int u = (int)units, even = max(1, (n + u / 2) / u) * u;
        n = even <= most ? even : even - u;
    }
    return n;
}

// By a whole CTA of `threads` threads after read_groups; `sums` are three words of
// shared memory.  Every CTA comes to the same.  Returns the SMs for the prefixes;
// total: places of their line.
__device__ __forceinline__ int plan_sms(const Groups &groups, const int32_t *context_lens, int Hk,
                                        int g, int B, const int32_t *lens, int pair_cost, int sms,
                                        bool broken, unsigned long long *sums, int tid, int threads,
                                        int64_t &total) {
    const int per_unit = 2 * (kPrefixTile / g);
    if (tid < 3) sums[tid] = 0;
    __syncthreads();
    unsigned long long tail = 0, places = 0, alone = 0;  // alone: units, groups
    for (int s = tid; s < B; s += threads)
        if (lens[s] > 0) tail += (unsigned)((lens[s] + kBlockSize - 1) / kBlockSize + pair_cost);
    if (!broken)
        for (int r = tid; r < groups.n; r += threads) {
            const PlanGroup p = load_group(groups, context_lens, r, per_unit);
            if (p.tiles == 0) continue;
            places += (unsigned long long)p.span() * p.units;
            alone += (unsigned long long)p.units << 32 | 1;
        }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        tail += __shfl_xor_sync(0xffffffffu, tail, o);
        places += __shfl_xor_sync(0xffffffffu, places, o);
        alone += __shfl_xor_sync(0xffffffffu, alone, o);
    }
    if ((tid & 31) == 0) {
        atomicAdd(&sums[0], tail);
        atomicAdd(&sums[1], places);
        atomicAdd(&sums[2], alone);
    }
    __syncthreads();
    total = (int64_t)sums[1] * Hk;
    alone = sums[2];
    return divide_sms(sums[1], sums[0], (int)(uint32_t)alone, (int64_t)(alone >> 32) * Hk, sms);
}

}  // namespace pa
