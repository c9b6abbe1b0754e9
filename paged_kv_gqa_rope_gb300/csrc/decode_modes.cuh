// What pa_decode_weights and pa_decode_shared have in common with decode.cu:
// the decode kernel's other results, and the groups of sequences that share a
// prefix as every kernel of a call reads them.
#pragma once

#include "common.cuh"
#include "internal.h"

namespace pa {

// Scores and row statistics besides the output (pa_decode_weights).
struct DecodeScores {
    float *scores;     // [blocks of all KV heads][16 tokens][g]: log2 units
    float2 *stats;     // [B][H]: {m, 1 / l}, a weight being 2^(score - m) / l
    int64_t *first;    // [B]: a sequence's first block in scores, -1: none kept
    int64_t capacity;  // blocks of all KV heads that scores holds
    int max_len;       // longest context that the rows of weights hold
};

// Sequences starts[r] .. starts[r + 1] - 1 name the same first blocks[r] blocks.
struct Groups {
    const int32_t *starts;
    const int32_t *blocks;
    int n, maxb;
};

// The groups whose prefixes are read once, as the tails' kernel leaves them for
// the kernels after it.  The prefixes' work lies on a line: group after group,
// KV head after KV head, unit after unit (2 * (128 / g) sequences: two tiles of
// 128 query rows), 128-key tile after tile; G CTAs take equal ranges of it.
struct alignas(16) PlanGroup {
    int64_t start;  // first tile of the group on the line
    int tiles;      // key tiles of a unit
    int blocks;     // blocks shared
    int s0;         // first sequence
    int members;
    int lead;       // sequence whose block table is read
    int units;      // units of a KV head
};
// What the join needs of a sequence.
struct alignas(16) SeqPlan {
    int64_t start;   // line: first tile of its unit, of KV head 0
    int64_t stride;  // tiles from a KV head's unit to the next head's
    int tiles;       // of its unit
    int local;       // row of its first Q head (of a KV head) in the unit
    int state;
    int tail;        // tokens behind the shared blocks
};
enum : int { kInGroup = 0, kAlone = -1, kLeftOut = -2 };  // SeqPlan::state
// Where a CTA's range begins: in tile t0 of unit `unit` (all KV heads counted) of
// group `group` of the plan, and how many tiles it has.  One load, instead of a
// search and 64-bit divisions at the start of every CTA (5.1 us to the first
// scores with those).
struct alignas(16) PlanCut {
    PlanGroup p;
    int64_t tiles;
    int group, unit, t0, pad[3];
};
// Records in the place of the output, over the tokens behind the shared blocks
// (pa_decode_shared): unnormalised O, then m and l of the row.
struct DecodeTails {
    float *rec;  // [B][H][D + 4]
    Groups groups;
    int64_t *total;   // tiles of the line
    PlanGroup *plan;  // [groups.n]: the groups with tiles
    SeqPlan *seqs;    // [B]
    PlanCut *cuts;    // [G]
    int G;            // CTAs of the prefix kernel
};

constexpr int kPrefixTile = 128;  // keys of a tile, and query rows
constexpr int kTileBlocks = kPrefixTile / kBlockSize;

// CTAs with a range (each of one tile at least, so that a unit's pieces are those
// of neighbouring CTAs), the first tile of CTA c's range, and the CTA whose range
// holds tile t.
__device__ __forceinline__ int plan_ctas(int64_t total, int grid) {
    return (int)min(total, (int64_t)grid);
}
__device__ __forceinline__ int64_t plan_cut(int64_t total, int c, int G) { return total * c / G; }
__device__ __forceinline__ int plan_cta(int64_t t, int64_t total, int G) {
    if (total < INT32_MAX / 1024)  // (G <= 160: the sum fits 32 bits)
        return (int)((((uint32_t)t + 1) * (uint32_t)G + (uint32_t)total - 1) / (uint32_t)total) - 1;
    return (int)(((t + 1) * G + total - 1) / total) - 1;
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

// The decode kernel in its other modes.  Its arrival counters (zero between
// calls) and the CTAs' records stand at the start of the workspace, at the same
// place and of the same size whatever the call's shape, and nothing else is
// written there: so one workspace serves calls of several shapes.
constexpr int kModePairs = 1 << 18;  // (sequence, KV head) pairs with a counter
size_t mode_workspace_bytes(int head_dim);
int launch_decode_scores(const DecodeCall &c, void *workspace, const DecodeScores &sc);
int launch_decode_tails(const DecodeCall &c, void *workspace, const DecodeTails &tl);

// A prefix is read once for its group if that saves at least this many blocks
// of a KV head, else by each sequence with the rest of its context (a single
// sequence has nothing to share).
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

// The plan of the groups read_groups has gone over, by one warp of every CTA:
// CTA 0 writes it down, CTA c the cut of the prefix kernel's CTA c.
__device__ __forceinline__ void write_plan(const DecodeTails &tl, const int32_t *skip,
                                           const int32_t *lens, int Hk, int g, int B, bool broken,
                                           int lane, int cta, int ctas) {
    const int mpt = kPrefixTile / g, per_unit = 2 * mpt;
    const bool writes = cta == 0;
    if (broken) {
        if (writes) {
            for (int s = lane; s < B; s += 32) tl.seqs[s].state = kLeftOut;
            if (lane == 0) *tl.total = 0;
        }
        return;
    }
    // Groups r0 .. r0 + 31, one a lane, and the tiles that each has of the line.
    auto load = [&](int r0, PlanGroup &p) -> int64_t {
        p = PlanGroup{};
        if (r0 + lane < tl.groups.n) {
            p.s0 = __ldg(tl.groups.starts + r0 + lane);
            p.members = __ldg(tl.groups.starts + r0 + lane + 1) - p.s0;
            p.lead = p.s0;
            while (p.lead < p.s0 + p.members && skip[p.lead] < 0) ++p.lead;
            p.blocks = p.lead < p.s0 + p.members ? skip[p.lead] : 0;
            p.tiles = (p.blocks + kTileBlocks - 1) / kTileBlocks;
            p.units = (p.members + per_unit - 1) / per_unit;
        }
        return (int64_t)p.tiles * p.units * Hk;
    };
    auto scan = [&](int64_t x) {
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x += y;
        }
        return x;
    };
    PlanGroup p;
    int64_t line = 0;
    int count = 0;
    for (int r0 = 0; r0 < tl.groups.n; r0 += 32) {
        const int64_t mine = load(r0, p), sum = scan(mine);
        p.start = line + sum - mine;
        if (writes) {
            const uint32_t has = __ballot_sync(0xffffffffu, mine > 0);
            if (mine > 0) tl.plan[count + __popc(has & ((1u << lane) - 1))] = p;
            count += __popc(has);
            for (int i = 0; i < min(32, tl.groups.n - r0); ++i) {
                const int s0 = __shfl_sync(0xffffffffu, p.s0, i);
                const int m = __shfl_sync(0xffffffffu, p.members, i);
                SeqPlan q = {};
                q.start = __shfl_sync(0xffffffffu, p.start, i);
                q.tiles = __shfl_sync(0xffffffffu, p.tiles, i);
                q.stride = (int64_t)q.tiles * __shfl_sync(0xffffffffu, p.units, i);
                for (int s = s0 + lane; s < s0 + m; s += 32) {
                    const int u = (s - s0) / per_unit, in = s - s0 - u * per_unit;
                    SeqPlan x = q;
                    x.start += (int64_t)u * x.tiles;
                    x.local = in / mpt * kPrefixTile + in % mpt * g;
                    x.state = skip[s] < 0 ? kLeftOut : q.tiles > 0 ? kInGroup : kAlone;
                    x.tail = lens[s];
                    tl.seqs[s] = x;
                }
            }
        }
        line += __shfl_sync(0xffffffffu, sum, 31);
    }
    if (writes && lane == 0) *tl.total = line;
    // The group that holds a cut, and where the cut lies in it.
    const int G = plan_ctas(line, tl.G);
    for (int c = cta; c < G; c += ctas) {
        const int64_t at = plan_cut(line, c, G);
        int64_t before = 0;
        int group = 0;
        for (int r0 = 0; r0 < tl.groups.n; r0 += 32) {
            const int64_t mine = load(r0, p), sum = scan(mine);
            p.start = before + sum - mine;
            const uint32_t has = __ballot_sync(0xffffffffu, mine > 0);
            if (p.start <= at && at < p.start + mine) {
                PlanCut cut = {};
                cut.p = p;
                cut.tiles = plan_cut(line, c + 1, G) - at;
                cut.group = group + __popc(has & ((1u << lane) - 1));
                cut.unit = (int)((at - p.start) / p.tiles);
                cut.t0 = (int)((at - p.start) % p.tiles);
                tl.cuts[c] = cut;
            }
            group += __popc(has);
            before += __shfl_sync(0xffffffffu, sum, 31);
            if (before > at) break;
        }
    }
}

}  // namespace pa
