// Decode of sequences that share a prefix (pa_decode_shared).
//
// A group's n sequences name the same first blocks, so its n g query rows of a KV
// head (g Q heads each) meet the same K and V: out = softmax(q K^T) V over prefix and
// own tokens is joined from parts that each leave the row's maximum m, sum l and
// unnormalised O,
//     M = max m_i,   out = sum 2^(m_i - M) O_i / sum 2^(m_i - M) l_i.
// Three kernels:
//   prefix  (below) the shared blocks, read once a group, on the tensor cores:
//           tiles of 128 query rows (128 / g sequences) x 128 keys, two tiles of rows
//           a unit, the units' key tiles laid on one line and cut evenly between the
//           CTAs of some of the SMs;
//   tails   decode.cu's kernel over what each sequence has behind them, on the other
//           SMs: it is launched as the prefix kernel's programmatic dependent and does
//           not wait for it;
//   join    one row's records after another, of the tail and of the pieces into which
//           CTA ranges cut the row's unit.
// The prefix kernel's CTAs each work out the plan (every CTA the same): which groups
// share enough, the line, and how the SMs are divided, by the work of both sides.
//
// Bound: HBM for up to 128 query rows a KV head (each key tile of 64 KB serves them
// all: 32 sequences, 32/32 heads, 65536 tokens at 6.3 TB/s), the tensor cores above
// (128 sequences, 64/8 heads, 65536 tokens at 1080 TFLOP/s, 5 % of the time the row sums'
// operations beside the other stream's exponentials; an issuing thread is held 1370
// cycles a job of 128 x 128 x 128 twice, at the 1.5 GHz that the power limit leaves).
// Serving batches of 8192 shared tokens are bound by latencies: about 4 us to the first
// tile, 2 a record, 3 for the join.
#include <algorithm>
#include <climits>
#include <mutex>

#include "decode_modes.cuh"
#include "tcgen05.cuh"

namespace pa {
namespace {

struct SharedArgs {
    const __half *q;
    const int32_t *block_tables;
    const int32_t *context_lens;
    __half *out;
    Groups groups;
    float *tails;  // records of the tails (DecodeTails), and the CTAs'
    float *tail_recs;
    const int32_t *tail_cut;
    PlanHead *head;
    SeqPlan *seqs;
    // Records of a unit's first piece, over the same rows, and of the piece with which
    // a CTA's range begins inside a unit, over the rows of two tiles.
    float *first;  // [B * H rows]
    float *more;   // [G][256 rows]
    int32_t *status;
    float scale_log2;
    int B, H, Hk, g, maxb, num_blocks, plane_k, plane_v, G;
};

// ------------------------------------------------------------------ prefixes

// Roles: warps 0-3 and 4-7 the softmax of stream 0 and 1 (thread = query row =
// TMEM lane), warp 8 the TMA producer of the Q and K tiles, warp 11 of the V tiles
// (a copy of 2 KB takes its thread about 70 cycles: with one producer a tile of 64 KB
// took 2.2 us), warps 9 and 10 the MMA issuers of stream 0 and 1 (one thread each;
// warp 9 owns the TMEM).
constexpr int kProducerWarp = 8;
constexpr int kMmaWarp = 9;
constexpr int kVProducerWarp = 11;
constexpr int kPrefixThreads = 12 * 32;
constexpr int kTmemCols = 512;
constexpr float kRescale = 8.f;   // the maximum moves only when a tile raises it by more
constexpr float kShift = 7.f;     // P = 2^(x - m + 7) <= 2^15
constexpr int kValidRing = 16;    // tiles whose mask of blocks is kept

template <int D>
struct PrefixLayout {
    static constexpr int kHalf = kPrefixTile * 128;    // 64 columns of a tile
    static constexpr int kTileBytes = kHalf * (D / 64);
    static constexpr int kKStages = D == 128 ? 3 : 5, kVStages = D == 128 ? 2 : 5;
    static constexpr int kK = 2 * kTileBytes;  // behind two Q tiles
    static constexpr int kV = kK + kKStages * kTileBytes;
    static constexpr int kBytes = kV + kVStages * kTileBytes;
    // barriers and small arrays, at most 1008 bytes to the 1024-byte boundary of
    // the tiles (the window starts 16-byte aligned)
    static constexpr int kMisc = 512 + kValidRing * 4 + 2 * kPrefixTile * 4;
    static constexpr size_t smem() { return kMisc + 1008 + kBytes; }
};

enum {
    B_QFULL = 0,
    B_QEMPTY = 1,  // both issuers: the segment's last scores done
    B_SFULL = 2,   // per stream: a score tile written
    B_PREADY = 4,  // per stream: its P written
    B_OUNIT = 6,   // per stream: the segment's last P.V done
    B_OFREE = 8,   // per stream: O read out
    B_STATS = 10,  // stream 1's row statistics written
    B_DRAIN = 11,  // per stream
    B_TURN = 13,   // per stream: the other issuer's turn is over
    B_KFULL = 15,  // up to 5 stages each
    B_KEMPTY = 20,
    B_VFULL = 25,
    B_VEMPTY = 30,
    B_COUNT = 35
};
static_assert(B_COUNT * 8 + 4 <= 448, "barrier area");

__device__ __forceinline__ float u2f(uint32_t x) { return __uint_as_float(x); }

__device__ __forceinline__ void tma_load_4d(void *dst, const CUtensorMap *map, uint64_t *bar,
                                            int c0, int c1, int c2, int c3) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(c3),
        "r"(smem_u32(bar))
        : "memory");
}

// 16 consecutive 32-bit columns of this thread's lane, waited for.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
        "%11, %12, %13, %14, %15}, [%16];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
          "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
}

// A load whose value nobody waits for.
__device__ __forceinline__ void touch(const int32_t *p) {
    [[maybe_unused]] int32_t v;
    asm volatile("ld.global.nc.s32 %0, [%1];" : "=r"(v) : "l"(p));
}

// The part of the CTA's range that lies in one unit.
struct PrefixSegment {
    PlanGroup p;
    int kvh, member0, tiles, t0;  // first member of the unit; key tiles, first of them
    bool pair;                    // two tiles of query rows: a stream each, else the
                                  // streams take the key tiles in turn
    __device__ __forceinline__ int count(int t) const {
        return pair ? tiles : (tiles + 1 - t) >> 1;
    }
};

// Walks a CTA's range; every role has its own.
struct PrefixWalk {
    int64_t left;  // places to go
    int group, unit, t0;
    PrefixSegment seg;
    __device__ __forceinline__ void begin(const PlanCut &c) {
        seg.p = c.p;
        left = c.places;
        group = c.group;
        unit = c.unit;
        t0 = c.t0;
    }
    __device__ __forceinline__ bool next(const SharedArgs &a) {
        const int mpt = kPrefixTile / a.g;
        while (left > 0) {
            if (unit == seg.p.units * a.Hk) {
                do {  // (places are left, so a group with some follows; to the last at most)
                    if (++group >= a.groups.n) return false;
                    seg.p = load_group(a.groups, a.context_lens, group, 2 * mpt);
                } while (seg.p.tiles == 0);
                unit = 0;
            }
            // the tiles whose first place is in the range
            const uint32_t wt = seg.p.weight, span = seg.p.span();
            const uint32_t to = t0 + left < span ? (uint32_t)(t0 + left) : span;
            seg.t0 = (int)((t0 + wt - 1) / wt);
            seg.tiles = min((int)((to + wt - 1) / wt), seg.p.tiles) - seg.t0;
            seg.kvh = unit / seg.p.units;
            seg.member0 = (unit - seg.kvh * seg.p.units) * 2 * mpt;
            seg.pair = seg.p.members - seg.member0 > mpt;
            left -= seg.p.span() - t0;  // (negative where the range ends inside)
            ++unit;
            t0 = 0;
            if (seg.tiles > 0) return true;  // (else it begins behind the unit's last tile)
        }
        return false;
    }
};

// Groups r0 .. r0 + 31, one a lane: the group, its places of the line and the sum
// of those up to it.
__device__ __forceinline__ int64_t load_groups(const SharedArgs &a, int r0, int lane, PlanGroup &p,
                                               int64_t &sum) {
    p = PlanGroup{};
    if (r0 + lane < a.groups.n)
        p = load_group(a.groups, a.context_lens, r0 + lane, 2 * (kPrefixTile / a.g));
    const int64_t mine = p.tiles > 0 ? (int64_t)p.span() * p.units * a.Hk : 0;
    sum = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += y;
    }
    return mine;
}

// By one warp: where this CTA's range begins.
__device__ __forceinline__ void find_cut(const SharedArgs &a, PlanCut *cut, int64_t total, int G,
                                         int lane) {
    const int64_t at = plan_cut(total, blockIdx.x, G);
    int64_t before = 0;
    for (int r0 = 0; r0 < a.groups.n && before <= at; r0 += 32) {
        PlanGroup p;
        int64_t sum;
        const int64_t mine = load_groups(a, r0, lane, p, sum);
        const int64_t start = before + sum - mine;
        if (start <= at && at < start + mine) {
            const int span = p.span();
            cut->p = p;
            cut->places = plan_cut(total, blockIdx.x + 1, G) - at;
            cut->group = r0 + lane;
            cut->unit = (int)(total < kShortLine ? (uint32_t)(at - start) / (uint32_t)span
                                                 : (at - start) / span);
            cut->t0 = (int)(at - start - (int64_t)cut->unit * span);
        }
        before += __shfl_sync(0xffffffffu, sum, 31);
    }
}

// By one CTA: what the tails' kernel and the join need.
__device__ __forceinline__ void write_plan(const SharedArgs &a, const int32_t *skip,
                                           const int32_t *lens, bool broken, int64_t total, int sms,
                                           int G, int tid) {
    if (tid == 0) *a.head = {total, G, sms < a.G ? 2 * (a.G - sms) : a.G};
    const int mpt = kPrefixTile / a.g, per_unit = 2 * mpt, lane = tid & 31;
    if (broken) {
        for (int s = tid; s < a.B; s += kPrefixThreads) {
            SeqPlan x = {};
            x.state = kLeftOut;
            a.seqs[s] = x;
        }
        return;
    }
    int64_t line = 0;
    for (int r0 = 0; r0 < a.groups.n; r0 += 32) {
        PlanGroup p;
        int64_t sum;
        const int64_t mine = load_groups(a, r0, lane, p, sum), start = line + sum - mine;
        // (a group a warp)
        for (int i = tid >> 5; i < min(32, a.groups.n - r0); i += kPrefixThreads / 32) {
            const int s0 = __shfl_sync(0xffffffffu, p.s0, i);
            const int m = __shfl_sync(0xffffffffu, p.members, i);
            SeqPlan q = {};
            q.start = __shfl_sync(0xffffffffu, start, i);
            const int tiles = __shfl_sync(0xffffffffu, p.tiles, i);
            const int span = __shfl_sync(0xffffffffu, p.span(), i);
            q.last = (tiles - 1) * __shfl_sync(0xffffffffu, p.weight, i);
            q.stride = (int64_t)span * __shfl_sync(0xffffffffu, p.units, i);
            for (int s = s0 + lane; s < s0 + m; s += 32) {
                const int u = (s - s0) / per_unit, in = s - s0 - u * per_unit;
                SeqPlan x = q;
                x.start += (int64_t)u * span;
                x.local = in / mpt * kPrefixTile + in % mpt * a.g;
                x.state = skip[s] < 0 ? kLeftOut : tiles > 0 ? kInGroup : kAlone;
                x.skip = max(skip[s], 0);
                x.tail = lens[s];
                a.seqs[s] = x;
            }
        }
        line += __shfl_sync(0xffffffffu, sum, 31);
    }
}

// The plan of up to 32 groups: every warp keeps them in its lanes, and one barrier is
// all the CTA needs (the steps for more groups, one after another, take 4 us).
struct FewGroups {
    unsigned long long tail[kPrefixThreads / 32];
    int lead[32];  // set to INT_MAX before the kernel's first barrier
};

__device__ __forceinline__ PlanCut plan_few(const SharedArgs &a, FewGroups *few, int tid) {
    const int lane = tid & 31, n = a.groups.n, maxb = a.groups.maxb;
    const int mpt = kPrefixTile / a.g, per_unit = 2 * mpt;
    // ---- all that is read, at once
    const int mine = min(lane, n - 1);
    int ctx = __ldg(a.context_lens + min(tid, a.B - 1));
    const int g0 = __ldg(a.groups.starts + mine), g1 = __ldg(a.groups.starts + mine + 1);
    const int named = __ldg(a.groups.blocks + mine);
    const bool broken = __any_sync(0xffffffffu, g0 > g1 || (lane == 0 && g0 != 0) ||
                                                    (mine == n - 1 && g1 != a.B));
    const bool in_range = named >= 0 && named <= maxb;
    const int kept = in_range ? shared_of(named, g1 - g0) : -1;
    // A sequence's group, shared blocks (-1: left out) and tokens behind them.
    auto sequence = [&](int s, int len, int &r, int &skip, int &own) {
        r = 0;
        for (int i = 0; i < n - 1; ++i) r += __shfl_sync(0xffffffffu, g1, i) <= s;
        const int want = __shfl_sync(0xffffffffu, named, r), k = __shfl_sync(0xffffffffu, kept, r);
        const bool fine = !broken && k >= 0 && len >= 1 && len <= maxb * kBlockSize &&
                          len >= want * kBlockSize;
        skip = fine ? k : -1;
        own = fine ? len - k * kBlockSize : 0;
    };
    unsigned long long tail = 0;
    int bad = broken;
    const int rounds = (a.B + kPrefixThreads - 1) / kPrefixThreads;
    for (int i = 0; i < rounds; ++i) {
        const int s = i * kPrefixThreads + tid;
        if (i > 0) ctx = __ldg(a.context_lens + min(s, a.B - 1));
        int r, skip, own;
        sequence(min(s, a.B - 1), ctx, r, skip, own);
        if (s >= a.B) continue;
        bad |= skip < 0;
        if (skip > 0) atomicMin(&few->lead[r], s);
        if (own > 0) tail += (unsigned)((own + kBlockSize - 1) / kBlockSize + kTailCost);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) tail += __shfl_xor_sync(0xffffffffu, tail, o);
    if (lane == 0) few->tail[tid >> 5] = tail;
    bad = __syncthreads_or(bad);
    // ---- the groups' places on the line, and this CTA's
    tail = 0;
#pragma unroll
    for (int i = 0; i < kPrefixThreads / 32; ++i) tail += few->tail[i];
    PlanGroup p;
    p.s0 = g0;
    p.members = g1 - g0;
    p.lead = few->lead[lane];
    p.blocks = lane < n && p.lead != INT_MAX ? kept : 0;
    p.tiles = (p.blocks + kTileBlocks - 1) / kTileBlocks;
    p.units = (p.members + per_unit - 1) / per_unit;
    p.weight = p.members > mpt ? kPairWeight : kTileWeight;
    const int64_t places = p.tiles > 0 ? (int64_t)p.span() * p.units * a.Hk : 0;
    int64_t end = places;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, end, o);
        if (lane >= o) end += y;
    }
    const int64_t start = end - places, total = __shfl_sync(0xffffffffu, end, 31);
    const uint32_t active = __ballot_sync(0xffffffffu, places > 0);
    const int64_t units =
        (int64_t)__shfl_sync(0xffffffffu, p.units, active ? __ffs(active) - 1 : 0) * a.Hk;
    const int sms =
        divide_sms((unsigned long long)(total / a.Hk), tail, __popc(active), units, a.G);
    const int G = plan_ctas(total, sms);

    PlanCut cut = {};
    if ((int)blockIdx.x < G) {
        const int64_t at = plan_cut(total, blockIdx.x, G);
        cut.places = plan_cut(total, blockIdx.x + 1, G) - at;
        const int r = __ffs(__ballot_sync(0xffffffffu, start <= at && at < end)) - 1;
        cut.group = r;
        cut.p.tiles = __shfl_sync(0xffffffffu, p.tiles, r);
        cut.p.blocks = __shfl_sync(0xffffffffu, p.blocks, r);
        cut.p.s0 = __shfl_sync(0xffffffffu, p.s0, r);
        cut.p.members = __shfl_sync(0xffffffffu, p.members, r);
        cut.p.lead = __shfl_sync(0xffffffffu, p.lead, r);
        cut.p.units = __shfl_sync(0xffffffffu, p.units, r);
        cut.p.weight = __shfl_sync(0xffffffffu, p.weight, r);
        const int64_t off = at - __shfl_sync(0xffffffffu, start, r);
        const int span = cut.p.span();
        cut.unit = (int)(total < kShortLine ? (uint32_t)off / (uint32_t)span : off / span);
        cut.t0 = (int)(off - (int64_t)cut.unit * span);
    }

    griddep_wait();
    if (blockIdx.x != 0) {
        griddep_launch_dependents();
    } else {  // what the tails' kernel and the join need
        if (bad && tid == 0) report(a.status, PA_DEV_BAD_LENGTH);
        if (tid == 0) *a.head = {total, G, sms < a.G ? 2 * (a.G - sms) : a.G};
        for (int i = 0; i < rounds; ++i) {
            const int s = i * kPrefixThreads + tid;
            if (rounds > 1) ctx = __ldg(a.context_lens + min(s, a.B - 1));
            int r, skip, own;
            sequence(min(s, a.B - 1), ctx, r, skip, own);
            const int in_group = s - __shfl_sync(0xffffffffu, p.s0, r);
            const int span = __shfl_sync(0xffffffffu, p.span(), r);
            const int tiles = __shfl_sync(0xffffffffu, p.tiles, r);
            const int u = in_group / per_unit, in = in_group - u * per_unit;
            SeqPlan x = {};
            x.tail = own;
            x.skip = max(skip, 0);
            x.state = skip < 0 ? kLeftOut : tiles > 0 ? kInGroup : kAlone;
            x.local = in / mpt * kPrefixTile + in % mpt * a.g;
            x.start = __shfl_sync(0xffffffffu, start, r) + (int64_t)u * span;
            x.stride = (int64_t)span * __shfl_sync(0xffffffffu, p.units, r);
            x.last = (tiles - 1) * __shfl_sync(0xffffffffu, p.weight, r);
            if (s < a.B) a.seqs[s] = x;
        }
        __threadfence();
        __syncthreads();
        griddep_launch_dependents();
    }
    return cut;
}

template <int D>
__global__ void __launch_bounds__(kPrefixThreads, 1)
    prefix_kernel(const __grid_constant__ CUtensorMap qmap,
                  const __grid_constant__ CUtensorMap kvmap, const SharedArgs a) {
    using L = PrefixLayout<D>;
    extern __shared__ __align__(16) uint8_t smem_raw[];
    uint64_t *bar = reinterpret_cast<uint64_t *>(smem_raw);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bar + B_COUNT);
    uint32_t *valid = reinterpret_cast<uint32_t *>(smem_raw + 512);  // [kValidRing]
    float *stats = reinterpret_cast<float *>(valid + kValidRing);    // [128] m, [128] l
    unsigned long long *plan_sums = reinterpret_cast<unsigned long long *>(smem_raw + 448);  // [3]
    uint8_t *smem = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + L::kMisc + 1023) & ~static_cast<uintptr_t>(1023));
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    if (tid < 32) reinterpret_cast<FewGroups *>(stats)->lead[tid] = INT_MAX;
    if (tid == 0) {
        mbar_init(&bar[B_QFULL], 1);
        mbar_init(&bar[B_QEMPTY], 2);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bar[B_SFULL + i], 1);
            mbar_init(&bar[B_PREADY + i], 128);
            mbar_init(&bar[B_OUNIT + i], 1);
            mbar_init(&bar[B_OFREE + i], 128);
            mbar_init(&bar[B_DRAIN + i], 1);
            mbar_init(&bar[B_TURN + i], 1);
        }
        mbar_init(&bar[B_STATS], 128);
        for (int i = 0; i < L::kKStages; ++i) {
            mbar_init(&bar[B_KFULL + i], 1);
            mbar_init(&bar[B_KEMPTY + i], 2);
        }
        for (int i = 0; i < L::kVStages; ++i) {
            mbar_init(&bar[B_VFULL + i], 1);
            mbar_init(&bar[B_VEMPTY + i], 2);
        }
        fence_barrier_init();
    }
    if (warp == kMmaWarp) {
        tc::alloc(tmem_slot, kTmemCols);
        tc::relinquish();
    }
    if (warp == kProducerWarp && lane == 0) {
        tma_prefetch_desc(&qmap);
        tma_prefetch_desc(&kvmap);
    }
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    // The plan reads only the call's metadata, which is complete (as pa_decode's); Q and
    // the cache, which may still be written, and the workspace wait for griddep_wait.
    // The tails' kernel may start once every CTA has passed it (the work before the
    // call is done then) and CTA 0 has written the plan.
    const uint32_t tmem = *tmem_slot;  // S_0 | S_1 | O_0 | O_1
    const int mpt = kPrefixTile / a.g;
    // ---- the plan
    PlanCut cut;
    if (a.groups.n <= 32) {
        cut = plan_few(a, reinterpret_cast<FewGroups *>(stats), tid);
        __syncthreads();  // (stats are free)
    } else {
        // with the room of the tiles for the sequences' lengths; what the steps read
        // first is asked for at once, so that they find it in L1
        touch(a.context_lens + min(tid, a.B - 1));
        touch(a.groups.starts + min(tid, a.groups.n));
        touch(a.groups.blocks + min(tid, a.groups.n - 1));
        PlanCut *shared_cut = reinterpret_cast<PlanCut *>(stats);
        int32_t *skip = reinterpret_cast<int32_t *>(smem), *lens = skip + a.B;
        const int bad = read_groups(a.groups, a.context_lens, a.B, skip, lens, tid, kPrefixThreads);
        int64_t total;
        const int sms = plan_sms(a.groups, a.context_lens, a.Hk, a.g, a.B, lens, kTailCost, a.G,
                                 bad == 2, plan_sums, tid, kPrefixThreads, total);
        const int G = plan_ctas(total, sms);
        if (tid == 0) shared_cut->places = 0;
        __syncthreads();
        griddep_wait();
        if (blockIdx.x != 0) {
            griddep_launch_dependents();
        } else {
            if (bad && tid == 0) report(a.status, PA_DEV_BAD_LENGTH);
            write_plan(a, skip, lens, bad == 2, total, sms, G, tid);
            __threadfence();
            __syncthreads();
            griddep_launch_dependents();
        }
        if (warp == 0 && (int)blockIdx.x < G) find_cut(a, shared_cut, total, G, lane);
        // (the tiles' room was written by the threads, and will be by TMA)
        tc::fence_proxy_async_smem();
        __syncthreads();
        cut = *shared_cut;
        __syncthreads();  // (stats are free)
    }
    PrefixWalk w;
    w.begin(cut);
    auto s_col = [](int t) { return (uint32_t)(t * kPrefixTile); };
    auto o_col = [](int t) { return (uint32_t)(2 * kPrefixTile + t * D); };

    if (warp == kProducerWarp || warp == kVProducerWarp) {
        // ============ producers: K tiles, and a segment's Q tiles behind its first
        // (whose stage frees before the Q tiles' last reader does; the first segment's
        // ahead of them); V tiles
        const bool is_v = warp == kVProducerWarp;
        const int stages = is_v ? L::kVStages : L::kKStages, plane = is_v ? a.plane_v : a.plane_k;
        uint64_t *const full = bar + (is_v ? B_VFULL : B_KFULL);
        uint64_t *const empty = bar + (is_v ? B_VEMPTY : B_KEMPTY);
        uint8_t *const ring = smem + (is_v ? L::kV : L::kK);
        const uint32_t q_bytes = (uint32_t)(a.g * mpt * 128 * (D / 64));
        int ok = 1, segs = 0, tile = 0;
        while (ok && w.next(a)) {
            const PrefixSegment &sg = w.seg;
            const int32_t *row = a.block_tables + (int64_t)sg.p.lead * a.maxb;
            auto block_at = [&](int j) -> int {  // lane's block of key tile j, -1: none
                const int b = (sg.t0 + j) * kTileBlocks + lane;
                if (lane >= kTileBlocks || j >= sg.tiles || b >= sg.p.blocks) return -1;
                const int blk = __ldg(row + b);
                if (blk >= 0 && blk < a.num_blocks) return blk;
                if (!is_v) report(a.status, PA_DEV_BAD_BLOCK);
                return -1;
            };
            auto load_q = [&]() {
                mbar_arrive_expect_tx(&bar[B_QFULL], q_bytes * (sg.pair ? 2 : 1));
                for (int t = 0; t < (sg.pair ? 2 : 1); ++t)
                    for (int hf = 0; hf < D / 64; ++hf)
                        tma_load_4d(smem + t * L::kTileBytes + hf * L::kHalf, &qmap, &bar[B_QFULL],
                                    0, hf, sg.kvh * a.g, sg.p.s0 + sg.member0 + t * mpt);
            };
            int blk = block_at(0);
            if (!is_v && segs == 0 && lane == 0) load_q();
            for (int j = 0; j < sg.tiles && ok; ++j, ++tile) {
                const int st = tile % stages;
                const uint32_t have = __ballot_sync(0xffffffffu, blk >= 0);
                // (a block that is missing comes from behind the pool: zeros)
                const int r0 = (blk >= 0 ? blk : a.num_blocks) * kBlockSize;
                blk = block_at(j + 1);
                ok = mbar_wait(&empty[st], ((tile / stages) & 1) ^ 1);
                if (lane == 0 && ok) {
                    if (!is_v) valid[tile % kValidRing] = have;
                    mbar_arrive_expect_tx(&full[st], L::kTileBytes);
                }
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                if (lane < kTileBlocks)
                    for (int hf = 0; hf < D / 64; ++hf)
                        tma_load_5d(ring + st * L::kTileBytes + hf * L::kHalf + lane * kBlockSize * 128,
                                    &kvmap, &full[st], 0, hf, sg.kvh, r0, plane);
                if (!is_v && j == 0 && segs > 0) {
                    ok = __all_sync(0xffffffffu, mbar_wait(&bar[B_QEMPTY], (segs - 1) & 1));
                    if (lane == 0 && ok) load_q();
                }
            }
            ++segs;
        }
        if (lane == 0) {
            if (!ok) report(a.status, PA_DEV_TIMEOUT);
            // Leave no copy in flight.
            for (int i = max(0, tile - stages); i < tile; ++i)
                mbar_wait(&full[i % stages], (i / stages) & 1);
            if (!is_v && segs > 0) mbar_wait(&bar[B_QFULL], (segs - 1) & 1);
        }
    } else if (warp == kMmaWarp || warp == kMmaWarp + 1) {
        // ============ MMA issuers.  A segment's jobs take the streams in turn: job i is
        // stream i & 1's, against key tile i / 2 of two tiles of query rows, or tile
        // i of one.  Turn i of the segment is thread i & 1's: O_t += P V of job i - 2,
        // and behind it, into the place where that P stood, the scores S_t = Q_t K^T
        // of job i (operations issued by one thread execute in order).  Strict turns
        // keep one stream's softmax beside the other's operations (free-running
        // threads fell in step, both softmaxes and then both products: 2.4 us a tile
        // of two), and while one thread issues, which holds it for the operations' run
        // time, the other waits for its barriers (one thread for both, which waited
        // between: 2096 cycles a job, 1370 of them issuing).
        const int t = warp - kMmaWarp;
        if (lane == 0) {
            constexpr uint32_t kIdescQK = tc::idesc_f16(kPrefixTile, kPrefixTile, false, false);
            constexpr uint32_t kIdescPV = tc::idesc_f16(kPrefixTile, D, false, true);
            const uint64_t dq0 = tc::smem_desc_sw128(smem_u32(smem), 16, 1024);
            const uint64_t dk0 = tc::smem_desc_sw128(smem_u32(smem + L::kK), 16, 1024);
            const uint64_t dv0 = tc::smem_desc_sw128(smem_u32(smem + L::kV), L::kHalf, 1024);
            bool ok = true;
            int tile = 0, segs = 0;  // key tiles, segments before this one
            int turns = 0;           // turns of this thread
            int g = 0, un = 0;       // jobs, segments with jobs of this stream
            // Tile j has been loaded.  (Each thread waits for every tile of a ring, in
            // order, and gives it back: so a wait by phase parity is exact.)
            auto k_wait = [&](int j) {
                return mbar_wait(&bar[B_KFULL + j % L::kKStages], (j / L::kKStages) & 1);
            };
            auto v_wait = [&](int j) {
                return mbar_wait(&bar[B_VFULL + j % L::kVStages], (j / L::kVStages) & 1);
            };
            while (ok && w.next(a)) {
                const PrefixSegment &sg = w.seg;
                const bool pair = sg.pair;
                const int jobs = pair ? 2 * sg.tiles : sg.tiles;
                const uint64_t dq = dq0 + (uint64_t)((pair && t ? L::kTileBytes : 0) >> 4);
                ok = mbar_wait(&bar[B_QFULL], segs & 1);
                ++segs;
                if (ok && t >= jobs) mbar_arrive(&bar[B_QEMPTY]);
                // (an even number of turns, so that thread 0 begins the next segment)
                for (int i = t; i < ((jobs + 3) & ~1) && ok; i += 2) {
                    const bool scores = i < jobs, values = i >= 2 && i < jobs + 2;
                    const int kj = tile + (pair ? i >> 1 : i), vj = tile + (pair ? (i - 2) >> 1 : i - 2);
                    if (!pair) {  // the other stream's tiles
                        if (i >= 3 && i - 3 < jobs) {
                            ok = v_wait(tile + i - 3);
                            mbar_arrive(&bar[B_VEMPTY + (tile + i - 3) % L::kVStages]);
                        }
                        if (i >= 1 && i - 1 < jobs) {
                            ok = ok && k_wait(tile + i - 1);
                            mbar_arrive(&bar[B_KEMPTY + (tile + i - 1) % L::kKStages]);
                        }
                    }
                    if (values) {
                        ok = ok && v_wait(vj) && mbar_wait(&bar[B_PREADY + t], g & 1);
                        // the stream's O of the segment before has to have been read
                        if (ok && i < 4 && un > 0) ok = mbar_wait(&bar[B_OFREE + t], (un - 1) & 1);
                    }
                    if (scores) ok = ok && k_wait(kj);
                    // (thread 0's first turn is free)
                    ok = ok && mbar_wait(&bar[B_TURN + t], (turns & 1) ^ (t == 0 ? 1 : 0));
                    ++turns;
                    if (!ok) break;
                    tc::fence_after();
                    if (values) {
                        const int st = vj % L::kVStages;
                        const uint64_t dv = dv0 + (uint64_t)((st * L::kTileBytes) >> 4);
#pragma unroll
                        for (int kk = 0; kk < kPrefixTile / 16; ++kk)
                            tc::mma_ts(tmem + o_col(t), tmem + s_col(t) + kk * 8,
                                       dv + (uint64_t)((kk * 16 * 128) >> 4), kIdescPV,
                                       (i >= 4 || kk > 0) ? 1u : 0u);
                        tc::commit(&bar[B_VEMPTY + st]);
                        if (i >= jobs) tc::commit(&bar[B_OUNIT + t]);
                        ++g;
                    }
                    if (scores) {
                        const int st = kj % L::kKStages;
                        const uint64_t dk = dk0 + (uint64_t)((st * L::kTileBytes) >> 4);
#pragma unroll
                        for (int kk = 0; kk < D / 16; ++kk) {
                            const uint64_t step = (uint64_t)(((kk >> 2) * L::kHalf + (kk & 3) * 32) >> 4);
                            tc::mma_ss(tmem + s_col(t), dq + step, dk + step, kIdescQK, kk > 0);
                        }
                        tc::commit(&bar[B_SFULL + t]);
                        tc::commit(&bar[B_KEMPTY + st]);
                        if (i + 2 >= jobs) tc::commit(&bar[B_QEMPTY]);
                    }
                    mbar_arrive(&bar[B_TURN + 1 - t]);
                }
                // (the last V tile, if it was the other's and this thread had no turn left)
                if (ok && !pair && ((jobs - 1) & 1) != t && jobs + 2 >= ((jobs + 3) & ~1)) {
                    ok = v_wait(tile + jobs - 1);
                    mbar_arrive(&bar[B_VEMPTY + (tile + jobs - 1) % L::kVStages]);
                }
                tile += sg.tiles;
                un += t < jobs;
            }
            if (!ok) report(a.status, PA_DEV_TIMEOUT);
            // Nothing of ours may still be running when the CTA frees TMEM.
            tc::commit(&bar[B_DRAIN + t]);
            mbar_wait(&bar[B_DRAIN + t], 0);
        }
        __syncwarp();
    } else {
        // ============ softmax of stream t
        const int t = warp >> 2, r = tid - t * 128;
        const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t s_tmem = tmem + lane_base + s_col(t), o_tmem = tmem + lane_base + o_col(t);
        const float sl2 = a.scale_log2;
        const uint64_t sl2x2 = f2_pack(sl2, sl2);
        bool ok = true;
        int g = 0, un = 0, tile = 0, merged = 0;
        while (ok && w.next(a)) {
            const PrefixSegment &sg = w.seg;
            const int n = sg.count(t);
            float m = -INFINITY, l = 0.f;
            for (int i = 0; i < n; ++i, ++g) {
                ok = __all_sync(0xffffffffu, mbar_wait(&bar[B_SFULL + t], g & 1));
                if (!ok) break;
                tc::fence_after();
                const uint32_t have = valid[(tile + (sg.pair ? i : 2 * i + t)) % kValidRing];
                uint32_t s0[32], s1[32], s2[32], s3[32];
                float x0, x1, x2, x3;
                tc::ld32_max_issue(s_tmem, s0, x0);
                tc::ld32_max_issue(s_tmem + 32, s1, x1);
                tc::ld32_max_issue(s_tmem + 64, s2, x2);
                tc::ld32_max_issue(s_tmem + 96, s3, x3);
                tc::wait_ld(s0, s1, x0, x1);
                tc::wait_ld(s2, s3, x2, x3);
                if (have != (1u << kTileBlocks) - 1) {
                    // blocks that are missing: 16 columns each
                    auto mask = [&](uint32_t (&s)[32], float &x, int b) {
                        x = -INFINITY;
#pragma unroll
                        for (int c = 0; c < 32; ++c) {
                            if (!(have >> (b + (c >> 4)) & 1)) s[c] = __float_as_uint(-INFINITY);
                            x = fmaxf(x, u2f(s[c]));
                        }
                    };
                    mask(s0, x0, 0);
                    mask(s1, x1, 2);
                    mask(s2, x2, 4);
                    mask(s3, x3, 6);
                }
                const float mt = fmaxf(fmax3(x0, x1, x2), x3) * sl2;
                const bool up = mt > m + kRescale;
                float f = 1.f;
                if (up) {
                    f = ex2(m - mt);  // 0 for the segment's first
                    l *= f;
                    m = mt;
                }
                if (i > 0 && __any_sync(0xffffffffu, up)) {
                    // (these scores were issued behind the last P.V, and their
                    // barrier tracks both: O is complete)
#pragma unroll 1
                    for (int c = 0; c < D; c += 16) {
                        uint32_t o[16];
                        tmem_ld16(o_tmem + c, o);
#pragma unroll
                        for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(u2f(o[k]) * f);
                        tc::st16(o_tmem + c, o);
                    }
                }
                const float base = (m == -INFINITY ? 0.f : m) - kShift;
                const uint64_t negm = f2_pack(-base, -base);
                // P is rounded to fp16 (by 2^-11 of a value at most), as pa_decode's: P V
                // then is one product, not the two of a value in two halves, whose error
                // against 64 bits would be 2.1e-4, the output's own rounding, in place of
                // 2.9e-4 (32 sequences over 8192 shared tokens, 64/8 heads: 25.6 us, in two
                // halves 31.6; 128 over 65536: 254 and 343).  The row sum adds the
                // rounded P, so that the output is an average of V by the weights that
                // multiplied it, as pa_decode's; it does so once the tile's P is given
                // away, beside the product (64/8 heads, 32 sequences over 8192 shared tokens:
                // 25.6 us, 128 over 65536: 254; summed ahead of that 25.7 and 257, P before
                // its rounding 25.4 and 243).
                uint32_t p[4][16];
                auto exps = [&](const uint32_t (&s)[32], int c, uint32_t (&p)[16]) {
#pragma unroll
                    for (int k = 0; k < 16; k += 2) {
                        float e0, e1, e2, e3;
                        f2_unpack(f2_fma(f2_pack(u2f(s[2 * k]), u2f(s[2 * k + 1])), sl2x2, negm), e0, e1);
                        f2_unpack(f2_fma(f2_pack(u2f(s[2 * k + 2]), u2f(s[2 * k + 3])), sl2x2, negm), e2, e3);
                        e0 = ex2(e0);
                        e1 = ex2(e1);
                        e2 = ex2(e2);
                        e3 = ex2(e3);
                        p[k] = pack_half2(e0, e1);
                        p[k + 1] = pack_half2(e2, e3);
                    }
                    tc::st16(s_tmem + c, p);
                };
                exps(s0, 0, p[0]);
                exps(s1, 16, p[1]);
                exps(s2, 32, p[2]);
                exps(s3, 48, p[3]);
                tc::wait_st();
                tc::fence_before();
                mbar_arrive(&bar[B_PREADY + t]);
                float y0 = 0.f, y1 = 0.f, y2 = 0.f, y3 = 0.f;
#pragma unroll
                for (int k = 0; k < 64; k += 2) {
                    add_halves(y0, y1, p[k / 16][k % 16]);
                    add_halves(y2, y3, p[k / 16][k % 16 + 1]);
                }
                l += (y0 + y1) + (y2 + y3);
            }
            tile += sg.tiles;
            if (!ok) break;
            if (n == 0) continue;

            // ---- the segment's record: m and l are of P = 2^(x - m + kShift)
            ok = __all_sync(0xffffffffu, mbar_wait(&bar[B_OUNIT + t], un & 1));
            ++un;
            if (!ok) break;
            tc::fence_after();
            float f0 = 1.f, f1 = 0.f;
            const bool both = !sg.pair && sg.tiles > 1;
            if (both) {
                // one tile of rows: stream 0 joins what both have of it
                if (t == 1) {
                    stats[r] = m;
                    stats[kPrefixTile + r] = l;
                    tc::fence_before();
                    mbar_arrive(&bar[B_STATS]);
                    continue;
                }
                ok = __all_sync(0xffffffffu, mbar_wait(&bar[B_STATS], merged & 1));
                // (stream 1's last P.V: its thread has waited for it)
                ++merged;
                if (!ok) break;
                tc::fence_after();
                const float m1 = stats[r], l1 = stats[kPrefixTile + r];
                const float M = fmaxf(m, m1);
                f0 = m == -INFINITY ? 0.f : ex2(m - M);
                f1 = m1 == -INFINITY ? 0.f : ex2(m1 - M);
                l = f0 * l + f1 * l1;
                m = M;
            }
            const int member = sg.member0 + (sg.pair ? t * mpt : 0) + r / a.g;
            const bool live = r < mpt * a.g && member < sg.p.members;
            Record rec;
            if (sg.t0 == 0) {
                rec.base = a.first;
                rec.rows = (int64_t)a.B * a.H;
                rec.row = ((int64_t)sg.kvh * a.B + sg.p.s0 + member) * a.g + r % a.g;
            } else {
                rec.base = a.more + (int64_t)blockIdx.x * 2 * kPrefixTile * (D + 4);
                rec.rows = 2 * kPrefixTile;
                rec.row = (sg.pair ? t * kPrefixTile : 0) + r;
            }
#pragma unroll 1
            for (int c = 0; c < D; c += 32) {
                uint32_t o[32], o1[32];
                tc::ld32_issue(o_tmem + c, o);
                tc::ld32_issue(both ? tmem + lane_base + o_col(1) + c : o_tmem + c, o1);
                tc::wait_ld(o, o1);
                if (both) {
#pragma unroll
                    for (int k = 0; k < 32; ++k)
                        o[k] = __float_as_uint(fmaf(f0, u2f(o[k]), f1 * u2f(o1[k])));
                }
                if (live) {
#pragma unroll
                    for (int k = 0; k < 32; k += 4)
                        *rec.cols((c + k) / 4) =
                            make_float4(u2f(o[k]), u2f(o[k + 1]), u2f(o[k + 2]), u2f(o[k + 3]));
                }
            }
            if (live) *rec.stat(D) = make_float2(m - kShift, l);
            tc::fence_before();
            mbar_arrive(&bar[B_OFREE + t]);
            if (both) mbar_arrive(&bar[B_OFREE + 1]);
        }
        if (!ok && lane == 0) report(a.status, PA_DEV_TIMEOUT);
    }

    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    if (warp == kMmaWarp) tc::dealloc(tmem, kTmemCols);
}

// 4-D fp16 map of q [B][H][D]: {64, D/64, H, B}, box {64, 1, g, 128/g}: the query
// rows of a tile, (sequence, head) one after another.
bool make_group_map(CUtensorMap *map, const void *base, int B, int H, int D, int g) {
    EncodeTiledFn enc = encode_tiled();
    if (!enc) return false;
    cuuint64_t dims[4] = {64, (cuuint64_t)(D / 64), (cuuint64_t)H, (cuuint64_t)B};
    cuuint64_t strides[3] = {128, (cuuint64_t)D * 2, (cuuint64_t)H * D * 2};
    cuuint32_t box[4] = {64, 1, (cuuint32_t)g, (cuuint32_t)(kPrefixTile / g)};
    cuuint32_t estr[4] = {1, 1, 1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4, const_cast<void *>(base), dims, strides,
               box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D>
int launch_prefix(const SharedArgs &a, const pa_cache_t *cache, cudaStream_t st) {
    static std::mutex mu;
    static bool attr_set[64] = {false};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return PA_ERR_CUDA;
    {
        std::lock_guard<std::mutex> lock(mu);
        if (!attr_set[dev]) {
            if (cudaFuncSetAttribute(prefix_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     (int)PrefixLayout<D>::smem()) != cudaSuccess) {
                cudaGetLastError();
                return PA_ERR_CUDA;
            }
            attr_set[dev] = true;
        }
    }
    CUtensorMap qmap, kvmap;
    if (!make_group_map(&qmap, a.q, a.B, a.H, D, a.g) || !make_cache_map(&kvmap, cache, 1, kBlockSize))
        return PA_ERR_CUDA;
    launch_dependent(prefix_kernel<D>, dim3(a.G), dim3(kPrefixThreads), PrefixLayout<D>::smem(), st,
                     qmap, kvmap, a);
    return launch_status();
}

constexpr int kJoinThreads = 256;
// Records in flight: 4 took 30.2 us for 32 sequences of 64/8 heads that share 8192 tokens
// (12 pieces a unit), 8 29.1, 12 28.5, 16 28.6.
constexpr int kJoinBatch = 12;

// Joins a row's records: a thread has four columns of a row, the 32 threads of a
// warp the same columns of 32 rows (in the records' order), blockIdx.y the columns.
template <int D>
__global__ void __launch_bounds__(kJoinThreads) join_kernel(const SharedArgs a) {
    griddep_wait();
    griddep_launch_dependents();
    const int lane = threadIdx.x & 31;
    const int c4 = blockIdx.y * (kJoinThreads / 32) + (threadIdx.x >> 5);
    const int64_t at = (int64_t)blockIdx.x * 32 + lane;  // (KV head, sequence, its Q head)
    if (at >= (int64_t)a.B * a.H) return;
    const int j = (int)at % a.g, s = (int)at / a.g % a.B, kvh = (int)at / a.g / a.B;
    const int64_t row = (int64_t)s * a.H + kvh * a.g + j, rows = (int64_t)a.B * a.H;
    // Every row that is not alone has a first piece of its prefix; it and the tail's
    // record do not wait for the plan, nor the other pieces for each other.
    float2 ml[kJoinBatch];
    float4 x[kJoinBatch];
    auto take = [&](int i, const Record &r) {
        ml[i] = __ldcg(r.stat(D));
        x[i] = __ldcg(r.cols(c4));
    };
    auto none = [&](int i) {
        ml[i] = make_float2(-INFINITY, 0.f);
        x[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    };
    take(0, {a.tails, rows, at});
    take(1, {a.first, rows, at});
    const int cut = __ldcg(a.tail_cut + s * a.Hk + kvh);
    const SeqPlan p = a.seqs[s];
    const PlanHead head = *a.head;
    if (p.state == kLeftOut) return;
    const Cut behind = cut_of(cut);  // the tail's pieces behind its first
    const int tail_more = p.tail > 0 ? behind.more : 0;
    int c0 = 0, more = 0;  // the prefix's
    if (p.state == kInGroup) {
        const int64_t start = p.start + kvh * p.stride;
        c0 = plan_cta(start, head.total, head.ctas);
        more = plan_cta(start + p.last, head.total, head.ctas) - c0;
    } else {
        if (tail_more == 0) return;  // (the tails' kernel has written it)
        none(1);
    }
    if (p.tail == 0) none(0);
    float M = -INFINITY, L = 0.f;
    float4 O = make_float4(0.f, 0.f, 0.f, 0.f);
    auto join = [&](int n) {
        float top = M;
        for (int i = 0; i < n; ++i) top = fmaxf(top, ml[i].x);
        auto factor = [&](float m) { return m == -INFINITY ? 0.f : ex2(m - top); };
        float f = factor(M);
        M = top;
        L *= f;
        O = make_float4(f * O.x, f * O.y, f * O.z, f * O.w);
        for (int i = 0; i < n; ++i) {
            f = factor(ml[i].x);
            L = fmaf(f, ml[i].y, L);
            O.x = fmaf(f, x[i].x, O.x);
            O.y = fmaf(f, x[i].y, O.y);
            O.z = fmaf(f, x[i].z, O.z);
            O.w = fmaf(f, x[i].w, O.w);
        }
    };
    join(2);
    for (int i0 = 0; i0 < tail_more + more; i0 += kJoinBatch) {
#pragma unroll
        for (int i = 0; i < kJoinBatch; ++i) {
            const int n = i0 + i;
            if (n < tail_more)
                take(i, piece_of(a.tail_recs, behind.cta + n, D, j));
            else if (n < tail_more + more)
                take(i, {a.more + (int64_t)(c0 + 1 + n - tail_more) * 2 * kPrefixTile * (D + 4),
                         2 * kPrefixTile, p.local + j});
            else
                none(i);
        }
        join(kJoinBatch);
    }
    const float inv = L == 0.f ? 0.f : 1.f / L;  // (no block in range: 0)
    *reinterpret_cast<uint2 *>(a.out + row * D + 4 * c4) =
        make_uint2(pack_half2(saturate16(O.x * inv), saturate16(O.y * inv)),
                   pack_half2(saturate16(O.z * inv), saturate16(O.w * inv)));
}

size_t up256(size_t n) { return (n + 255) & ~(size_t)255; }

constexpr int kMaxGroups = 4096;
constexpr int kMaxCtas = 160;  // (152 SMs)

size_t rows_bytes(int B, int H, int D) {
    return up256((size_t)B * H * ((size_t)D + 4) * sizeof(float));
}

template <int D>
int launch_join(const SharedArgs &a, cudaStream_t st) {
    const int64_t rows = (int64_t)a.B * a.H;
    launch_dependent(join_kernel<D>, dim3((unsigned)((rows + 31) / 32), D / 4 / (kJoinThreads / 32)),
                     dim3(kJoinThreads), 0, st, a);
    return launch_status();
}

}  // namespace
}  // namespace pa

using namespace pa;

extern "C" size_t pa_decode_shared_workspace_bytes(int num_seqs, int n_heads, int n_kv_heads,
                                                   int head_dim) {
    if (num_seqs <= 0 || n_heads <= 0 || n_kv_heads <= 0 || head_dim <= 0) return 0;
    // (the parts first: each must fit by itself before it is counted in 64 bits)
    const unsigned __int128 row_bytes = (head_dim + (int64_t)4) * sizeof(float);
    const unsigned __int128 n =
        row_bytes * (2 * (unsigned __int128)num_seqs * n_heads + 2 * kPrefixTile * kMaxCtas) +
        (unsigned __int128)num_seqs * sizeof(SeqPlan) +
        (unsigned __int128)num_seqs * n_kv_heads * sizeof(int32_t);
    if (n > SIZE_MAX - mode_workspace_bytes(head_dim) - 8 * 256) return 0;
    return up256(mode_workspace_bytes(head_dim)) + 256 +
           up256((size_t)num_seqs * sizeof(SeqPlan)) +
           up256((size_t)num_seqs * n_kv_heads * sizeof(int32_t)) +
           2 * rows_bytes(num_seqs, n_heads, head_dim) +
           rows_bytes(kMaxCtas, 2 * kPrefixTile, head_dim);
}

extern "C" int pa_decode_shared(const void *q, const pa_cache_t *cache, int layer,
                                const int32_t *block_tables, int max_blocks_per_seq,
                                const int32_t *context_lens, int num_seqs,
                                const int32_t *group_starts, const int32_t *shared_blocks,
                                int num_groups, int n_heads, int n_kv_heads, int head_dim,
                                float scale, void *workspace, size_t workspace_bytes, void *out,
                                int32_t *dev_status, pa_stream_t stream) {
    const int rc = check_decode_args(q, cache, layer, block_tables, max_blocks_per_seq,
                                     context_lens, num_seqs, n_heads, n_kv_heads, head_dim, scale,
                                     out);
    if (rc != PA_OK) return rc;
    if (num_groups < 0) return PA_ERR_INVALID;
    // (rows of the records are counted in int32)
    if (num_groups > kMaxGroups || (int64_t)num_seqs * n_heads > INT32_MAX)
        return PA_ERR_UNSUPPORTED;
    if (num_seqs == 0) return PA_OK;
    if (num_groups == 0 || !group_starts || !shared_blocks || !workspace ||
        (reinterpret_cast<uintptr_t>(workspace) & 255u))
        return PA_ERR_INVALID;
    const size_t need =
        pa_decode_shared_workspace_bytes(num_seqs, n_heads, n_kv_heads, head_dim);
    if (workspace_bytes < need) return PA_ERR_WORKSPACE;
    const int G = std::min(sm_count(), kMaxCtas);
    if (G < 1) return PA_ERR_CUDA;

    uint8_t *at = static_cast<uint8_t *>(workspace);
    uint8_t *p = at + up256(mode_workspace_bytes(head_dim));
    SharedArgs a = {};
    a.head = reinterpret_cast<PlanHead *>(p);
    p += 256;
    a.seqs = reinterpret_cast<SeqPlan *>(p);
    p += up256((size_t)num_seqs * sizeof(SeqPlan));
    int32_t *const tail_cut = reinterpret_cast<int32_t *>(p);
    a.tail_cut = tail_cut;
    a.tail_recs = mode_records(at);
    p += up256((size_t)num_seqs * n_kv_heads * sizeof(int32_t));
    float *const tails = reinterpret_cast<float *>(p);
    a.tails = tails;
    p += rows_bytes(num_seqs, n_heads, head_dim);
    a.first = reinterpret_cast<float *>(p);
    p += rows_bytes(num_seqs, n_heads, head_dim);
    a.more = reinterpret_cast<float *>(p);
    a.groups = {group_starts, shared_blocks, num_groups, max_blocks_per_seq, num_seqs};
    a.q = static_cast<const __half *>(q);
    a.plane_k = layer;
    a.plane_v = cache->layers + layer;
    a.block_tables = block_tables;
    a.context_lens = context_lens;
    a.out = static_cast<__half *>(out);
    a.status = dev_status;
    a.scale_log2 = (scale == 0.f ? 1.0f / sqrtf((float)head_dim) : scale) * 1.4426950408889634f;
    a.B = num_seqs;
    a.H = n_heads;
    a.Hk = n_kv_heads;
    a.g = n_heads / n_kv_heads;
    a.maxb = max_blocks_per_seq;
    a.num_blocks = cache->num_blocks;
    a.G = G;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const DecodeCall c = {q,        cache,   layer,      block_tables, max_blocks_per_seq,
                          context_lens, num_seqs, n_heads, n_kv_heads, head_dim,
                          scale,    out,     dev_status, st};
    int rc2 = head_dim == 128 ? launch_prefix<128>(a, cache, st) : launch_prefix<64>(a, cache, st);
    if (rc2 == PA_OK) rc2 = launch_decode_tails(c, at, DecodeTails{{tails, tail_cut}, a.head, a.seqs});
    if (rc2 != PA_OK) return rc2;
    return head_dim == 128 ? launch_join<128>(a, st) : launch_join<64>(a, st);
}

extern "C" int pa_prepare_shared(int num_seqs, const int32_t *block_tables,
                                 int max_blocks_per_seq, const int32_t *context_lens,
                                 int block_size, int32_t *group_starts, int32_t *shared_blocks,
                                 int32_t *num_groups) {
    if (num_seqs < 0 || max_blocks_per_seq < 0 || block_size <= 0 || !num_groups)
        return PA_ERR_INVALID;
    if (num_seqs > 0 && (!block_tables || !context_lens || !group_starts || !shared_blocks))
        return PA_ERR_INVALID;
    for (int s = 0; s < num_seqs; ++s)
        if (context_lens[s] < 0 ||
            (int64_t)context_lens[s] > (int64_t)max_blocks_per_seq * block_size)
            return PA_ERR_INVALID;
    // Sequence s joins the group before it if that saves more than it costs the
    // others: with c blocks in common among n sequences, (n - 1) c reads of a block
    // are saved.
    int n = 0, members = 0, common = 0;
    if (group_starts) group_starts[0] = 0;
    for (int s = 0; s < num_seqs; ++s) {
        const int full = context_lens[s] / block_size;  // blocks without an empty place
        const int32_t *row = block_tables + (int64_t)s * max_blocks_per_seq;
        if (members > 0) {
            const int32_t *lead = row - max_blocks_per_seq;  // (the one before has the same)
            const int most = common < full ? common : full;
            int c = 0;
            while (c < most && row[c] >= 0 && row[c] == lead[c]) ++c;
            const int64_t now = members == 1 ? 0 : (int64_t)(members - 1) * common;
            if (c > 0 && (int64_t)members * c >= now) {
                common = c;
                ++members;
                shared_blocks[n - 1] = c;
                continue;
            }
        }
        group_starts[n] = s;
        shared_blocks[n] = 0;
        ++n;
        members = 1;
        common = full;
    }
    if (group_starts) group_starts[n] = num_seqs;
    *num_groups = n;
    return PA_OK;
}
