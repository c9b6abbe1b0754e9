// Eviction from the paged fp16 cache by accumulated attention weight
// (pa_kv_evict; the weights are pa_decode_weights').
//
// Of a sequence's n tokens each KV head keeps k = min(n, budget): the first
// `sinks`, the last `recent` and, of the others, the m = k - sinks - recent of
// the largest weight, of equal ones the first.  Two kernels:
//
//   select  one CTA per (sequence, KV head), or where there are few of them a
//           cluster of up to eight, which keep the weights in registers, 32768 tokens
//           a CTA.  Where the tables allow rows past what the cluster then holds
//           (262112 tokens of eight CTAs) it is one CTA that reads those past 32768
//           again, once a digit and once for the places.  The m-th largest weight among
//           the others is found digit by digit (11 + 11 + 10 bits of a key that
//           orders like the weights): a histogram of the digit over the keys that
//           agree on the digits before it, and the digit at which the count from the
//           top passes m.  Then one sum in token order of the larger keys and of the
//           equal ones: token t's new place is the number of larger ones before it
//           and of the equal ones as far as they have room.  Weights move there, and
//           the list of the (sequence, KV head) gets the row's move, slot of t ->
//           slot of the place (or none, where it stays).
//   move    streams the rows of the lists, K and V, one CTA per (sequence, KV
//           head, plane, column slice).  In place a row's new place can be
//           another row's old one.  The list is in order and no place lies behind
//           its token, so a store can only hit rows that moves up to its own have
//           read: a CTA loads a round of moves, waits for all of its threads, and
//           stores them; the next round's loads are issued ahead of the stores.
//           Columns are independent of each other, so slices need no order between
//           them.  The order costs a long list its parts (one of 32767 tokens cut to
//           4096, 8 KV heads: 25.6 us in place, 20.4 into other blocks, both kernels, in
//           a graph) and many lists nothing (32 x 8 of 1000 to 5000 cut to 1024: 54.8
//           and 55.4).  Into other blocks no order is needed at all, and the rounds of a
//           list are dealt out to several CTAs.
//
// Bound: HBM, 8 d bytes a kept (token, KV head) that moves; for single sequences
// the latency of the select kernel's few CTAs.
#include <algorithm>
#include <mutex>

#include "common.cuh"
#include "internal.h"

namespace pa {
namespace {

constexpr int kSelThreads = 512;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kSelItems = 4;  // consecutive tokens of a thread in a chunk
constexpr int kChunk = kSelThreads * kSelItems;
constexpr int kDigits = 2048;
constexpr int kMoveThreads = 256;
constexpr int kMoveUnroll = 4;
constexpr int kMaxSeqs = 4096;
constexpr int kMaxCluster = 8;
// Bytes of rows that the select kernel asks L2 for at its end, while HBM is idle (256
// lists of 1024 tokens, d = 128: 56.0 us without, 54.1 with 16 MB, 53.8 with 32, 55.3 with
// 64, 57.9 with all 128 MB, which push each other out).
constexpr int64_t kAheadBytes = 32 << 20;

struct EvictArgs {
    const int32_t *block_tables;
    const int32_t *context_lens;
    const float *weights;
    float *weights_out;
    const int32_t *out_tables;
    int32_t *out_lens;
    int32_t *moved;  // [B][Hk] length of each list, ~length where some rows stay in their blocks
    int32_t *kept;   // [B] new lengths, -1: sequence left out
    int2 *moves;     // [B][Hk][cap] {from, to} slots
    __half *kplane;
    __half *vplane;
    int32_t *status;
    int64_t stride;  // floats between rows of weights
    int B, Hk, maxb, out_maxb, budget, sinks, recent, cap, num_blocks, d;
    int ahead;  // rows of each list asked for ahead
};

// A key that orders like the weight: NaN below everything, -0 equal to +0.
__device__ __forceinline__ uint32_t key_of(float w) {
    if (w != w) return 0u;
    const uint32_t b = __float_as_uint(w + 0.f);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}

// Inclusive sum over a warp's lanes.
template <typename T>
__device__ __forceinline__ T warp_sums(T x, int lane) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const T y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    return x;
}

// Larger keys in the low half, equal ones in the high half (both fit: a list has at
// most INT32_MAX tokens).
using Counts = unsigned long long;

// The cluster's barrier (of all threads; orders shared and global memory within the
// cluster), this CTA's place in it, and a word of another CTA's shared memory.
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::
                     : "memory");
}
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ int ld_cluster(const int *p, uint32_t rank) {
    uint32_t at;
    int v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_u32(p)), "r"(rank));
    asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
    return v;
}

// (two words, 8-byte aligned)
__device__ __forceinline__ int2 ld_cluster2(const int *p, uint32_t rank) {
    uint32_t at;
    int2 v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_u32(p)), "r"(rank));
    asm volatile("ld.shared::cluster.v2.s32 {%0, %1}, [%2];"
                 : "=r"(v.x), "=r"(v.y)
                 : "r"(at)
                 : "memory");
    return v;
}

// C chunks of tokens a CTA stay in registers.  `size` CTAs (a cluster) work on a
// list, each on `slice` tokens of it; with one CTA the last chunks may go on in
// memory.
template <int C>
__global__ void __launch_bounds__(kSelThreads, C > 4 ? 1 : 2)
    evict_select_kernel(const EvictArgs a, int size) {
    griddep_launch_dependents();
    griddep_wait();
    __shared__ __align__(16) int hist[3][kDigits];
    __shared__ Counts sums[C * kSelWarps];
    __shared__ __align__(8) int groups[3][kDigits / 32];  // sums of 32 digits, from the top
    __shared__ int found[3];
    __shared__ __align__(8) int mine_of[2];
    const int h = blockIdx.x / size, s = blockIdx.y;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int rank = size > 1 ? (int)cluster_rank() : 0;
    const int64_t pair = (int64_t)s * a.Hk + h;
    const int n = a.context_lens[s];
    const int k = min(n, a.budget);
    const bool ok = n >= 0 && n <= a.maxb * kBlockSize && n <= a.stride &&
                    (int64_t)k <= (int64_t)a.out_maxb * kBlockSize;
    if (tid == 0 && h == 0 && rank == 0) a.kept[s] = ok ? k : -1;
    if (!ok) {
        if (tid == 0 && rank == 0) {
            if (h == 0) report(a.status, PA_DEV_BAD_LENGTH);
            a.moved[pair] = 0;
        }
        return;
    }
    const float *w = a.weights + pair * a.stride;
    float *w_out = a.weights_out + pair * a.stride;
    const int32_t *row = a.block_tables + (int64_t)s * a.maxb;
    const int32_t *out_row = a.out_tables + (int64_t)s * a.out_maxb;
    int2 *list = a.moves + pair * a.cap;
    // this CTA's tokens: first .. last - 1
    const unsigned slice = size > 1 ? ((n + size - 1) / size + 3) & ~3u : (unsigned)n;
    const unsigned first = min((unsigned)n, rank * slice), last = min((unsigned)n, first + slice);

    // A thread's tokens of the chunk that begins at c0.
    const bool wide = a.stride % 4 == 0 && aligned16(a.weights);
    auto load = [&](unsigned c0, float (&x)[kSelItems]) {
        const unsigned t = c0 + tid * kSelItems;
        if (wide && t + kSelItems <= last) {
            const float4 v = *reinterpret_cast<const float4 *>(w + t);
            x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
        } else {
#pragma unroll
            for (int j = 0; j < kSelItems; ++j) x[j] = t + j < last ? w[t + j] : 0.f;
        }
    };
    float x[C][kSelItems];
#pragma unroll
    for (int c = 0; c < C; ++c) load(first + c * kChunk, x[c]);
    for (int i = tid; i < 3 * kDigits; i += kSelThreads) (&hist[0][0])[i] = 0;
    // (does any kept row's block stand in both tables?)
    int same = 0;
    for (int j = tid; j < (k + kBlockSize - 1) / kBlockSize; j += kSelThreads)
        same |= row[j] == out_row[j];
    same = __syncthreads_or(same);

    // ---- the m-th largest key of tokens [lo, hi), and how many equal to it to keep
    const bool all = n <= a.budget;
    const unsigned lo = max(first, all ? 0 : a.sinks), hi = min(last, all ? 0 : n - a.recent);
    uint32_t limit = 0xffffffffu;  // (no key is that large)
    int equal = 0;
    if (!all && k > a.sinks + a.recent) {
        int want = k - a.sinks - a.recent;  // of more than that many tokens
        uint32_t mask = 0;
        limit = 0;
#pragma unroll 1
        for (int d = 0; d < 3; ++d) {
            const int shift = d == 0 ? 21 : d == 1 ? 10 : 0;
            const uint32_t digit = d == 2 ? 1023 : 2047;
            auto count = [&](unsigned c0, const float (&y)[kSelItems]) {
#pragma unroll
                for (int j = 0; j < kSelItems; ++j) {
                    const unsigned t = c0 + tid * kSelItems + j;
                    const uint32_t key = key_of(y[j]);
                    if (t >= lo && t < hi && (key & mask) == limit)
                        atomicAdd(&hist[d][(key >> shift) & digit], 1);
                }
            };
#pragma unroll
            for (int c = 0; c < C; ++c)
                if (first + c * kChunk < hi) count(first + c * kChunk, x[c]);
            for (unsigned c0 = first + C * kChunk; c0 < hi; c0 += kChunk) {
                float y[kSelItems];
                load(c0, y);
                count(c0, y);
            }
            // thread i holds four digits, from the top: 2047 - 4 i and down
            static_assert(kDigits == 4 * kSelThreads, "a vector of four");
            __syncthreads();
            const int4 own = *reinterpret_cast<const int4 *>(&hist[d][kDigits - 4 * (tid + 1)]);
            int sum = own.x + own.y + own.z + own.w;
#pragma unroll
            for (int o = 1; o < 8; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            if ((tid & 7) == 0) groups[d][tid / 8] = sum;
            if (size > 1)
                cluster_sync();
            else
                __syncthreads();
            // One warp looks for the group of 32 digits, then for the digit (the whole
            // histograms of a cluster of eight, read by all, took 3 us a digit).
            if (warp == 0) {
                int2 g[kMaxCluster];
#pragma unroll
                for (int q = 0; q < kMaxCluster; ++q)
                    g[q] = q < size ? ld_cluster2(&groups[d][2 * lane], q) : make_int2(0, 0);
                int a0 = 0, a1 = 0;
#pragma unroll
                for (int q = 0; q < kMaxCluster; ++q) a0 += g[q].x, a1 += g[q].y;
                int before = warp_sums(a0 + a1, lane) - a0 - a1;
                int at = -1;  // this lane's group, if it is the one
                if (before < want && want <= before + a0) at = 2 * lane;
                before += at < 0 ? a0 : 0;
                if (at < 0 && before < want && want <= before + a1) at = 2 * lane + 1;
                const int who = __ffs(__ballot_sync(0xffffffffu, at >= 0)) - 1;
                at = __shfl_sync(0xffffffffu, at, who);
                before = __shfl_sync(0xffffffffu, before, who);
                const int mine = kDigits - 1 - 32 * at - lane;
                int c[kMaxCluster], cnt = 0;
#pragma unroll
                for (int q = 0; q < kMaxCluster; ++q)
                    c[q] = q < size ? ld_cluster(&hist[d][mine], q) : 0;
#pragma unroll
                for (int q = 0; q < kMaxCluster; ++q) cnt += c[q];
                before += warp_sums(cnt, lane) - cnt;
                if (before < want && want <= before + cnt) {
                    found[0] = mine;
                    found[1] = want - before;
                    found[2] = cnt;
                }
            }
            __syncthreads();
            limit |= (uint32_t)found[0] << shift;
            mask |= digit << shift;
            equal = want = found[1];
            if (found[2] == want && limit > 0) {
                // all keys that agree so far are kept (one key, more often than not):
                // those are the keys above the largest one below them
                --limit;
                equal = 0;
                break;
            }
            // (barriers of the next digit come before found changes)
        }
    }

    // ---- new places
    auto counts = [&](unsigned c0, const float (&y)[kSelItems]) -> Counts {
        Counts v = 0;
#pragma unroll
        for (int j = 0; j < kSelItems; ++j) {
            const unsigned t = c0 + tid * kSelItems + j;
            const uint32_t key = key_of(y[j]);
            const bool other = t >= lo && t < hi;
            if (t < last) v += other && key == limit ? (Counts)1 << 32
                               : all || !other || key > limit ? 1 : 0;
        }
        return v;
    };
    // The chunk's kept tokens, `v` counted before this thread's.
    auto place = [&](unsigned c0, const float (&y)[kSelItems], Counts v) {
        unsigned larger = (unsigned)v;
        int ties = (int)(v >> 32);
#pragma unroll
        for (int j = 0; j < kSelItems; ++j) {
            const unsigned t = c0 + tid * kSelItems + j;
            if (t >= last) break;
            const uint32_t key = key_of(y[j]);
            const bool other = t >= lo && t < hi;
            const bool tie = other && key == limit;
            const unsigned i = larger + min(ties, equal);
            const bool keep = tie ? ties < equal : all || !other || key > limit;
            ties += tie;
            larger += keep && !tie;
            if (!keep) continue;
            w_out[i] = y[j];
            list[i].x = (int)t;
        }
    };
    Counts v[C];
#pragma unroll
    for (int c = 0; c < C; ++c) {
        v[c] = 0;
        if (lane == 31) sums[c * kSelWarps + warp] = 0;
        if (first + c * kChunk >= last) continue;
        const Counts mine = counts(first + c * kChunk, x[c]), upto = warp_sums(mine, lane);
        if (lane == 31) sums[c * kSelWarps + warp] = upto;
        v[c] = upto - mine;
    }
    __syncthreads();
    if (warp == 0) {
        Counts carry = 0;
        for (int i0 = 0; i0 < C * kSelWarps; i0 += 32) {
            const Counts mine = i0 + lane < C * kSelWarps ? sums[i0 + lane] : 0;
            const Counts upto = warp_sums(mine, lane);
            if (i0 + lane < C * kSelWarps) sums[i0 + lane] = carry + upto - mine;
            carry += __shfl_sync(0xffffffffu, upto, 31);
        }
        if (lane == 0) mine_of[0] = (int)(unsigned)carry, mine_of[1] = (int)(carry >> 32);
    }
    // (behind this barrier every weight in registers has been read: its places in
    // `weights` may be written)
    Counts base = 0;
    if (size > 1) {
        cluster_sync();
        const int2 c = lane < rank ? ld_cluster2(mine_of, lane) : make_int2(0, 0);
        base = (Counts)(unsigned)c.x | (Counts)(unsigned)c.y << 32;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) base += __shfl_xor_sync(0xffffffffu, base, o);
    } else {
        __syncthreads();
    }
    if (tid == 0 && rank == 0) a.moved[pair] = same ? ~k : k;
#pragma unroll
    for (int c = 0; c < C; ++c)
        if (first + c * kChunk < last)
            place(first + c * kChunk, x[c], base + sums[c * kSelWarps + warp] + v[c]);
    Counts total = (Counts)(unsigned)mine_of[0] | (Counts)(unsigned)mine_of[1] << 32;
    for (unsigned c0 = first + C * kChunk; c0 < last; c0 += kChunk) {  // (one CTA)
        float y[kSelItems];
        load(c0, y);
        const Counts mine = counts(c0, y), upto = warp_sums(mine, lane);
        __syncthreads();  // sums of the chunk before are read
        if (lane == 31) sums[warp] = upto;
        __syncthreads();  // (and this chunk's weights)
        Counts before = total + upto - mine;
        for (int u = 0; u < kSelWarps; ++u) {
            before += u < warp ? sums[u] : 0;
            total += sums[u];
        }
        place(c0, y, before);
    }
    const unsigned me = rank * kSelThreads + tid, everyone = size * kSelThreads;
    for (unsigned t = k + me; t < (unsigned)n; t += everyone) w_out[t] = 0.f;

    // ---- tokens to slots, apart from the places: so the block ids' loads do not wait
    // for each other
    if (size > 1)
        cluster_sync();  // (and the last reads of another CTA's shared memory are done)
    else
        __syncthreads();
#pragma unroll 4
    for (unsigned i = me; i < (unsigned)k; i += everyone) {
        const int t = list[i].x;
        const int src = row[t / kBlockSize], dst = out_row[i / kBlockSize];
        int2 mv = make_int2(-1, -1);
        if (src < 0 || src >= a.num_blocks || dst < 0 || dst >= a.num_blocks) {
            report(a.status, PA_DEV_BAD_BLOCK);
        } else {
            const int from = src * kBlockSize + t % kBlockSize;
            const int to = dst * kBlockSize + (int)(i % kBlockSize);
            if (from != to) {
                mv = make_int2(from, to);
                if (i < (unsigned)a.ahead) {
                    const int64_t at = ((int64_t)from * a.Hk + h) * a.d;
                    for (int c = 0; c < a.d; c += 64) {  // (128 bytes)
                        prefetch_l2(a.kplane + at + c);
                        prefetch_l2(a.vplane + at + c);
                    }
                }
            }
        }
        list[i] = mv;
    }
}

template <int D>
__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(const EvictArgs a, int slices,
                                                                  int parts) {
    // (No launch_dependents: this kernel writes the new lengths, and the decode calls
    // read their lengths ahead of their wait for the kernel before.)
    griddep_wait();
    const int h = blockIdx.y, s = blockIdx.z / parts, part = blockIdx.z % parts, tid = threadIdx.x;
    const int64_t pair = (int64_t)s * a.Hk + h;
    if (blockIdx.x == 0 && h == 0 && part == 0 && tid == 0 && a.kept[s] >= 0) {
        a.out_lens[s] = a.kept[s];
        __threadfence();  // (seen by kernels that start when this one's CTAs are done)
    }
    const int moved = a.moved[pair];
    if (moved < 0 && part > 0) return;  // in place: one CTA, in order
    const unsigned n = moved < 0 ? ~moved : moved;
    __half *plane = blockIdx.x & 1 ? a.vplane : a.kplane;
    const int width = D / 8 / slices;  // 16-byte pieces of a slice
    const int rows = kMoveThreads / width, r = tid / width;
    uint4 *base = reinterpret_cast<uint4 *>(plane) + (blockIdx.x >> 1) * width + tid % width;
    const int2 *list = a.moves + pair * a.cap;
    const unsigned round = rows * kMoveUnroll, step = moved < 0 ? round : parts * round;

    auto at = [&](int slot) { return base + ((int64_t)slot * a.Hk + h) * (D / 8); };
    int2 mv[kMoveUnroll];  // of the round after the one in x
    uint4 x[kMoveUnroll];
    int to[kMoveUnroll];
    auto moves = [&](unsigned i0) {
#pragma unroll
        for (int j = 0; j < kMoveUnroll; ++j) {
            const unsigned i = i0 + j * rows + r;
            mv[j] = i < n ? list[i] : make_int2(-1, -1);
        }
    };
    auto load = [&]() {
#pragma unroll
        for (int j = 0; j < kMoveUnroll; ++j) {
            to[j] = mv[j].y;
            if (mv[j].x >= 0) x[j] = *at(mv[j].x);
        }
    };
    unsigned i0 = part * round;
    moves(i0);
    load();
    moves(i0 + step);
    for (; i0 < n; i0 += step) {
        uint4 y[kMoveUnroll];
        int yt[kMoveUnroll];
#pragma unroll
        for (int j = 0; j < kMoveUnroll; ++j) {
            y[j] = x[j];
            yt[j] = to[j];
        }
        __syncthreads();  // this round's rows are read
        load();
        moves(i0 + 2 * step);
#pragma unroll
        for (int j = 0; j < kMoveUnroll; ++j)
            if (yt[j] >= 0) *at(yt[j]) = y[j];
    }
}

template <int C>
void launch_select(const EvictArgs &a, int size, cudaStream_t st) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(a.Hk * size, a.B);
    cfg.blockDim = dim3(kSelThreads);
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = size;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = size > 1 ? 2 : 1;
    cudaLaunchKernelEx(&cfg, evict_select_kernel<C>, a, size);  // (errors: launch_status)
}

size_t header_bytes(int B, int Hk) {
    return ((size_t)B * Hk * 4 + (size_t)B * 4 + 255) & ~(size_t)255;
}

}  // namespace
}  // namespace pa

using namespace pa;

extern "C" size_t pa_kv_evict_workspace_bytes(int num_seqs, int n_kv_heads, int budget) {
    if (num_seqs <= 0 || n_kv_heads <= 0 || budget <= 0) return 0;
    const unsigned __int128 n = (unsigned __int128)num_seqs * n_kv_heads * 4 +
                                (unsigned __int128)num_seqs * 4 + 255 +
                                (unsigned __int128)num_seqs * n_kv_heads * budget * 8;
    if (n > SIZE_MAX) return 0;
    return header_bytes(num_seqs, n_kv_heads) + (size_t)num_seqs * n_kv_heads * budget * 8;
}

extern "C" int pa_kv_evict(const pa_cache_t *cache, int layer, const int32_t *block_tables,
                           int max_blocks_per_seq, const int32_t *context_lens, int num_seqs,
                           int n_kv_heads, int head_dim, const float *weights, float *weights_out,
                           int64_t weights_stride, int budget, int sinks, int recent,
                           const int32_t *out_block_tables, int out_max_blocks_per_seq,
                           int32_t *out_context_lens, void *workspace, size_t workspace_bytes,
                           int32_t *dev_status, pa_stream_t stream) {
    if (num_seqs < 0 || n_kv_heads <= 0 || max_blocks_per_seq <= 0 ||
        max_blocks_per_seq > kMaxBlocksPerSeq || out_max_blocks_per_seq <= 0 ||
        out_max_blocks_per_seq > kMaxBlocksPerSeq || budget <= 0 || sinks < 0 || recent < 0 ||
        (int64_t)sinks + recent > budget || weights_stride <= 0)
        return PA_ERR_INVALID;
    if (head_dim != 64 && head_dim != 128) return PA_ERR_UNSUPPORTED;
    if (num_seqs > kMaxSeqs || n_kv_heads > 65535) return PA_ERR_UNSUPPORTED;
    if (!cache_ok(cache, layer, n_kv_heads, head_dim)) return PA_ERR_INVALID;
    if (num_seqs == 0) return PA_OK;
    if (!block_tables || !context_lens || !weights || !weights_out || !out_block_tables ||
        !out_context_lens || !workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u))
        return PA_ERR_INVALID;
    const unsigned __int128 rows = (unsigned __int128)num_seqs * n_kv_heads * weights_stride * 4;
    if (rows > SIZE_MAX || (weights_out != weights && ranges_overlap(weights, (uint64_t)rows,
                                                                     weights_out, (uint64_t)rows)))
        return PA_ERR_INVALID;
    const int cap = std::min(budget, max_blocks_per_seq * kBlockSize);
    const size_t need = pa_kv_evict_workspace_bytes(num_seqs, n_kv_heads, cap);
    if (need == 0 || workspace_bytes < need) return PA_ERR_WORKSPACE;

    EvictArgs a;
    a.block_tables = block_tables;
    a.context_lens = context_lens;
    a.weights = weights;
    a.weights_out = weights_out;
    a.out_tables = out_block_tables;
    a.out_lens = out_context_lens;
    a.moved = static_cast<int32_t *>(workspace);
    a.kept = a.moved + (int64_t)num_seqs * n_kv_heads;
    a.moves = reinterpret_cast<int2 *>(static_cast<uint8_t *>(workspace) +
                                       header_bytes(num_seqs, n_kv_heads));
    a.kplane = cache_plane(cache, 0, layer);
    a.vplane = cache_plane(cache, 1, layer);
    a.status = dev_status;
    a.stride = weights_stride;
    a.B = num_seqs;
    a.Hk = n_kv_heads;
    a.maxb = max_blocks_per_seq;
    a.out_maxb = out_max_blocks_per_seq;
    a.budget = budget;
    a.sinks = sinks;
    a.recent = recent;
    a.cap = cap;
    a.num_blocks = cache->num_blocks;
    a.d = head_dim;
    a.ahead = (int)std::min<int64_t>(
        cap, kAheadBytes / ((int64_t)num_seqs * n_kv_heads * 4 * head_dim));
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    // As many CTAs a list as find an SM each, of a chunk of tokens at least, and
    // registers for the tokens that a table row can hold, as far as they go.  (The
    // lengths are on the device.  One sequence of 32767 tokens cut to 4096, 8 KV heads,
    // in a graph: 20.4 us with a table of 32768 tokens, 26.6 of 131072 to 262112, 51.6
    // past that; 32 of 1000 to 5000 cut to 1024: 55 of 5008, 72 of 8192 and more.)
    const int longest = max_blocks_per_seq * kBlockSize;
    int size = 1;
    while (size < kMaxCluster && size * kChunk < longest &&
           (int64_t)2 * size * n_kv_heads * num_seqs <= sm_count())
        size *= 2;
    if (longest / size > 16 * kChunk - 4) size = 1;  // (a cluster keeps all in registers)
    const int64_t each = ((int64_t)longest + size - 1) / size + 3;
    if (each <= kChunk)
        launch_select<1>(a, size, st);
    else if (each <= 4 * kChunk)
        launch_select<4>(a, size, st);
    else
        launch_select<16>(a, size, st);
    const int rc = launch_status();
    if (rc != PA_OK) return rc;
    // Whole rows where that already gives several CTAs to every SM, else slices down
    // to 64 bytes (two DRAM sectors), and parts of the lists.
    const int64_t want = 2 * (int64_t)sm_count(), lists = 2 * (int64_t)n_kv_heads * num_seqs;
    int slices = 1;
    while (slices < head_dim / 32 && slices * lists < want) slices *= 2;
    const int parts = (int)std::min<int64_t>(8, std::max<int64_t>(1, want / (slices * lists)));
    const dim3 grid(2 * slices, n_kv_heads, num_seqs * parts);
    if (head_dim == 128)
        launch_dependent(evict_move_kernel<128>, grid, dim3(kMoveThreads), 0, st, a, slices, parts);
    else
        launch_dependent(evict_move_kernel<64>, grid, dim3(kMoveThreads), 0, st, a, slices, parts);
    return launch_status();
}
