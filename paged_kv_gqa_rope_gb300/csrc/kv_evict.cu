// Eviction from the paged fp16 cache by accumulated attention weight
// (pa_kv_evict; the weights are pa_decode_weights').
//
// Of a sequence's n tokens each KV head keeps k = min(n, budget): the first
// `sinks`, the last `recent` and, of the others, the m = k - sinks - recent of
// the largest weight, of equal ones the first.  Two kernels:
//
//   select  one CTA per (sequence, KV head).  The m-th largest weight among the
//           others is found digit by digit (11 + 11 + 10 bits of a key that
//           orders like the weights): a histogram of the digit over the keys
//           that agree on the digits before it, and the digit at which the count
//           from the top passes m.  Then one pass in token order: token t is kept
//           if its key is larger, or equal and among the first of the equal ones
//           that still have room; the tokens kept before it give its new place i.
//           Weights move there, and the row's move (slot of t -> slot of i) goes
//           into the (sequence, KV head)'s list unless it stays where it is.
//   move    streams the rows of the lists, K and V, one CTA per (sequence, KV
//           head, plane, column slice).  In place a row's new place can be
//           another row's old one.  The list is in order and i <= t, so a store
//           can only hit rows that moves up to its own have read: a CTA loads a
//           round of moves, waits for all of its threads, and stores them; the
//           next round's loads are issued ahead of the stores.  Columns are
//           independent of each other, so slices need no order between them.
//
// Bound: HBM, 8 d bytes a kept (token, KV head) that moves; for single sequences
// the select kernel's passes over few CTAs.
#include <algorithm>
#include <mutex>

#include "common.cuh"
#include "internal.h"

namespace pa {
namespace {

constexpr int kSelThreads = 1024;
constexpr int kSelItems = 4;  // consecutive tokens of a thread in the ordered pass
constexpr int kDigits = 2048;
constexpr int kMoveThreads = 256;
constexpr int kMoveUnroll = 4;
constexpr int kMaxSeqs = 4096;

struct EvictArgs {
    const int32_t *block_tables;
    const int32_t *context_lens;
    const float *weights;
    float *weights_out;
    const int32_t *out_tables;
    int32_t *out_lens;
    int32_t *moved;  // [B][Hk] moves of each list
    int32_t *kept;   // [B] new lengths, -1: sequence left out
    int2 *moves;     // [B][Hk][cap] {from, to} slots
    __half *kplane;
    __half *vplane;
    int32_t *status;
    int64_t stride;  // floats between rows of weights
    int B, Hk, maxb, out_maxb, budget, sinks, recent, cap, num_blocks;
};

// A key that orders like the weight: NaN below everything, -0 equal to +0.
__device__ __forceinline__ uint32_t key_of(float w) {
    if (w != w) return 0u;
    const uint32_t b = __float_as_uint(w + 0.f);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}

// Exclusive sum of v over the CTA's threads and its total (all threads call).
__device__ __forceinline__ int block_scan(int v, int *sm, int &total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    __syncthreads();  // sm of an earlier call is read
    if (lane == 31) sm[warp] = x;
    __syncthreads();
    if (warp == 0) {
        int y = sm[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int z = __shfl_up_sync(0xffffffffu, y, o);
            if (lane >= o) y += z;
        }
        sm[lane] = y;
    }
    __syncthreads();
    total = sm[kSelThreads / 32 - 1];
    return x - v + (warp ? sm[warp - 1] : 0);
}

__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(const EvictArgs a) {
    griddep_launch_dependents();
    griddep_wait();
    __shared__ int hist[kDigits];
    __shared__ int scan[32];
    __shared__ int found[2];
    const int h = blockIdx.x, s = blockIdx.y, tid = threadIdx.x;
    const int64_t pair = (int64_t)s * a.Hk + h;
    const int n = a.context_lens[s];
    const int k = min(n, a.budget);
    const bool ok = n >= 0 && n <= a.maxb * kBlockSize && n <= a.stride &&
                    (int64_t)k <= (int64_t)a.out_maxb * kBlockSize;
    if (tid == 0) {
        if (h == 0) a.kept[s] = ok ? k : -1;
        if (!ok) {
            if (h == 0) report(a.status, PA_DEV_BAD_LENGTH);
            a.moved[pair] = 0;
        }
    }
    if (!ok) return;
    const float *w = a.weights + pair * a.stride;
    float *w_out = a.weights_out + pair * a.stride;

    // ---- the m-th largest key of tokens [lo, hi), and how many equal to it to keep
    const bool all = n <= a.budget;
    const int lo = all ? 0 : a.sinks, hi = all ? 0 : n - a.recent;
    uint32_t limit = 0;
    int equal = 0;
    if (!all) {
        int want = k - a.sinks - a.recent;  // of the hi - lo > want tokens
        uint32_t mask = 0;
        equal = want;
        for (int shift = 21; want > 0; shift = shift == 21 ? 10 : 0) {
            const int bits = shift == 0 ? 10 : 11;
            for (int i = tid; i < kDigits; i += kSelThreads) hist[i] = 0;
            __syncthreads();
            for (unsigned t = lo + tid; t < (unsigned)hi; t += kSelThreads) {
                const uint32_t key = key_of(w[t]);
                if ((key & mask) == limit) atomicAdd(&hist[(key >> shift) & ((1u << bits) - 1)], 1);
            }
            __syncthreads();
            // thread i holds the digits 2047 - 2i and 2046 - 2i: counts from the top
            const int d0 = kDigits - 1 - 2 * tid;
            const int c0 = hist[d0], c1 = hist[d0 - 1];
            int total;
            const int before = block_scan(c0 + c1, scan, total);
            if (before < want && want <= before + c0) {
                found[0] = d0;
                found[1] = want - before;
            } else if (before + c0 < want && want <= before + c0 + c1) {
                found[0] = d0 - 1;
                found[1] = want - before - c0;
            }
            __syncthreads();
            limit |= (uint32_t)found[0] << shift;
            mask |= ((1u << bits) - 1) << shift;
            equal = want = found[1];
            __syncthreads();
            if (shift == 0) break;
        }
        if (k == a.sinks + a.recent) limit = 0xffffffffu;  // (no key is that large)
    }

    // ---- the ordered pass
    const int32_t *row = a.block_tables + (int64_t)s * a.maxb;
    const int32_t *out_row = a.out_tables + (int64_t)s * a.out_maxb;
    int2 *list = a.moves + pair * a.cap;
    int places = 0, ties = 0, count = 0;  // so far: kept, equal ones met, moves listed
    for (unsigned t0 = 0; t0 < (unsigned)n; t0 += kSelThreads * kSelItems) {
        float x[kSelItems];
        int keep[kSelItems], eq[kSelItems];
        int nk = 0, ne = 0;
#pragma unroll
        for (int j = 0; j < kSelItems; ++j) {
            const unsigned t = t0 + tid * kSelItems + j;
            x[j] = t < (unsigned)n ? w[t] : 0.f;
            const uint32_t key = key_of(x[j]);
            const bool other = t >= (unsigned)lo && t < (unsigned)hi;
            eq[j] = other && key == limit;
            keep[j] = t < (unsigned)n && (all || !other || key > limit);
            nk += keep[j];
            ne += eq[j];
        }
        // equal ones first: which of them still have room (both counts in one sum)
        int total;
        const int base = block_scan(ne, scan, total);
        int e = ties + base;
        ties += total;
#pragma unroll
        for (int j = 0; j < kSelItems; ++j) {
            if (eq[j] && e < equal) {
                keep[j] = 1;
                ++nk;
            }
            e += eq[j];
        }
        int i = places + block_scan(nk, scan, total);
        places += total;
        int2 mv[kSelItems];
        int nm = 0;
#pragma unroll
        for (int j = 0; j < kSelItems; ++j) {
            const unsigned t = t0 + tid * kSelItems + j;
            mv[j] = make_int2(-1, -1);
            if (!keep[j]) continue;
            // (every weight of this round has been read: the sums above wait for all)
            w_out[i] = x[j];
            const int src = row[t / kBlockSize], dst = out_row[i / kBlockSize];
            if (src < 0 || src >= a.num_blocks || dst < 0 || dst >= a.num_blocks) {
                report(a.status, PA_DEV_BAD_BLOCK);
            } else {
                const int from = src * kBlockSize + (int)(t % kBlockSize);
                const int to = dst * kBlockSize + i % kBlockSize;
                if (from != to) {
                    mv[j] = make_int2(from, to);
                    ++nm;
                }
            }
            ++i;
        }
        int c = count + block_scan(nm, scan, total);
        count += total;
#pragma unroll
        for (int j = 0; j < kSelItems; ++j)
            if (mv[j].x >= 0) list[c++] = mv[j];
    }
    for (unsigned t = k + tid; t < (unsigned)n; t += kSelThreads) w_out[t] = 0.f;
    if (tid == 0) a.moved[pair] = count;
}

template <int D>
__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(const EvictArgs a, int slices) {
    // (No launch_dependents: this kernel writes the new lengths, and pa_decode
    // reads its lengths ahead of its wait for the kernel before.)
    griddep_wait();
    const int h = blockIdx.y, s = blockIdx.z, tid = threadIdx.x;
    const int64_t pair = (int64_t)s * a.Hk + h;
    if (blockIdx.x == 0 && h == 0 && tid == 0 && a.kept[s] >= 0) a.out_lens[s] = a.kept[s];
    const unsigned n = a.moved[pair];
    __half *plane = blockIdx.x & 1 ? a.vplane : a.kplane;
    const int width = D / 8 / slices;  // 16-byte pieces of a slice
    const int rows = kMoveThreads / width, r = tid / width;
    uint4 *base = reinterpret_cast<uint4 *>(plane) + (blockIdx.x >> 1) * width + tid % width;
    const int2 *list = a.moves + pair * a.cap;
    const int round = rows * kMoveUnroll;

    auto at = [&](int slot) { return base + ((int64_t)slot * a.Hk + h) * (D / 8); };
    uint4 x[kMoveUnroll];
    int to[kMoveUnroll];
    auto load = [&](unsigned i0) {
#pragma unroll
        for (int j = 0; j < kMoveUnroll; ++j) {
            const unsigned i = i0 + j * rows + r;
            to[j] = -1;
            if (i < n) {
                const int2 mv = list[i];
                to[j] = mv.y;
                x[j] = *at(mv.x);
            }
        }
    };
    load(0);
    for (unsigned i0 = 0; i0 < n; i0 += round) {
        uint4 y[kMoveUnroll];
        int yt[kMoveUnroll];
#pragma unroll
        for (int j = 0; j < kMoveUnroll; ++j) {
            y[j] = x[j];
            yt[j] = to[j];
        }
        __syncthreads();  // this round's rows are read
        load(i0 + round);
#pragma unroll
        for (int j = 0; j < kMoveUnroll; ++j)
            if (yt[j] >= 0) *at(yt[j]) = y[j];
    }
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
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    launch_dependent(evict_select_kernel, dim3(n_kv_heads, num_seqs), dim3(kSelThreads), 0, st, a);
    const int rc = launch_status();
    if (rc != PA_OK) return rc;
    // Whole rows where that already gives a CTA to every SM, else slices down to
    // 64 bytes (two DRAM sectors).
    int slices = 1;
    while (slices < head_dim / 32 && (int64_t)2 * slices * n_kv_heads * num_seqs < 4 * sm_count())
        slices *= 2;
    const dim3 grid(2 * slices, n_kv_heads, num_seqs);
    if (head_dim == 128)
        launch_dependent(evict_move_kernel<128>, grid, dim3(kMoveThreads), 0, st, a, slices);
    else
        launch_dependent(evict_move_kernel<64>, grid, dim3(kMoveThreads), 0, st, a, slices);
    return launch_status();
}
