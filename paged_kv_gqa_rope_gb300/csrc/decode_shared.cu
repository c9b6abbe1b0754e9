// Decode of sequences that share a prefix (pa_decode_shared).
#include <algorithm>

#include "decode_modes.cuh"

namespace pa {
namespace {

struct SharedArgs {
    const __half *q;
    const __half *kplane;
    const __half *vplane;
    const int32_t *block_tables;
    const int32_t *context_lens;
    __half *out;
    DecodeTails tl;
    float *first;  // [B][H][D + 4]: records of units' first pieces
    float *more;   // [G][256][D + 4]: of the piece with which a CTA's range begins inside a unit
    int32_t *status;
    float scale_log2;
    int B, H, Hk, g, maxb, num_blocks, G;
};

constexpr int kPrefixThreads = 1024;

// One piece after another of the CTA's range: four threads a query row.
template <int D>
__global__ void __launch_bounds__(kPrefixThreads) prefix_kernel(const SharedArgs a) {
    griddep_launch_dependents();
    griddep_wait();
    constexpr int kPart = D / 4, kRec = D + 4;
    __shared__ __align__(16) __half ks[kBlockSize][D];
    __shared__ __align__(16) __half vs[kBlockSize][D];
    const int64_t total = a.tl.head->total;
    const int G = plan_ctas(total, a.G);
    if ((int)blockIdx.x >= G) return;
    const int64_t end = plan_cut(total, blockIdx.x + 1, G);
    const int tid = threadIdx.x, local = tid >> 2, part = tid & 3;
    const int mpt = kPrefixTile / a.g, tile = local / kPrefixTile, in = local % kPrefixTile;
    int r = 0;
    for (int64_t pos = plan_cut(total, blockIdx.x, G); pos < end;) {
        PlanGroup p = a.tl.plan[r];
        while (pos >= p.start + (int64_t)p.tiles * p.units * a.Hk) p = a.tl.plan[++r];
        const int64_t off = pos - p.start;
        const int unit = (int)(off / p.tiles), t0 = (int)(off % p.tiles);
        const int nt = (int)min((int64_t)(p.tiles - t0), end - pos);
        const int kvh = unit / p.units, u = unit % p.units;
        const int member = u * 2 * mpt + tile * mpt + in / a.g;
        const bool live = in < mpt * a.g && member < p.members;
        const int64_t row = (int64_t)(p.s0 + (live ? member : 0)) * a.H + kvh * a.g + in % a.g;
        float q[kPart], o[kPart], m = -INFINITY, l = 0.f;
        for (int i = 0; i < kPart; ++i) {
            q[i] = live ? __half2float(a.q[row * D + part * kPart + i]) * a.scale_log2 : 0.f;
            o[i] = 0.f;
        }
        for (int b = t0 * kTileBlocks; b < min((t0 + nt) * kTileBlocks, p.blocks); ++b) {
            const int blk = a.block_tables[(int64_t)p.lead * a.maxb + b];
            const bool ok = blk >= 0 && blk < a.num_blocks;
            if (!ok) {
                if (tid == 0) report(a.status, PA_DEV_BAD_BLOCK);
                continue;
            }
            __syncthreads();
            for (int i = tid; i < kBlockSize * D; i += kPrefixThreads) {
                const int64_t at = ((int64_t)(blk * kBlockSize + i / D) * a.Hk + kvh) * D + i % D;
                ks[i / D][i % D] = a.kplane[at];
                vs[i / D][i % D] = a.vplane[at];
            }
            __syncthreads();
            for (int t = 0; t < kBlockSize; ++t) {
                float x = 0.f;
                for (int i = 0; i < kPart; ++i) x += q[i] * __half2float(ks[t][part * kPart + i]);
                x += __shfl_xor_sync(0xffffffffu, x, 1);
                x += __shfl_xor_sync(0xffffffffu, x, 2);
                const float mn = fmaxf(m, x), f = ex2(m - mn), e = ex2(x - mn);
                m = mn;
                l = l * f + e;
                for (int i = 0; i < kPart; ++i)
                    o[i] = o[i] * f + e * __half2float(vs[t][part * kPart + i]);
            }
        }
        if (live) {
            float *rec = t0 == 0 ? a.first + row * kRec
                                 : a.more + ((int64_t)blockIdx.x * 2 * kPrefixTile + local) * kRec;
            for (int i = 0; i < kPart; ++i) rec[part * kPart + i] = o[i];
            if (part == 0) {
                rec[D] = m;
                rec[D + 1] = l;
            }
        }
        pos += nt;
    }
}

constexpr int kJoinThreads = 256;

// A warp per (sequence, Q head): joins the row's records.
template <int D>
__global__ void __launch_bounds__(kJoinThreads) join_kernel(const SharedArgs a) {
    griddep_wait();
    griddep_launch_dependents();
    constexpr int kRec = D + 4, kVec = D / 32;
    const int lane = threadIdx.x & 31;
    const int64_t row = (int64_t)blockIdx.x * (kJoinThreads / 32) + (threadIdx.x >> 5);
    if (row >= (int64_t)a.B * a.H) return;
    const int s = (int)(row / a.H), h = (int)(row % a.H);
    const int group = a.tl.seq_group[s];
    if (group == kLeftOut) return;
    int tail = a.context_lens[s], pieces = 0, c0 = 0, local = 0;
    if (group >= 0) {
        const PlanGroup p = a.tl.plan[group];
        const int64_t total = a.tl.head->total;
        const int G = plan_ctas(total, a.G);
        const int mpt = kPrefixTile / a.g, kvh = h / a.g, member = s - p.s0;
        const int u = member / (2 * mpt), in = member % (2 * mpt);
        const int64_t start = p.start + ((int64_t)kvh * p.units + u) * p.tiles;
        c0 = plan_cta(start, total, G);
        pieces = plan_cta(start + p.tiles - 1, total, G) - c0 + 1;
        local = in / mpt * kPrefixTile + in % mpt * a.g + h % a.g;
        tail -= p.blocks * kBlockSize;
    }
    // record 0: the tail's (if there is one), then the pieces'
    const int lead = tail > 0 ? 1 : 0, n = lead + pieces;
    auto rec = [&](int i) -> const float * {
        if (i < lead) return a.tl.rec + row * kRec;
        if (i == lead) return a.first + row * kRec;
        return a.more + ((int64_t)(c0 + i - lead) * 2 * kPrefixTile + local) * kRec;
    };
    float M = -INFINITY;
    for (int i = lane; i < n; i += 32) M = fmaxf(M, rec(i)[D]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    float L = 0.f, O[kVec];
#pragma unroll
    for (int v = 0; v < kVec; ++v) O[v] = 0.f;
    for (int i = 0; i < n; ++i) {
        const float *p = rec(i);
        const float f = p[D] == -INFINITY ? 0.f : ex2(p[D] - M);
        L = fmaf(f, p[D + 1], L);
#pragma unroll
        for (int v = 0; v < kVec; ++v) O[v] = fmaf(f, p[v * 32 + lane], O[v]);
    }
#pragma unroll
    for (int v = 0; v < kVec; ++v) a.out[row * D + v * 32 + lane] = __float2half_rn(L == 0.f ? 0.f : O[v] / L);
}

size_t up256(size_t n) { return (n + 255) & ~(size_t)255; }

constexpr int kMaxGroups = 4096;
constexpr int kMaxCtas = 160;  // (152 SMs)

size_t rows_bytes(int B, int H, int D) { return up256((size_t)B * H * (D + 4) * sizeof(float)); }

template <int D>
int launch_shared(const SharedArgs &a, cudaStream_t st) {
    launch_dependent(prefix_kernel<D>, dim3(a.G), dim3(kPrefixThreads), 0, st, a);
    const int rc = launch_status();
    if (rc != PA_OK) return rc;
    const int64_t rows = (int64_t)a.B * a.H, per = kJoinThreads / 32;
    launch_dependent(join_kernel<D>, dim3((unsigned)((rows + per - 1) / per)), dim3(kJoinThreads),
                     0, st, a);
    return launch_status();
}

}  // namespace
}  // namespace pa

using namespace pa;

extern "C" size_t pa_decode_shared_workspace_bytes(int num_seqs, int n_heads, int n_kv_heads,
                                                   int head_dim) {
    if (num_seqs <= 0 || n_heads <= 0 || n_kv_heads <= 0 || head_dim <= 0) return 0;
    return up256(mode_workspace_bytes(head_dim)) + 256 + up256((size_t)kMaxGroups * sizeof(PlanGroup)) +
           up256((size_t)num_seqs * 4) + 2 * rows_bytes(num_seqs, n_heads, head_dim) +
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
    if (num_groups > kMaxGroups || (int64_t)num_seqs * n_kv_heads > kModePairs)
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
    if ((int64_t)num_seqs * n_heads > INT32_MAX) return PA_ERR_UNSUPPORTED;

    uint8_t *at = static_cast<uint8_t *>(workspace);
    uint8_t *p = at + up256(mode_workspace_bytes(head_dim));
    SharedArgs a = {};
    a.tl.head = reinterpret_cast<PlanHead *>(p);
    p += 256;
    a.tl.plan = reinterpret_cast<PlanGroup *>(p);
    p += up256((size_t)kMaxGroups * sizeof(PlanGroup));
    a.tl.seq_group = reinterpret_cast<int32_t *>(p);
    p += up256((size_t)num_seqs * 4);
    a.tl.rec = reinterpret_cast<float *>(p);
    p += rows_bytes(num_seqs, n_heads, head_dim);
    a.first = reinterpret_cast<float *>(p);
    p += rows_bytes(num_seqs, n_heads, head_dim);
    a.more = reinterpret_cast<float *>(p);
    a.tl.groups = {group_starts, shared_blocks, num_groups, max_blocks_per_seq};
    a.q = static_cast<const __half *>(q);
    a.kplane = cache_plane(cache, 0, layer);
    a.vplane = cache_plane(cache, 1, layer);
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
    const int rc2 = launch_decode_tails(c, at, a.tl);
    if (rc2 != PA_OK) return rc2;
    return head_dim == 128 ? launch_shared<128>(a, st) : launch_shared<64>(a, st);
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
            if (members == 1) shared_blocks[n - 1] = 0;
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
