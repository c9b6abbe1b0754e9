// Decode that accumulates attention weights (pa_decode_weights).
//
// With x[h][t] the scaled score of Q head h and token t in log2 units,
//     out[h]  = sum_t p[h][t] v[t],   p[h][t] = 2^(x[h][t] - m_h) / l_h,
//     weights_out[kv head][t] = weights[kv head][t] + sum over its Q heads of p[h][t].
// A token's p is known only once its row's last token has been seen, so the
// decode kernel leaves the scores (fp32, 4 g bytes a (token, KV head), against
// 4 d for its K and V row) and each row's m and 1/l behind; this kernel turns
// them into weights, and joins the outputs of the pairs (sequence, KV head) that the
// decode kernel's CTAs have left in pieces.  Reading K a second time instead would cost
// 2 d bytes.
//
// Bound: L2 and HBM, 4 g + 8 bytes a (token, KV head).
#include <algorithm>

#include "decode_modes.cuh"

namespace pa {
namespace {

constexpr int kWeightThreads = 128;
constexpr int kWeightTokens = 4;
constexpr int kFewPieces = 8;  // that a thread reads at once

struct WeightArgs {
    DecodeScores sc;
    const float *weights;  // nullptr: zeros
    float *weights_out;
    __half *out;
    float *recs;  // the decode kernel's CTAs'
    int64_t stride;
    int B, H, Hk, d;
};

// The line's data are not needed any more.
__device__ __forceinline__ void discard_l2(const float *p) {
    asm volatile("discard.global.L2 [%0], 128;" ::"l"(p) : "memory");
}

// grid (chunks of tokens, Hk, B).  A thread has kWeightTokens tokens at a time, all
// their loads in flight together with the statistics' (a token at a time: 12 us of
// the serving batch of 64/8 heads and 4097 tokens).  32 CTAs an SM at most: twice as
// many, most of them without tokens, cost a ragged batch 3.6 us.
template <int G>
__global__ void __launch_bounds__(kWeightThreads, 8) weights_kernel(const WeightArgs a) {
    griddep_wait();
    griddep_launch_dependents();
    const int h = blockIdx.y, s = blockIdx.z;
    // (The length is the one that the decode kernel read: context_lens, should they have
    // changed since, could lead past the scores and the rows of weights.)
    const SeqScores q = a.sc.seqs[s];
    const int64_t first = q.first;
    const int n = first == -1 ? 0 : q.len;  // (-1: no scores kept)
    const Cut cut = cut_of(a.sc.pieces.cut[s * a.Hk + h]);
    if (first == -2) return;
    __shared__ float2 stats[G];
    auto piece = [&](int i, int j) {
        return i == 0 ? Record{a.sc.pieces.rec, (int64_t)a.B * a.H, ((int64_t)h * a.B + s) * G + j}
                      : piece_of(a.recs, cut.cta + i - 1, a.d, j);
    };
    __shared__ float factors[kFewPieces][G];
    // The rows' statistics: of a pair in few pieces a thread has a row, of others a warp
    // has a row at a time, a lane a piece (for all: weights_ragged +1.3 us).
    auto read_stats = [&]() {
        const int tid = threadIdx.x, lane = tid & 31;
        if (cut.more == 0) {
            if (tid < G) stats[tid] = a.sc.stats[(int64_t)s * a.H + h * G + tid];
        } else if (cut.more < kFewPieces) {
            if (tid < G) {
                float2 ml[kFewPieces];
                float M = -INFINITY, L = 0.f;
#pragma unroll
                for (int i = 0; i < kFewPieces; ++i)
                    ml[i] = i <= cut.more ? *piece(i, tid).stat(a.d) : make_float2(-INFINITY, 0.f);
#pragma unroll
                for (int i = 0; i < kFewPieces; ++i) M = fmaxf(M, ml[i].x);
#pragma unroll
                for (int i = 0; i < kFewPieces; ++i) {
                    const float f = ml[i].x == -INFINITY ? 0.f : ex2(ml[i].x - M);
                    factors[i][tid] = f;
                    L = fmaf(f, ml[i].y, L);
                }
                const bool none = L == 0.f;  // (no block in range: weights and output 0)
                stats[tid] = none ? make_float2(0.f, 0.f) : make_float2(M, 1.f / L);
            }
        } else {
            for (int j = tid / 32; j < G; j += kWeightThreads / 32) {
                float M = -INFINITY, L = 0.f;
                for (int i0 = 0; i0 <= cut.more; i0 += 32) {
                    const float2 ml = i0 + lane <= cut.more ? *piece(i0 + lane, j).stat(a.d)
                                                            : make_float2(-INFINITY, 0.f);
                    float top = ml.x;
#pragma unroll
                    for (int o = 16; o > 0; o >>= 1)
                        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
                    top = fmaxf(M, top);
                    float sum = ml.x == -INFINITY ? 0.f : ex2(ml.x - top) * ml.y;
#pragma unroll
                    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
                    L = fmaf(M == -INFINITY ? 0.f : ex2(M - top), L, sum);
                    M = top;
                }
                const bool none = L == 0.f;
                if (lane == 0) stats[j] = none ? make_float2(0.f, 0.f) : make_float2(M, 1.f / L);
            }
        }
        __syncthreads();
    };
    bool known = false;
    const float *x =
        a.sc.scores + (first + (int64_t)((n + kBlockSize - 1) / kBlockSize) * h) * kBlockSize * G;
    const int64_t kept = (int64_t)((n + kBlockSize - 1) / kBlockSize) * kBlockSize * G;  // from x
    const int64_t row = ((int64_t)s * a.Hk + h) * a.stride;
    constexpr int kStep = kWeightThreads * kWeightTokens;
    for (int64_t t0 = (int64_t)blockIdx.x * kStep; t0 < n; t0 += (int64_t)gridDim.x * kStep) {
        float v[kWeightTokens][G], w[kWeightTokens];
#pragma unroll
        for (int i = 0; i < kWeightTokens; ++i) {
            const int64_t t = t0 + i * kWeightThreads + threadIdx.x;
            w[i] = 0.f;
            if (t < n) {
                if constexpr (G % 4 == 0) {
#pragma unroll
                    for (int j = 0; j < G; j += 4) {
                        const float4 y = __ldcs(reinterpret_cast<const float4 *>(x + t * G + j));
                        v[i][j] = y.x, v[i][j + 1] = y.y, v[i][j + 2] = y.z, v[i][j + 3] = y.w;
                    }
                } else if constexpr (G % 2 == 0) {
#pragma unroll
                    for (int j = 0; j < G; j += 2) {
                        const float2 y = __ldcs(reinterpret_cast<const float2 *>(x + t * G + j));
                        v[i][j] = y.x, v[i][j + 1] = y.y;
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < G; ++j) v[i][j] = __ldcs(x + t * G + j);
                }
                if (a.weights) w[i] = a.weights[row + t];
            }
        }
        if (!known) read_stats();
        known = true;
        float p[kWeightTokens] = {};
#pragma unroll
        for (int j = 0; j < G; ++j) {
            const float2 st = stats[j];
#pragma unroll
            for (int i = 0; i < kWeightTokens; ++i) p[i] = fmaf(ex2(v[i][j] - st.x), st.y, p[i]);
        }
#pragma unroll
        for (int i = 0; i < kWeightTokens; ++i) {
            const int64_t t = t0 + i * kWeightThreads + threadIdx.x;
            if (t < n) a.weights_out[row + t] = w[i] + p[i];
        }
        if constexpr (G % 2 == 0) {
            // The scores have been read: their lines need not be written to HBM (64/8
            // heads, 32 x 4097 tokens: 103.3 -> 98.0 us).  With G even a block's are whole
            // lines, and a warp's 32 tokens' are G of them.
            __syncwarp();
            const int lane = threadIdx.x & 31;
#pragma unroll
            for (int i = 0; i < kWeightTokens; ++i) {
                const int64_t at = (t0 + i * kWeightThreads + (threadIdx.x & ~31)) * G + lane * 32;
                if (lane < G && at + 32 <= kept) discard_l2(x + at);
            }
        }
    }
    // (the last CTA has the fewest tokens)
    if (cut.more == 0 || blockIdx.x != gridDim.x - 1) return;
    if (!known) read_stats();
    for (int i0 = threadIdx.x; i0 < G * (a.d / 4); i0 += kWeightThreads) {
        const int j = i0 / (a.d / 4), c = i0 - j * (a.d / 4);
        float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
        auto add = [&](float f, const float4 &O) {
            y.x = fmaf(f, O.x, y.x);
            y.y = fmaf(f, O.y, y.y);
            y.z = fmaf(f, O.z, y.z);
            y.w = fmaf(f, O.w, y.w);
        };
        if (cut.more < kFewPieces) {
            float4 O[kFewPieces];
#pragma unroll
            for (int i = 0; i < kFewPieces; ++i)
                O[i] = i <= cut.more ? *piece(i, j).cols(c) : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int i = 0; i < kFewPieces; ++i) add(factors[i][j], O[i]);
        } else {
            const float M = stats[j].x;
#pragma unroll 8
            for (int i = 0; i <= cut.more; ++i) {
                const float m = piece(i, j).stat(a.d)->x;
                add(m == -INFINITY ? 0.f : ex2(m - M), *piece(i, j).cols(c));
            }
        }
        const float inv = stats[j].y;
        *reinterpret_cast<uint2 *>(a.out + ((int64_t)s * a.H + h * G + j) * a.d + 4 * c) =
            make_uint2(pack_half2(saturate16(y.x * inv), saturate16(y.y * inv)),
                       pack_half2(saturate16(y.z * inv), saturate16(y.w * inv)));
    }
}

size_t up256(size_t n) { return (n + 255) & ~(size_t)255; }

// Workspace: the decode kernel's, the statistics, the sequences' places and lengths, the cut
// pairs, their first pieces, scores.
size_t record_bytes(int B, int H, int D) {
    return up256((size_t)B * H * ((size_t)D + 4) * sizeof(float));
}
size_t fixed_bytes(int B, int H, int Hk, int D) {
    return up256(mode_workspace_bytes(D)) + up256((size_t)B * H * sizeof(float2)) +
           up256((size_t)B * sizeof(SeqScores)) + up256((size_t)B * Hk * sizeof(int32_t)) +
           record_bytes(B, H, D);
}

}  // namespace
}  // namespace pa

using namespace pa;

extern "C" size_t pa_decode_weights_workspace_bytes(int num_seqs, int n_heads, int n_kv_heads,
                                                    int head_dim, int64_t score_blocks) {
    if (num_seqs <= 0 || n_heads <= 0 || n_kv_heads <= 0 || head_dim <= 0 || score_blocks <= 0)
        return 0;
    // (the parts first: each must fit by itself before it is counted in 64 bits)
    const unsigned __int128 n =
        (unsigned __int128)score_blocks * kBlockSize * n_heads * 4 +
        (unsigned __int128)num_seqs * n_heads * (head_dim + (int64_t)6) * sizeof(float) +
        (unsigned __int128)num_seqs * n_kv_heads * sizeof(int32_t);
    if (n > SIZE_MAX / 2) return 0;
    return (size_t)score_blocks * kBlockSize * n_heads * 4 +
           fixed_bytes(num_seqs, n_heads, n_kv_heads, head_dim);
}

extern "C" int pa_decode_weights(const void *q, const pa_cache_t *cache, int layer,
                                 const int32_t *block_tables, int max_blocks_per_seq,
                                 const int32_t *context_lens, int num_seqs, int n_heads,
                                 int n_kv_heads, int head_dim, float scale, const float *weights,
                                 float *weights_out, int64_t weights_stride, void *workspace,
                                 size_t workspace_bytes, void *out, int32_t *dev_status,
                                 pa_stream_t stream) {
    const int rc = check_decode_args(q, cache, layer, block_tables, max_blocks_per_seq,
                                     context_lens, num_seqs, n_heads, n_kv_heads, head_dim, scale,
                                     out);
    if (rc != PA_OK) return rc;
    if (weights_stride <= 0) return PA_ERR_INVALID;
    if (n_kv_heads > 65535) return PA_ERR_UNSUPPORTED;  // (a grid's y)
    if (num_seqs == 0) return PA_OK;
    if (!weights_out || !workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u))
        return PA_ERR_INVALID;
    const unsigned __int128 rows = (unsigned __int128)num_seqs * n_kv_heads * weights_stride * 4;
    if (rows > SIZE_MAX || (weights && weights_out != weights &&
                            ranges_overlap(weights, (uint64_t)rows, weights_out, (uint64_t)rows)))
        return PA_ERR_INVALID;
    const size_t fixed = fixed_bytes(num_seqs, n_heads, n_kv_heads, head_dim);
    const size_t block = (size_t)kBlockSize * n_heads * sizeof(float);  // of all KV heads
    if (workspace_bytes < fixed + block) return PA_ERR_WORKSPACE;

    uint8_t *at = static_cast<uint8_t *>(workspace);
    uint8_t *p = at + up256(mode_workspace_bytes(head_dim));
    WeightArgs w;
    w.sc.stats = reinterpret_cast<float2 *>(p);
    p += up256((size_t)num_seqs * n_heads * sizeof(float2));
    w.sc.seqs = reinterpret_cast<SeqScores *>(p);
    p += up256((size_t)num_seqs * sizeof(SeqScores));
    w.sc.pieces.cut = reinterpret_cast<int32_t *>(p);
    p += up256((size_t)num_seqs * n_kv_heads * sizeof(int32_t));
    w.sc.pieces.rec = reinterpret_cast<float *>(p);
    w.sc.scores = reinterpret_cast<float *>(at + fixed);
    w.sc.capacity = (int64_t)((workspace_bytes - fixed) / block) * n_kv_heads;
    w.sc.max_len = (int)std::min<int64_t>(weights_stride, INT32_MAX);
    w.weights = weights;
    w.weights_out = weights_out;
    w.stride = weights_stride;
    w.out = static_cast<__half *>(out);
    w.recs = mode_records(workspace);
    w.B = num_seqs;
    w.H = n_heads;
    w.Hk = n_kv_heads;
    w.d = head_dim;
    const DecodeCall c = {q,        cache,   layer,      block_tables, max_blocks_per_seq,
                          context_lens, num_seqs, n_heads, n_kv_heads, head_dim,
                          scale,    out,     dev_status, static_cast<cudaStream_t>(stream)};
    const int rc2 = launch_decode_scores(c, at, w.sc);
    if (rc2 != PA_OK) return rc2;
    // CTAs for the longest row the table allows, as long as they are few
    const int64_t pairs = (int64_t)num_seqs * n_kv_heads;
    const int64_t longest = (int64_t)max_blocks_per_seq * kBlockSize;
    constexpr int kStep = kWeightThreads * kWeightTokens;
    const int64_t chunks = std::min((longest + kStep - 1) / kStep,
                                    std::max<int64_t>(1, (32 * (int64_t)sm_count() + pairs - 1) / pairs));
    const dim3 grid((unsigned)chunks, n_kv_heads, num_seqs), block_dim(kWeightThreads);
    switch (n_heads / n_kv_heads) {
#define PA_CASE(G) \
    case G: launch_dependent(weights_kernel<G>, grid, block_dim, 0, c.stream, w); break;
        PA_CASE(1) PA_CASE(2) PA_CASE(3) PA_CASE(4) PA_CASE(5) PA_CASE(6) PA_CASE(7) PA_CASE(8)
#undef PA_CASE
    }
    return launch_status();
}
