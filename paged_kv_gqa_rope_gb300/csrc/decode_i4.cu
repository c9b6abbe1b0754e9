// Single-token GQA decode against the 4-bit pool (include/pa.h,
// pa_cache_i4_t): out = softmax(scale q K^T) V with K and V standing for
// m + s c.
//
// One CTA per (sequence, KV head); its warps take the blocks in turn.  A lane
// holds one half of one token's K row for the scores of the g heads, then a
// few columns of O for P V; the running maximum and sum of the softmax are
// per warp and head, and the warps' results are joined at the end.
#include "common.cuh"
#include "internal.h"
#include "kv_int4.cuh"

namespace pa {
namespace {

constexpr int kMaxSeqs = 4096;
constexpr int kGroupPad = 8;
constexpr int kWarps = 8;

struct DecodeI4Args {
    const __half *q;
    const uint8_t *tiles;
    const int32_t *block_tables;
    const int32_t *context_lens;
    __half *out;
    int32_t *status;
    float scale_log2;
    int B, H, Hk, g, maxb, num_blocks;
};

template <int D>
__global__ void __launch_bounds__(kWarps * 32) decode_i4_kernel(const DecodeI4Args a) {
    using T = I4Tile<D>;
    constexpr int kCols = D / 32;
    __shared__ float sm_q[kGroupPad][D];
    __shared__ float sm_o[kWarps][kGroupPad][D];
    __shared__ float sm_m[kWarps][kGroupPad], sm_l[kWarps][kGroupPad];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int kvh = blockIdx.x % a.Hk, s = blockIdx.x / a.Hk;
    const int ctx = __ldg(a.context_lens + s);
    if (ctx < 1 || ctx > a.maxb * kBlockSize) {
        if (tid == 0 && kvh == 0) report(a.status, PA_DEV_BAD_LENGTH);
        return;
    }
    for (int i = tid; i < a.g * D; i += kWarps * 32)
        sm_q[i / D][i % D] =
            __half2float(a.q[((int64_t)s * a.H + kvh * a.g) * D + i]) * a.scale_log2;
    __syncthreads();
    float m[kGroupPad], l[kGroupPad], o[kGroupPad][kCols];
    for (int h = 0; h < kGroupPad; ++h) {
        m[h] = -INFINITY;
        l[h] = 0.f;
        for (int c = 0; c < kCols; ++c) o[h][c] = 0.f;
    }
    const int nblk = (ctx + kBlockSize - 1) / kBlockSize;
    const int j = lane & 15, half = lane >> 4;
    for (int b = warp; b < nblk; b += kWarps) {
        const int blk = __ldg(a.block_tables + (int64_t)s * a.maxb + b);
        if (blk < 0 || blk >= a.num_blocks) {
            if (lane == 0) report(a.status, PA_DEV_BAD_BLOCK);
            continue;
        }
        const uint8_t *kt = a.tiles + ((int64_t)blk * a.Hk + kvh) * T::kPair, *vt = kt + T::kBytes;
        const bool live = b * kBlockSize + j < ctx;
        float x[kGroupPad] = {};
        for (int gr = half * (T::kGroups / 2); gr < (half + 1) * (T::kGroups / 2); ++gr) {
            const float st = __half2float(*(const __half *)(kt + T::step(j, gr)));
            const float ls = __half2float(*(const __half *)(kt + T::least_k(j, gr)));
            for (int t = 0; t < 4; ++t) {
                const uint32_t w = *(const uint32_t *)(kt + T::k_word(j, gr, t));
                for (int i = 0; i < 8; ++i) {
                    const float k = ls + st * (float)((w >> (4 * i)) & 15u);
                    for (int h = 0; h < a.g; ++h) x[h] += k * sm_q[h][32 * gr + 8 * t + i];
                }
            }
        }
        for (int h = 0; h < a.g; ++h) {
            x[h] += __shfl_xor_sync(0xffffffffu, x[h], 16);
            if (!live) x[h] = -INFINITY;
            float bm = x[h];
            for (int f = 8; f >= 1; f >>= 1) bm = fmaxf(bm, __shfl_xor_sync(0xffffffffu, bm, f));
            const float mn = fmaxf(m[h], bm), al = ex2(m[h] - mn);
            m[h] = mn;
            x[h] = ex2(x[h] - mn);
            l[h] = l[h] * al + (half == 0 ? x[h] : 0.f);
            for (int c = 0; c < kCols; ++c) o[h][c] *= al;
        }
        for (int t = 0; t < kBlockSize && b * kBlockSize + t < ctx; ++t) {
            float v[kCols];
            for (int c = 0; c < kCols; ++c) {  // columns 32 c + lane
                const float st = __half2float(*(const __half *)(vt + T::step(t, c)));
                const float ls = __half2float(*(const __half *)(vt + T::least_v(t, c)));
                const uint32_t w = *(const uint16_t *)(vt + T::v_half(t, c, lane >> 2));
                v[c] = ls + st * (float)((w >> (4 * (lane & 3))) & 15u);
            }
            for (int h = 0; h < a.g; ++h) {
                const float p = __shfl_sync(0xffffffffu, x[h], t);
                for (int c = 0; c < kCols; ++c) o[h][c] += p * v[c];
            }
        }
    }
    for (int h = 0; h < a.g; ++h) {
        for (int f = 16; f >= 1; f >>= 1) l[h] += __shfl_xor_sync(0xffffffffu, l[h], f);
        if (lane == 0) {
            sm_m[warp][h] = m[h];
            sm_l[warp][h] = l[h];
        }
        for (int c = 0; c < kCols; ++c) sm_o[warp][h][32 * c + lane] = o[h][c];
    }
    __syncthreads();
    for (int i = tid; i < a.g * D; i += kWarps * 32) {
        const int h = i / D, d = i % D;
        float M = -INFINITY, L = 0.f, O = 0.f;
        for (int w = 0; w < kWarps; ++w) M = fmaxf(M, sm_m[w][h]);
        for (int w = 0; w < kWarps; ++w) {
            const float f = M == -INFINITY ? 0.f : ex2(sm_m[w][h] - M);
            L += f * sm_l[w][h];
            O += f * sm_o[w][h][d];
        }
        a.out[((int64_t)s * a.H + kvh * a.g) * D + i] = __float2half_rn(L > 0.f ? O / L : 0.f);
    }
}

}  // namespace
}  // namespace pa

using namespace pa;

extern "C" size_t pa_decode_i4_workspace_bytes(int num_seqs, int n_heads, int n_kv_heads,
                                               int head_dim) {
    if (num_seqs <= 0 || n_heads <= 0 || n_kv_heads <= 0 || head_dim <= 0) return 0;
    return 256;
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
    a.status = dev_status;
    a.scale_log2 = scale * 1.4426950408889634f;
    a.B = num_seqs;
    a.H = n_heads;
    a.Hk = n_kv_heads;
    a.g = n_heads / n_kv_heads;
    a.maxb = max_blocks_per_seq;
    a.num_blocks = cache->num_blocks;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (head_dim == 128)
        decode_i4_kernel<128><<<num_seqs * n_kv_heads, kWarps * 32, 0, st>>>(a);
    else
        decode_i4_kernel<64><<<num_seqs * n_kv_heads, kWarps * 32, 0, st>>>(a);
    return launch_status();
}
