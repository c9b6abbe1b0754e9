// The rotary append with other layouts than rope_kv.cu's: pairs of neighbours
// or of halves, a part of the head, tables scaled for long contexts
// (pa_rope_kv_write_layout, pa_rope_table_init_scaled).
//
// The first r values x of every Q and K row are turned pairwise, pair i by the
// angle of table row positions[t], column i:
//     a' = fl32(fl32(a c) - fl32(b s)),   b' = fl32(fl32(a s) + fl32(b c)),
// (a, b) = (x_2i, x_2i+1) interleaved or (x_i, x_(i + r/2)) half, rounded once to
// fp16; the other d - r values pass unchanged.
//
// Bound: HBM (4 d bytes a Q head, 8 d a KV head and token: each row in once, out
// once).  A work item is 32 bytes of a row, its two 16-byte pieces chosen so
// that both ends of every pair are in it: pieces 2u and 2u + 1, or for the half
// layout u and u + r/16 (then, behind the rotated part, neighbours again).  So no
// thread waits for another, and a warp's loads cover whole lines either way.
#include <math.h>

#include <algorithm>
#include <new>

#include "common.cuh"
#include "internal.h"

namespace pa {
namespace {

struct LayoutArgs {
    const __half *q;
    __half *q_out;
    const __half *k;
    const __half *v;
    const int32_t *positions;
    const int32_t *slots;
    const float2 *table;  // [max_pos][rotary / 2] {cos, sin}
    __half *kcache;       // K plane of the layer: [num_slots][Hk][d]
    __half *vcache;
    int64_t num_slots;
    int32_t *status;
    int num_tokens, n_heads, n_kv_heads, max_pos, rotary;
    bool stream;  // see kStreamBytes
};

// Rows are read once, with the evict-first policy; batches that write more than
// this (half of L2) also store with it, since nobody finds their rows in L2 anyway
// (16 prompts, 64/8 heads, 352 MB: 54.6 us, 96 % of the copy bandwidth, against 61.7
// with the policy on neither side and 62 with it on one).  Smaller ones leave Q, K
// and V where the attention that follows reads them.
constexpr int64_t kStreamBytes = 64 << 20;

__device__ __forceinline__ void put(uint4 *p, const uint4 &x, bool stream) {
    if (stream)
        __stcs(p, x);
    else
        *p = x;
}

// One pair in the pinned fp32 arithmetic (no contraction into FMA).
__device__ __forceinline__ void turn(float &a, float &b, float c, float s) {
    const float x = __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s));
    b = __fadd_rn(__fmul_rn(a, s), __fmul_rn(b, c));
    a = x;
}

// Eight pairs (lo_i, hi_i), the angles at cs .. cs + 7.
__device__ __forceinline__ void turn_halves(uint4 &lo, uint4 &hi, const float4 *cs) {
    uint32_t *l = reinterpret_cast<uint32_t *>(&lo), *h = reinterpret_cast<uint32_t *>(&hi);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float4 t = __ldg(cs + i);  // two angles
        float2 a = __half22float2(*reinterpret_cast<const __half2 *>(l + i));
        float2 b = __half22float2(*reinterpret_cast<const __half2 *>(h + i));
        turn(a.x, b.x, t.x, t.y);
        turn(a.y, b.y, t.z, t.w);
        l[i] = pack_half2(a.x, a.y);
        h[i] = pack_half2(b.x, b.y);
    }
}

// The pieces p0 and p1 of a row's work item u; the first nrot items are rotated.
template <bool HALF>
__device__ __forceinline__ void pieces_of(int u, int nrot, int &p0, int &p1) {
    if (HALF && u < nrot) {
        p0 = u;
        p1 = u + nrot;
    } else {
        p0 = 2 * u;
        p1 = 2 * u + 1;
    }
}

template <int D, bool HALF>
__global__ void __launch_bounds__(kTokenThreads) rope_layout_kernel(const LayoutArgs a) {
    // As rope_kv_write_kernel: the next kernel may set up now, and nothing is
    // read or written before the kernel ahead has finished.
    griddep_launch_dependents();
    griddep_wait();
    constexpr int kItems = D / 16;
    const int H = a.n_heads, Hk = a.n_kv_heads;
    const int t = (int)(blockIdx.z * gridDim.y + blockIdx.y);
    const int i = (int)(blockIdx.x * blockDim.x + threadIdx.x);
    if (t >= a.num_tokens || i >= (H + 2 * Hk) * kItems) return;
    const int u = i % kItems, row = i / kItems;

    const int pos = __ldg(a.positions + t);
    if (pos < 0 || pos >= a.max_pos) {
        if (i == 0) report(a.status, PA_DEV_BAD_POSITION);
        return;
    }
    const int slot = __ldg(a.slots + t);
    const bool write_cache = slot >= 0 && slot < a.num_slots;
    if (slot >= a.num_slots && i == 0) report(a.status, PA_DEV_BAD_SLOT);

    const int nrot = a.rotary / 16;  // items with rotated values
    int p0, p1;
    const uint4 *src;
    uint4 *dst;
    if (row >= H + Hk) {
        if (!write_cache) return;
        const int h = row - H - Hk;
        src = reinterpret_cast<const uint4 *>(a.v + ((int64_t)t * Hk + h) * D);
        dst = reinterpret_cast<uint4 *>(a.vcache + ((int64_t)slot * Hk + h) * D);
        put(dst + 2 * u, __ldcs(src + 2 * u), a.stream);
        put(dst + 2 * u + 1, __ldcs(src + 2 * u + 1), a.stream);
        return;
    }
    if (row < H) {
        src = reinterpret_cast<const uint4 *>(a.q + ((int64_t)t * H + row) * D);
        dst = reinterpret_cast<uint4 *>(a.q_out + ((int64_t)t * H + row) * D);
    } else {
        if (!write_cache) return;
        const int h = row - H;
        src = reinterpret_cast<const uint4 *>(a.k + ((int64_t)t * Hk + h) * D);
        dst = reinterpret_cast<uint4 *>(a.kcache + ((int64_t)slot * Hk + h) * D);
    }
    pieces_of<HALF>(u, nrot, p0, p1);
    uint4 x0 = __ldcs(src + p0), x1 = __ldcs(src + p1);
    if (u < nrot) {
        const float4 *cs =
            reinterpret_cast<const float4 *>(a.table + (int64_t)pos * (a.rotary / 2) + 8 * u);
        if (HALF) {
            turn_halves(x0, x1, cs);
        } else {
            x0 = rope_rotate8(x0, __ldg(cs), __ldg(cs + 1));
            x1 = rope_rotate8(x1, __ldg(cs + 2), __ldg(cs + 3));
        }
    }
    put(dst + p0, x0, a.stream);
    put(dst + p1, x1, a.stream);
}

template <int D, bool HALF>
int launch_layout(const LayoutArgs &a, cudaStream_t st) {
    const dim3 grid = token_grid(a.num_tokens, (a.n_heads + 2 * a.n_kv_heads) * (D / 16));
    launch_dependent(rope_layout_kernel<D, HALF>, grid, dim3(kTokenThreads), 0, st, a);
    return launch_status();
}

// Angular frequencies of the r / 2 pairs; false for parameters out of range.
bool frequencies(double *f, int r, double theta, const pa_rope_scaling_t *sc, double *magnitude) {
    const int n = r / 2;
    const int kind = sc ? sc->kind : PA_ROPE_UNSCALED;
    *magnitude = 1.0;
    if (!(theta > 1.0) || !isfinite(theta)) return false;
    if (kind != PA_ROPE_UNSCALED && (!(sc->factor >= 1.0) || !isfinite(sc->factor))) return false;
    if (sc && sc->attention != 0.0) {
        if (!(sc->attention > 0.0) || !isfinite(sc->attention)) return false;
        *magnitude = sc->attention;
    }
    if (kind == PA_ROPE_NTK) theta *= pow(sc->factor, (double)r / (double)(r - 2));
    if (!isfinite(theta)) return false;
    for (int i = 0; i < n; ++i) f[i] = 1.0 / pow(theta, (double)(2 * i) / (double)r);
    if (kind == PA_ROPE_UNSCALED || kind == PA_ROPE_NTK) return true;
    if (kind == PA_ROPE_LINEAR) {
        for (int i = 0; i < n; ++i) f[i] /= sc->factor;
        return true;
    }
    if (kind != PA_ROPE_YARN && kind != PA_ROPE_BANDS) return false;
    if (sc->original_positions <= 0 || !(sc->low > 0.0) || !(sc->high > sc->low) ||
        !isfinite(sc->high))
        return false;
    const double turns = sc->original_positions / 6.283185307179586476925286766559;
    // (YaRN's ramp is linear in i, between the pairs that turn `high` and `low` times)
    const double first = floor((double)r * log(turns / sc->high) / (2.0 * log(theta)));
    const double last = ceil((double)r * log(turns / sc->low) / (2.0 * log(theta)));
    const double lo = std::max(first, 0.0), hi = std::min(last, (double)(r - 1));
    for (int i = 0; i < n; ++i) {
        double keep;  // 1: the pair's own frequency, 0: divided by the factor
        if (kind == PA_ROPE_BANDS)
            keep = (turns * f[i] - sc->low) / (sc->high - sc->low);
        else
            keep = 1.0 - (i - lo) / (hi > lo ? hi - lo : 0.001);
        keep = std::min(std::max(keep, 0.0), 1.0);
        f[i] = f[i] * keep + f[i] / sc->factor * (1.0 - keep);
    }
    if (kind == PA_ROPE_YARN && sc->attention == 0.0) *magnitude = 0.1 * log(sc->factor) + 1.0;
    return true;
}

}  // namespace
}  // namespace pa

using namespace pa;

extern "C" int pa_rope_table_init_scaled(void *device_table, int max_positions, int rotary_dim,
                                         double theta, const pa_rope_scaling_t *scaling,
                                         pa_stream_t stream) {
    if (!device_table || !aligned16(device_table) || max_positions <= 0) return PA_ERR_INVALID;
    if (rotary_dim <= 0 || rotary_dim % 16 != 0 || rotary_dim > 128) return PA_ERR_UNSUPPORTED;
    double f[64], magnitude;
    if (!frequencies(f, rotary_dim, theta, scaling, &magnitude)) return PA_ERR_INVALID;
    const size_t n = (size_t)max_positions * rotary_dim;
    float *host = new (std::nothrow) float[n];
    if (!host) return PA_ERR_CUDA;
    for (int m = 0; m < max_positions; ++m) {
        float *row = host + (size_t)m * rotary_dim;
        for (int i = 0; i < rotary_dim / 2; ++i) {
            const double ang = (double)m * f[i];
            row[2 * i] = (float)(magnitude * cos(ang));
            row[2 * i + 1] = (float)(magnitude * sin(ang));
        }
    }
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const bool ok = cudaMemcpyAsync(device_table, host, n * sizeof(float), cudaMemcpyHostToDevice,
                                    st) == cudaSuccess &&
                    cudaStreamSynchronize(st) == cudaSuccess;
    delete[] host;
    if (!ok) cudaGetLastError();
    return ok ? PA_OK : PA_ERR_CUDA;
}

extern "C" int pa_rope_kv_write_layout(const void *q, void *q_out, const void *k, const void *v,
                                       const int32_t *positions, const int32_t *slot_mapping,
                                       int num_tokens, int n_heads, int n_kv_heads, int head_dim,
                                       int layout, int rotary_dim, const void *rope_table,
                                       int max_positions, const pa_cache_t *cache, int layer,
                                       int32_t *dev_status, pa_stream_t stream) {
    if (num_tokens < 0 || n_heads <= 0 || n_kv_heads <= 0 || n_heads % n_kv_heads != 0 ||
        max_positions <= 0 || (layout != PA_ROPE_INTERLEAVED && layout != PA_ROPE_HALF))
        return PA_ERR_INVALID;
    if (head_dim != 64 && head_dim != 128) return PA_ERR_UNSUPPORTED;
    if (rotary_dim <= 0 || rotary_dim > head_dim) return PA_ERR_INVALID;
    if (rotary_dim % 16 != 0) return PA_ERR_UNSUPPORTED;
    if (!cache_ok(cache, layer, n_kv_heads, head_dim)) return PA_ERR_INVALID;
    if (num_tokens == 0) return PA_OK;
    if (!q || !q_out || !k || !v || !positions || !slot_mapping || !rope_table)
        return PA_ERR_INVALID;
    if (!aligned16(q) || !aligned16(q_out) || !aligned16(k) || !aligned16(v) ||
        !aligned16(rope_table))
        return PA_ERR_INVALID;
    // (items of a token in int32; as pa_rope_kv_write bounds a call's)
    if (((int64_t)n_heads + 2 * (int64_t)n_kv_heads) * (head_dim / 16) > INT32_MAX / 2 ||
        (int64_t)num_tokens * ((int64_t)n_heads + 2 * (int64_t)n_kv_heads) * (head_dim / 8) >
            (int64_t)1 << 40)
        return PA_ERR_INVALID;
    const uint64_t qn = (uint64_t)num_tokens * n_heads * head_dim * 2;
    const uint64_t kn = (uint64_t)num_tokens * n_kv_heads * head_dim * 2;
    if ((q_out != q && ranges_overlap(q, qn, q_out, qn)) || ranges_overlap(q_out, qn, k, kn) ||
        ranges_overlap(q_out, qn, v, kn))
        return PA_ERR_INVALID;

    LayoutArgs a;
    a.q = static_cast<const __half *>(q);
    a.q_out = static_cast<__half *>(q_out);
    a.k = static_cast<const __half *>(k);
    a.v = static_cast<const __half *>(v);
    a.positions = positions;
    a.slots = slot_mapping;
    a.table = static_cast<const float2 *>(rope_table);
    a.kcache = cache_plane(cache, 0, layer);
    a.vcache = cache_plane(cache, 1, layer);
    a.num_slots = (int64_t)cache->num_blocks * cache->block_size;
    a.status = dev_status;
    a.num_tokens = num_tokens;
    a.n_heads = n_heads;
    a.n_kv_heads = n_kv_heads;
    a.max_pos = max_positions;
    a.rotary = rotary_dim;
    a.stream = (int64_t)num_tokens * (n_heads + 2 * (int64_t)n_kv_heads) * head_dim * 2 > kStreamBytes;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const bool half = layout == PA_ROPE_HALF;
    if (head_dim == 128)
        return half ? launch_layout<128, true>(a, st) : launch_layout<128, false>(a, st);
    return half ? launch_layout<64, true>(a, st) : launch_layout<64, false>(a, st);
}
