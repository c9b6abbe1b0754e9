// The 4-bit KV pool's tile (layout and scheme: include/pa.h, pa_cache_i4_t),
// shared by the kernels that write it, read it back and attend to it.
#pragma once

#include <cuda_fp16.h>
#include <stdint.h>

#include "internal.h"

namespace pa {

// One block of 16 tokens of one KV head, K or V: codes, then steps and least
// values.  All offsets in bytes from the tile's start.
template <int D>
struct I4Tile {
    static constexpr int kGroups = D / 32;
    static constexpr int kCodes = 8 * D;
    static constexpr int kBytes = 10 * D;   // K or V
    static constexpr int kPair = 2 * kBytes;  // K, then V

    // The 32-bit word with the codes of K row j, values 32 g + 8 t .. + 7.
    __host__ __device__ static constexpr int k_word(int j, int g, int t) {
        return j * (D / 2) + t * (4 * kGroups) + 4 * g;
    }
    // The 16-bit word with the codes of V row j, values 32 g + 4 u .. + 3.
    __host__ __device__ static constexpr int v_half(int j, int g, int u) {
        return 2 * (2 * (kGroups * (4 * (8 * (j >> 3) + u) + ((j & 7) >> 1)) + g) + (j & 1));
    }
    // The step of row j, group g.
    __host__ __device__ static constexpr int step(int j, int g) {
        return kCodes + 2 * (4 * (kGroups * ((j & 7) >> 1) + g) + 2 * (j >> 3) + (j & 1));
    }
    // The least value of row j, group g.
    __host__ __device__ static constexpr int least_k(int j, int g) {
        return kCodes + 2 * (16 * kGroups + kGroups * j + g);
    }
    __host__ __device__ static constexpr int least_v(int j, int g) {
        return 32 * kGroups + step(j, g);
    }
};

__device__ __forceinline__ __half2 as_half2(uint32_t w) {
    return *reinterpret_cast<const __half2 *>(&w);
}
__device__ __forceinline__ uint32_t as_u32(__half2 h) {
    return *reinterpret_cast<const uint32_t *>(&h);
}

// x[1] .. x[n] become their running sums; one warp.
__device__ __forceinline__ void prefix_sums(int64_t *x, int n, int lane) {
    int64_t carry = 0;
    for (int base = 1; base <= n; base += 32) {
        const int i = base + lane;
        int64_t v = i <= n ? x[i] : 0;
#pragma unroll
        for (int f = 1; f < 32; f <<= 1) {
            const int64_t u = __shfl_up_sync(0xffffffffu, v, f);
            if (lane >= f) v += u;
        }
        if (i <= n) x[i] = v + carry;
        carry += __shfl_sync(0xffffffffu, v, 31);
    }
}

inline bool cache_i4_ok(const pa_cache_i4_t *c, int layer, int n_kv_heads, int head_dim) {
    return c && c->base && (reinterpret_cast<uintptr_t>(c->base) & 255u) == 0 &&
           c->block_size == kBlockSize && c->n_kv_heads == n_kv_heads &&
           c->head_dim == head_dim && layer >= 0 && layer < c->layers && c->num_blocks > 0;
}

// Tile pair of (block 0, KV head 0) of a layer.
inline uint8_t *cache_i4_layer(const pa_cache_i4_t *c, int layer) {
    return c->base + (int64_t)layer * c->num_blocks * c->n_kv_heads * (20 * c->head_dim);
}

}  // namespace pa
