"""CPU oracle for the paged-KV / GQA / RoPE attention hot path.

TEST INFRASTRUCTURE ONLY.  This module is imported by the tests, by the
smoke check and by the CPU-baseline leg of the benchmark, never by the
product path.  It shares no code with the CUDA library: it restates, in plain
numpy (float64 for the attention arithmetic), what the pages define:

* "nano-vllm notes - Llama", sections prepare_prefill / prepare_decode:
  the flattened token stream, positions, cu_seqlens_q/k, slot_mapping,
  block_tables, context_lens (the worked examples 3,5,2 -> [0,3,8,10];
  prompts of 5 and 3 -> positions [0,1,2,3,4,0,1,2]; decode positions [5,3]
  with context_lens [6,4]).
* "nano-vllm notes - Llama", section allocate_kv_cache: the pool
  [2, layers, blocks, block_size, n_kv_heads, head_dim].
* "Meta Llama source deep-dive", section 3.3 (precompute_freqs_cis,
  apply_rotary_emb) and section 9 (RoPE derivation): adjacent pairs
  (x_2i, x_2i+1) rotated counter-clockwise by m * theta^(-2i/d).
* "Meta Llama source deep-dive", sections 3.4 (repeat_kv: Q head h reads KV
  head h // n_rep), 3.5 (scores = q k^T / sqrt(d), softmax, times V) and
  3.8 (causal mask with a cached prefix: zeros of width start_pos, then the
  upper triangle at -inf); "personal chatgpt 22 - llama2 generate",
  sections 2-3 (M_ij = 0 for j <= i, -inf otherwise; decode needs no mask).
* "llama2.zig", section 5.4: softmax subtracts the row maximum.

Every function here has a pin in tests/test_oracle_pins.py (worked examples,
closed forms, invariants, brute force against a library routine).

Pinned rounding of the RoPE step (the pages compute it in fp32 and store the
result back in the input dtype, "type_as"; they do not fix the order of the
fp32 operations, so this module fixes one and the CUDA path must match it bit
for bit):
  angle  = m * inv_freq_i           in float64, inv_freq_i = 1 / theta**(2i/d)
  c, s   = cos(angle), sin(angle)   in float64, each rounded once to float32
  x'     = fl32(fl32(x*c) - fl32(y*s))
  y'     = fl32(fl32(x*s) + fl32(y*c))          (no fused multiply-add)
  stored = round-to-nearest-even float16 of x', y'
"""

from __future__ import annotations

import math

import numpy as np


# ---------------------------------------------------------------------------
# Step a0: metadata of the flattened token stream
# ---------------------------------------------------------------------------

def cu_seqlens(lengths) -> np.ndarray:
    """Cumulative sequence lengths starting at 0 ("nano-vllm notes - Llama",
    prepare_prefill: cu_seqlens_q.append(cu_seqlens_q[-1] + seqlen_q))."""
    out = [0]
    for n in lengths:
        out.append(out[-1] + int(n))
    return np.asarray(out, dtype=np.int32)


def prefill_metadata(num_cached, num_new, block_tables, block_size):
    """Metadata for one prefill call ("nano-vllm notes - Llama",
    prepare_prefill).  For sequence s with `start` tokens cached and
    `seqlen_q` new ones: end = start + seqlen_q, seqlen_k = end, the new
    tokens sit at positions start..end-1, and each one is written to the slot
    block_table[s][pos // block_size] * block_size + pos % block_size.

    Returns dict(positions, cu_seqlens_q, cu_seqlens_k, slot_mapping,
    max_seqlen_q, max_seqlen_k)."""
    positions, slots, lq, lk = [], [], [], []
    for s in range(len(num_new)):
        start = int(num_cached[s])
        end = start + int(num_new[s])
        lq.append(end - start)
        lk.append(end)
        for pos in range(start, end):
            positions.append(pos)
            blk = int(block_tables[s][pos // block_size])
            slots.append(blk * block_size + pos % block_size)
    return dict(
        positions=np.asarray(positions, np.int32),
        cu_seqlens_q=cu_seqlens(lq),
        cu_seqlens_k=cu_seqlens(lk),
        slot_mapping=np.asarray(slots, np.int32),
        max_seqlen_q=max(lq) if lq else 0,
        max_seqlen_k=max(lk) if lk else 0,
    )


def decode_metadata(num_cached, block_tables, block_size):
    """Metadata for one decode step ("nano-vllm notes - Llama",
    prepare_decode): each sequence feeds its last token, at position
    num_cached[s]; after its K/V is appended the sequence holds
    context_lens[s] = num_cached[s] + 1 tokens (the page's example: positions
    [5,3], context_lens [6,4])."""
    positions, slots, ctx = [], [], []
    for s in range(len(num_cached)):
        pos = int(num_cached[s])
        positions.append(pos)
        ctx.append(pos + 1)
        blk = int(block_tables[s][pos // block_size])
        slots.append(blk * block_size + pos % block_size)
    return dict(
        positions=np.asarray(positions, np.int32),
        slot_mapping=np.asarray(slots, np.int32),
        context_lens=np.asarray(ctx, np.int32),
    )


# ---------------------------------------------------------------------------
# Step a1: rotary position embedding
# ---------------------------------------------------------------------------

def rope_inv_freq(head_dim: int, theta: float = 10000.0) -> list:
    """theta_i = 1 / theta**(2i/d) for i < d/2 ("Meta Llama source
    deep-dive", 3.3 precompute_freqs_cis; 9.2 theta_i = 10000^(-2i/d)).
    Python floats (IEEE double, C library pow)."""
    return [1.0 / (theta ** ((2 * i) / head_dim)) for i in range(head_dim // 2)]


def rope_cos_sin(position: int, head_dim: int, theta: float = 10000.0):
    """float64 angle m * theta_i, cos and sin from the C library, each rounded
    once to float32 (the pinned table entry for one position)."""
    inv = rope_inv_freq(head_dim, theta)
    c = np.empty(head_dim // 2, np.float32)
    s = np.empty(head_dim // 2, np.float32)
    for i, f in enumerate(inv):
        ang = float(position) * f
        c[i] = math.cos(ang)
        s[i] = math.sin(ang)
    return c, s


def rope_pinned(x16: np.ndarray, positions, head_dim: int, theta: float = 10000.0) -> np.ndarray:
    """Rotate each adjacent pair (x_2i, x_2i+1) of every head of token t by
    positions[t] * theta_i with the pinned float32 arithmetic of the module
    docstring; returns float16 of the same shape [T, n_heads, d]."""
    x16 = np.asarray(x16, np.float16)
    out = np.empty_like(x16)
    cache = {}
    for t in range(x16.shape[0]):
        m = int(positions[t])
        if m not in cache:
            cache[m] = rope_cos_sin(m, head_dim, theta)
        c, s = cache[m]
        xe = x16[t, :, 0::2].astype(np.float32)
        xo = x16[t, :, 1::2].astype(np.float32)
        re = (xe * c) - (xo * s)          # each op rounds to float32
        im = (xe * s) + (xo * c)
        out[t, :, 0::2] = re.astype(np.float16)
        out[t, :, 1::2] = im.astype(np.float16)
    return out


def rope_exact(x, positions, head_dim: int, theta: float = 10000.0) -> np.ndarray:
    """The same rotation entirely in float64, no rounding of the result:
    (x + i y) * e^{i m theta_i} ("Meta Llama source deep-dive", 9.3)."""
    x = np.asarray(x, np.float64)
    inv = np.asarray(rope_inv_freq(head_dim, theta), np.float64)
    out = np.empty_like(x)
    for t in range(x.shape[0]):
        ang = float(positions[t]) * inv
        c, s = np.cos(ang), np.sin(ang)
        xe, xo = x[t, :, 0::2], x[t, :, 1::2]
        out[t, :, 0::2] = xe * c - xo * s
        out[t, :, 1::2] = xe * s + xo * c
    return out


# ---------------------------------------------------------------------------
# Step a2: K/V write into the paged cache
# ---------------------------------------------------------------------------

def new_cache(layers, num_blocks, block_size, n_kv_heads, head_dim) -> np.ndarray:
    """The pool of "nano-vllm notes - Llama", allocate_kv_cache:
    [2, layers, num_blocks, block_size, n_kv_heads, head_dim] float16."""
    return np.zeros((2, layers, num_blocks, block_size, n_kv_heads, head_dim), np.float16)


def kv_write(cache: np.ndarray, layer: int, k16, v16, slot_mapping) -> None:
    """Store token t's K and V at physical slot slot_mapping[t]: block
    slot // block_size, row slot % block_size.  A negative slot means "no
    write" (a padding token).  In place, bit for bit."""
    bs = cache.shape[3]
    for t, slot in enumerate(slot_mapping):
        slot = int(slot)
        if slot < 0:
            continue
        cache[0, layer, slot // bs, slot % bs] = k16[t]
        cache[1, layer, slot // bs, slot % bs] = v16[t]


def gather_kv(cache: np.ndarray, layer: int, table_row, n_tokens: int):
    """Logical tokens 0..n_tokens-1 of one sequence, read through its block
    table: K, V float64 [n_tokens, n_kv_heads, d]."""
    bs = cache.shape[3]
    K = np.empty((n_tokens,) + cache.shape[4:], np.float64)
    V = np.empty_like(K)
    for lb in range((n_tokens + bs - 1) // bs):      # logical block lb
        blk = int(table_row[lb])
        rows = min(bs, n_tokens - lb * bs)
        K[lb * bs:lb * bs + rows] = cache[0, layer, blk, :rows]
        V[lb * bs:lb * bs + rows] = cache[1, layer, blk, :rows]
    return K, V


# ---------------------------------------------------------------------------
# Steps a3 / a4: attention
# ---------------------------------------------------------------------------

def _softmax_rows(scores: np.ndarray) -> np.ndarray:
    """Row softmax with the row maximum subtracted first ("llama2.zig" 5.4).
    Entries at -inf get weight 0."""
    m = scores.max(axis=-1, keepdims=True)
    e = np.exp(scores - m)
    return e / e.sum(axis=-1, keepdims=True)


def attention_prefill(q16, cache, layer, cu_seqlens_q, cu_seqlens_k, block_tables,
                      n_heads, n_kv_heads, scale=None, seqs=None) -> np.ndarray:
    """Varlen causal attention over a flattened stream.

    Sequence s owns query rows cu_seqlens_q[s]..cu_seqlens_q[s+1]-1 and has
    seqlen_k = cu_seqlens_k[s+1]-cu_seqlens_k[s] keys, of which the first
    p = seqlen_k - seqlen_q are a cached prefix.  Query row i sits at
    absolute position p + i and sees keys j <= p + i: the prefix block of
    zeros followed by the causal triangle ("Meta Llama source deep-dive",
    3.8; M_ij of "personal chatgpt 22", section 2).  Q head h uses KV head
    h // (n_heads / n_kv_heads) (repeat_kv, 3.4).  scores = q.k * scale with
    scale = 1/sqrt(d) by default, softmax, times V (3.5).  float64.

    q16: [T, n_heads, d] (already rotated).  Returns float64 [T, n_heads, d];
    rows of sequences not in `seqs` (when given) are left NaN."""
    T, H, d = q16.shape
    assert H == n_heads and n_heads % n_kv_heads == 0
    g = n_heads // n_kv_heads
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    out = np.full((T, H, d), np.nan)
    B = len(cu_seqlens_q) - 1
    for s in (range(B) if seqs is None else seqs):
        q0, q1 = int(cu_seqlens_q[s]), int(cu_seqlens_q[s + 1])
        lq = q1 - q0
        lk = int(cu_seqlens_k[s + 1]) - int(cu_seqlens_k[s])
        if lq == 0:
            continue
        p = lk - lq
        K, V = gather_kv(cache, layer, block_tables[s], lk)
        i = np.arange(lq)[:, None]
        j = np.arange(lk)[None, :]
        mask = np.where(j <= p + i, 0.0, -np.inf)
        Q = q16[q0:q1].astype(np.float64)
        for h in range(H):
            kv = h // g
            scores = (Q[:, h, :] @ K[:, kv, :].T) * scale + mask
            out[q0:q1, h, :] = _softmax_rows(scores) @ V[:, kv, :]
    return out


def attention_decode(q16, cache, layer, block_tables, context_lens,
                     n_heads, n_kv_heads, scale=None, seqs=None) -> np.ndarray:
    """Single-token decode: the query of sequence s (at position
    context_lens[s]-1, its K/V already appended) attends to all
    context_lens[s] cached keys; no mask is needed because every cached key
    is in its past ("personal chatgpt 22", section 3; "Meta Llama source
    deep-dive", 3.8 decode branch).  Written out per head as a plain weighted
    sum, independently of attention_prefill.

    q16: [B, n_heads, d].  Returns float64 [B, n_heads, d] (NaN rows for
    sequences not in `seqs`)."""
    B, H, d = q16.shape
    g = n_heads // n_kv_heads
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    out = np.full((B, H, d), np.nan)
    for s in (range(B) if seqs is None else seqs):
        n = int(context_lens[s])
        K, V = gather_kv(cache, layer, block_tables[s], n)
        for h in range(H):
            kv = h // g
            qv = q16[s, h].astype(np.float64)
            sc = (K[:, kv, :] @ qv) * scale          # [n]
            w = np.exp(sc - sc.max())
            out[s, h] = (w @ V[:, kv, :]) / w.sum()
    return out


# ---------------------------------------------------------------------------
# NEXT-4: int8 KV cache ("Meta Llama source deep-dive", 8.4: a quantised KV
# cache stored as int8 saves memory; the page gives no scheme, so this is
# the reading the CUDA path also follows)
# ---------------------------------------------------------------------------
#
# Each (token, KV head) row x of head_dim fp16 values (K after the pinned
# RoPE, V as given) is stored as int8 codes and one float32 scale:
#   amax  = max_i |x_i|                       (exact in float32)
#   scale = fl32(amax / 127)                  (0 when amax is 0)
#   q_i   = clamp(rint(fl32(x_i / scale)), -127, 127)   rint: ties to even
# and read back as q_i * scale.  Layout: codes [2, layers, blocks,
# block_size, n_kv_heads, head_dim] int8; scales [2, layers, blocks,
# n_kv_heads, block_size] float32 (a block's 16 scales of one head are
# contiguous).

def kv_quantize_int8(x16):
    """Rows of the last axis -> (codes int8, scales float32 [...])."""
    x = np.asarray(x16, np.float16).astype(np.float32)
    amax = np.abs(x).max(axis=-1)
    scale = (amax / np.float32(127.0)).astype(np.float32)
    safe = np.where(scale > 0, scale, np.float32(1.0)).astype(np.float32)
    r = np.rint((x / safe[..., None]).astype(np.float32))
    codes = np.clip(r, -127, 127).astype(np.int8)
    codes[scale == 0] = 0
    return codes, scale


def new_cache_i8(layers, num_blocks, block_size, n_kv_heads, head_dim):
    codes = np.zeros((2, layers, num_blocks, block_size, n_kv_heads, head_dim), np.int8)
    scales = np.zeros((2, layers, num_blocks, n_kv_heads, block_size), np.float32)
    return codes, scales


def kv_write_i8(codes, scales, layer: int, k16, v16, slot_mapping) -> None:
    """Quantise token t's K and V rows and store them at slot
    slot_mapping[t] (negative: no write)."""
    bs = codes.shape[3]
    kq, ks = kv_quantize_int8(k16)
    vq, vs = kv_quantize_int8(v16)
    for t, slot in enumerate(slot_mapping):
        slot = int(slot)
        if slot < 0:
            continue
        b, r = slot // bs, slot % bs
        codes[0, layer, b, r], codes[1, layer, b, r] = kq[t], vq[t]
        scales[0, layer, b, :, r], scales[1, layer, b, :, r] = ks[t], vs[t]


def dequantize_cache_i8(codes, scales) -> np.ndarray:
    """The float64 cache the int8 one stands for: q * scale."""
    s = np.swapaxes(scales, -1, -2)[..., None].astype(np.float64)  # [..., bs, Hk, 1]
    return codes.astype(np.float64) * s


def attention_decode_i8(q16, codes, scales, layer, block_tables, context_lens,
                        n_heads, n_kv_heads, scale=None, seqs=None) -> np.ndarray:
    """Decode against the int8 cache: the decode formula on the values the
    codes and scales stand for."""
    return attention_decode(q16, dequantize_cache_i8(codes, scales), layer, block_tables,
                            context_lens, n_heads, n_kv_heads, scale=scale, seqs=seqs)


# ---------------------------------------------------------------------------
# 4-bit KV cache (the quantised cache of "Meta Llama source deep-dive", 8.4;
# the page gives no scheme, so this is the reading the CUDA path also follows)
# ---------------------------------------------------------------------------
#
# Each (token, KV head) row of head_dim fp16 values (K after the pinned RoPE,
# V as given) is cut into groups of 32; a group x stands as
#   m   = min x (fp16),  s = fl32((max x - m) / 15) rounded up to fp16,
#   c_i = clamp(rint(fl32(fl32(x_i - m) / s)), 0, 15), 0 where s is 0,
# and reads back as m + s c_i.  A group with a NaN or an infinity stores
# m = NaN (0x7fff), s = 0 and codes 0.  Tiles: see kv_i4_places.

def kv_quantize_int4(x16):
    """Rows [..., d] -> codes uint8 [..., d], steps and least values fp16 [..., d/32]."""
    x = np.asarray(x16, np.float16)
    x = x.reshape(*x.shape[:-1], -1, 32).astype(np.float32)
    odd = ~np.isfinite(x).all(axis=-1)
    x = np.where(odd[..., None], np.float32(0), x)
    m = x.min(axis=-1) + np.float32(0)  # -0 becomes +0
    r = (x.max(axis=-1) - m) / np.float32(15.0)
    s = r.astype(np.float16)
    s = np.where(s.astype(np.float32) < r, np.nextafter(s, np.float16(np.inf)), s)
    s32 = s.astype(np.float32)
    safe = np.where(s32 > 0, s32, np.float32(1))
    c = np.rint((x - m[..., None]) / safe[..., None])
    c = np.where(s32[..., None] > 0, np.clip(c, 0, 15), 0).astype(np.uint8)
    nan = np.uint16(0x7FFF).view(np.float16)
    s, m = np.where(odd, np.float16(0), s), np.where(odd, nan, m.astype(np.float16))
    return c.reshape(*np.shape(x16)), s.astype(np.float16), m.astype(np.float16)


def kv_i4_places(d, is_v):
    """Where a tile of 16 rows keeps things: (byte, shift) of the code of (row,
    value) [16, d], and the fp16 index, counted from the end of the 8 d bytes of
    codes, of the step and the least value of (row, group) [16, d/32]."""
    G = d // 32
    byte, shift = np.zeros((16, d), np.int64), np.zeros((16, d), np.int64)
    step, least = np.zeros((16, G), np.int64), np.zeros((16, G), np.int64)
    for j in range(16):
        for g in range(G):
            step[j, g] = 4 * (G * (j % 8 // 2) + g) + 2 * (j // 8) + j % 2
            least[j, g] = 16 * G + (step[j, g] if is_v else G * j + g)
            for y in range(32):
                if is_v:
                    unit = G * (4 * (8 * (j // 8) + y // 4) + j % 8 // 2) + g
                    byte[j, 32 * g + y] = 2 * (2 * unit + j % 2) + y % 4 // 2
                else:
                    byte[j, 32 * g + y] = j * d // 2 + y // 8 * 4 * G + 4 * g + y % 8 // 2
                shift[j, 32 * g + y] = 4 * (y % 2)
    return byte, shift, step, least


def new_cache_i4(layers, num_blocks, n_kv_heads, head_dim):
    return np.zeros((layers, num_blocks, n_kv_heads, 2, 10 * head_dim), np.uint8)


def kv_write_i4(tiles, layer: int, k16, v16, slot_mapping) -> None:
    """Quantise token t's K and V rows and store them at slot slot_mapping[t]
    (negative: no write)."""
    d = tiles.shape[-1] // 10
    for kv, x in ((0, k16), (1, v16)):
        byte, shift, step, least = kv_i4_places(d, kv == 1)
        codes, s, m = kv_quantize_int4(x)
        for t, slot in enumerate(slot_mapping):
            slot = int(slot)
            if slot < 0:
                continue
            j = slot % 16
            for h in range(x.shape[1]):
                tile = tiles[layer, slot // 16, h, kv]
                for y in range(d):
                    keep = 0xF0 if shift[j, y] == 0 else 0x0F
                    tile[byte[j, y]] = (tile[byte[j, y]] & keep) | (int(codes[t, h, y]) << shift[j, y])
                params = tile[8 * d:].view(np.float16)
                params[step[j]], params[least[j]] = s[t, h], m[t, h]


def pack_cache_i4(cache16):
    """The 4-bit form of an fp16 pool [2, L, NB, 16, Hk, d], every row quantised."""
    two, L, NB, bs, Hk, d = cache16.shape
    tiles = np.zeros((L, NB, Hk, 2, 10 * d), np.uint8)
    for kv in (0, 1):
        byte, shift, step, least = kv_i4_places(d, kv == 1)
        codes, s, m = kv_quantize_int4(np.swapaxes(cache16[kv], 2, 3))  # [L, NB, Hk, 16, d]
        packed = np.zeros((L, NB, Hk, 8 * d), np.uint8)
        for nib in (0, 4):
            at = shift == nib
            packed[..., byte[at]] |= codes[..., at] << np.uint8(nib)
        params = np.zeros((L, NB, Hk, d), np.float16)
        params[..., step], params[..., least] = s, m
        tiles[..., kv, :8 * d] = packed
        tiles[..., kv, 8 * d:] = params.view(np.uint8)
    return tiles


def dequantize_cache_i4(tiles) -> np.ndarray:
    """The float64 pool [2, L, NB, 16, Hk, d] the tiles stand for: m + s c."""
    L, NB, Hk, two, n = tiles.shape
    d = n // 10
    out = np.empty((2, L, NB, 16, Hk, d))
    for kv in (0, 1):
        byte, shift, step, least = kv_i4_places(d, kv == 1)
        x = np.ascontiguousarray(tiles[..., kv, :])
        codes = (x[..., byte] >> shift) & 15
        p = x[..., 8 * d:].view(np.float16).astype(np.float64)
        val = np.repeat(p[..., least], 32, -1) + np.repeat(p[..., step], 32, -1) * codes
        out[kv] = np.swapaxes(val, 2, 3)
    return out


def read_rows_i4(values64) -> np.ndarray:
    """fp16 rows as the library reads them back: the value (exact in float64)
    saturated and rounded once to fp16."""
    return np.minimum(values64, 65504).astype(np.float16)


# ---------------------------------------------------------------------------
# Long contexts: other rotary layouts and scaled tables, decode's attention
# weights, eviction by them (a shared prefix changes nothing that is computed:
# attention_decode is its oracle)
# ---------------------------------------------------------------------------

def rope_scaled_frequencies(rotary_dim, theta=10000.0, scaling=None, factor=1.0,
                            original_positions=0, low=1.0, high=4.0, attention=0.0):
    """(frequencies of the rotary_dim / 2 pairs, magnitude of the table's entries),
    Python floats."""
    r, n = rotary_dim, rotary_dim // 2
    magnitude = attention or 1.0
    if scaling == "ntk":
        theta = theta * factor ** (r / (r - 2))
    f = [1.0 / theta ** (2 * i / r) for i in range(n)]
    if scaling in (None, "ntk"):
        return f, magnitude
    if scaling == "linear":
        return [x / factor for x in f], magnitude
    turns = original_positions / (2 * math.pi)
    if scaling == "bands":
        keep = [(turns * x - low) / (high - low) for x in f]
    else:
        def pair(t):  # the pair that turns t times over the original positions
            return r * math.log(turns / t) / (2 * math.log(theta))
        first, last = max(math.floor(pair(high)), 0), min(math.ceil(pair(low)), r - 1)
        width = last - first if last > first else 0.001
        keep = [1 - (i - first) / width for i in range(n)]
        magnitude = attention or 0.1 * math.log(factor) + 1.0
    keep = [min(max(k, 0.0), 1.0) for k in keep]
    return [x * k + x / factor * (1 - k) for x, k in zip(f, keep)], magnitude


def rope_scaled_table(max_positions, rotary_dim, **scaling):
    """float32 [max_positions, rotary_dim / 2, 2] {cos, sin}, rounded once from
    float64."""
    f, a = rope_scaled_frequencies(rotary_dim, **scaling)
    ang = np.arange(max_positions, dtype=np.float64)[:, None] * np.asarray(f)
    return np.stack([a * np.cos(ang), a * np.sin(ang)], -1).astype(np.float32)


def rope_layout_pinned(x16, positions, table, half):
    """rope_pinned with the pairs of a layout among the first 2 * table.shape[1]
    values, the angles from a table; the other values unchanged."""
    x16 = np.asarray(x16, np.float16)
    r = 2 * table.shape[1]
    out = x16.copy()
    a, b = (slice(0, r // 2), slice(r // 2, r)) if half else (slice(0, r, 2), slice(1, r, 2))
    x, y = x16[..., a].astype(np.float32), x16[..., b].astype(np.float32)
    c, s = (table[np.asarray(positions)][:, None, :, i] for i in (0, 1))
    out[..., a] = ((x * c) - (y * s)).astype(np.float16)  # each op rounds to float32
    out[..., b] = ((x * s) + (y * c)).astype(np.float16)
    return out


def decode_weights(q16, cache, layer, block_tables, context_lens, n_heads, n_kv_heads, scale=None):
    """For every sequence, float64 [n_kv_heads, context_lens[s]]: each cached token's
    softmax weight, summed over the Q heads of the KV head."""
    B, H, d = q16.shape
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    out = []
    for s in range(B):
        n = int(context_lens[s])
        K, _ = gather_kv(cache, layer, block_tables[s], n)
        w = np.zeros((n_kv_heads, n))
        for h in range(H):
            kv = h // (H // n_kv_heads)
            w[kv] += _softmax_rows((K[:, kv] @ q16[s, h].astype(np.float64)) * scale)
        out.append(w)
    return out


def evict_keep(weights, budget, sinks, recent):
    """Tokens kept of a (sequence, KV head) with the given weights, in order: the first
    `sinks`, the last `recent`, and the largest of the others (NaN the smallest, of equal
    ones the earlier), `budget` in all."""
    n = len(weights)
    if n <= budget:
        return list(range(n))
    fixed = list(range(sinks)) + list(range(n - recent, n))
    others = sorted(range(sinks, n - recent),
                    key=lambda t: (np.isnan(weights[t]), -weights[t] if weights[t] == weights[t] else 0, t))
    return sorted(fixed + others[:budget - sinks - recent])


def evict(cache, layer, block_tables, context_lens, weights, budget, sinks, recent, out_tables):
    """In place on `cache` and `weights` [B, n_kv_heads, stride]: rows and weights of the
    kept tokens move to the first places.  Returns the new lengths."""
    bs = cache.shape[3]
    old, lens = cache.copy(), np.asarray(context_lens).copy()
    for s, n in enumerate(context_lens):
        n = int(n)
        for h in range(weights.shape[1]):
            kept = evict_keep(weights[s, h, :n], budget, sinks, recent)
            moved = weights[s, h, kept]
            weights[s, h, :n] = 0
            weights[s, h, :len(kept)] = moved
            for i, t in enumerate(kept):
                cache[:, layer, out_tables[s][i // bs], i % bs, h] = \
                    old[:, layer, block_tables[s][t // bs], t % bs, h]
        lens[s] = min(n, budget)
    return lens
