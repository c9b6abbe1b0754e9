"""Cases of the 4-bit KV cache's operators: quantising new tokens as they are
written and reading them back, reading a cached history back, decode attention
and varlen prefill attention over the cache.

`run` computes a case with elementary torch operations in 32 bits (`own` false)
or with the library's entry points (`own` true); `exact` computes it in 64 bits
from the definition.

The cache holds, for every (token, KV head) row x of K (rotated) and of V and
every group of 32 of its values, the group's least value m (fp16), a step
s = (max - min) / 15 rounded up to fp16, and for each value the 4-bit code
c = clamp(rint((x - m) / s), 0, 15) (0 where s is 0); it stands for m + s c.
A block of 16 tokens of one KV head is a K tile and a V tile of 10 d bytes each:
8 d bytes of codes, then the steps and the least values.  With G = d / 32, the
code of token j, value x = 32 g + y, is the nibble
    K  y % 2 of byte  j d/2 + (y / 8) 4 G + 4 g + (y % 8) / 2
    V  y % 2 of byte  2 (2 (G (4 (8 (j / 8) + y / 4) + (j % 8) / 2) + g) + j % 2) + (y % 4) / 2
and the step of (j, g) is the fp16 4 (G ((j % 8) / 2) + g) + 2 (j / 8) + j % 2 after
the codes; the least values follow the 16 G steps, for K at G j + g and for V in
the order of the steps.  The pool is [layers][blocks][KV heads][K, V][10 d].
"""

import math
import random

import torch

own = False

DEV = "cuda"
HEADS = [(4, 2, 64), (14, 2, 64), (32, 4, 64), (12, 4, 128), (16, 8, 128), (8, 1, 128),
         (32, 8, 128), (64, 8, 128), (32, 32, 128), (40, 40, 128)]  # (Q heads, KV heads, d)


def listed():
    def case(name, kind, heads, kv_heads, d, batch, new, past, mix):
        return dict(name=name, kind=kind, heads=heads, kv_heads=kv_heads, head_dim=d, batch=batch,
                    new_lo=new[0], new_hi=new[1], past_lo=past[0], past_hi=past[1], mix=mix)

    return [
        # decode attention, one new token per sequence: three short sequences of a
        # small model (latency alone)
        case("decode_small", "decode", 4, 2, 64, 3, (1, 1), (2, 8), 1),
        # one long sequence, the interactive user with a long document
        case("decode_one_long", "decode", 64, 8, 128, 1, (1, 1), (32767, 32767), 2),
        # the serving batches of the benchmark: grouped heads, one KV head per Q head
        case("decode_gqa", "decode", 64, 8, 128, 32, (1, 1), (4096, 4096), 3),
        case("decode_mha", "decode", 32, 32, 128, 32, (1, 1), (2048, 2048), 4),
        # continuous batching: histories from 16 to 16384 tokens side by side
        case("decode_ragged", "decode", 32, 8, 128, 64, (1, 1), (16, 16384), 5),
        # the new tokens of one decode step, quantised as they are written, read back
        case("store_step", "store", 32, 8, 128, 256, (1, 1), (16, 1000), 6),
        # the new tokens of a batch of prompts
        case("store_prompts", "store", 64, 8, 128, 16, (128, 2048), (0, 1024), 7),
        # histories read back as fp16 rows: a small model's, and a serving batch's
        case("read_small_heads", "read", 32, 4, 64, 7, (0, 0), (1, 700), 8),
        case("read_batch", "read", 32, 8, 128, 32, (0, 0), (1000, 5000), 9),
        # prompts that attend to themselves and to a cached prefix: the smallest, grouped
        # heads, one KV head per Q head
        case("prefill_small", "prefill", 4, 2, 64, 3, (2, 5), (0, 0), 10),
        case("prefill_gqa", "prefill", 32, 8, 128, 6, (400, 1500), (500, 8000), 11),
        case("prefill_mha", "prefill", 40, 40, 128, 8, (200, 2048), (100, 1024), 12),
    ]


def _between(rng, lo, hi):
    """A whole number, uniform over its logarithm."""
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["decode", "decode", "store", "read", "prefill"])
    heads, kv_heads, d = rng.choice(HEADS)
    c = dict(kind=kind, heads=heads, kv_heads=kv_heads, head_dim=d, new_lo=1, new_hi=1,
             past_lo=0, past_hi=0, mix=rng.randrange(1 << 20))
    if kind == "prefill":
        c["new_hi"] = _between(rng, 1, 2000)
        c["past_hi"] = rng.choice([0, _between(rng, 1, 8000)])
        most = 5e8 / (heads * c["new_hi"] * (c["new_hi"] + c["past_hi"]))  # padded scores
        c["batch"] = _between(rng, 1, max(1, min(32, int(most))))
        c["new_lo"] = _between(rng, 1, c["new_hi"])
        return c
    size = {"decode": 2.6e8, "read": 1.2e8, "store": 2e7}[kind] / (kv_heads * d)  # padded tokens
    if kind == "store":
        c["new_hi"] = rng.choice([1, _between(rng, 1, 2048)])
        c["batch"] = _between(rng, 1, max(1, min(256, int(size / c["new_hi"]))))
        c["new_lo"] = _between(rng, 1, c["new_hi"])
        c["past_hi"] = rng.choice([0, _between(rng, 1, 1000)])
        return c
    c["past_hi"] = _between(rng, 1, 32767)
    c["batch"] = _between(rng, 1, max(1, min(200, int(size / (c["past_hi"] + 1)))))
    c["past_lo"] = _between(rng, 1, c["past_hi"])
    if kind == "read":
        c["new_lo"] = c["new_hi"] = 0
    return c


def _lengths(case):
    """Each sequence's cached and new tokens, by the case alone."""
    rng = random.Random(case["mix"])

    def some(lo, hi):
        if lo == hi:
            return [lo] * case["batch"]
        return [min(hi, max(lo, _between(rng, max(lo, 1), hi))) if lo or rng.random() < 0.8 else 0
                for _ in range(case["batch"])]

    return some(case["past_lo"], case["past_hi"]), some(case["new_lo"], case["new_hi"])


def work(case):
    past, new = _lengths(case)
    H, Hk, d = case["heads"], case["kv_heads"], case["head_dim"]
    held = 1.25 * d * Hk  # bytes of one token's K and V in the cache
    T, N = sum(new), sum(past) + sum(new)
    if case["kind"] == "decode":
        return dict(bytes=N * held + 4 * T * H * d + N / 4, flops=4 * H * d * N)
    if case["kind"] == "read":
        return dict(bytes=N * (held + 4 * d * Hk) + N / 4, flops=2 * N * 2 * d * Hk)
    if case["kind"] == "store":  # Q and the RoPE rows in, K and V in, all of them out, the cache
        return dict(bytes=T * (4 * H * d + 4 * d + 8 * d * Hk + held + 8), flops=T * 12 * (H + Hk) * d)
    pairs = sum(n * p + n * (n + 1) // 2 for p, n in zip(past, new))
    return dict(bytes=N * held + 4 * T * H * d + N / 4, flops=4 * d * H * pairs)


# ------------------------------------------------------------------ inputs

def _quantise(x):
    """Codes (uint8), steps and least values (fp16) of fp16 rows [..., d]."""
    x = x.float().unflatten(-1, (-1, 32))
    m = x.amin(-1, keepdim=True)
    # (a division by a tensor: by a Python number it is a product with the rounded 1 / 15)
    r = (x.amax(-1, keepdim=True) - m) / torch.full_like(m, 15.0)
    s = r.half()
    s = torch.where(s.float() < r, (s.view(torch.int16) + 1).view(torch.float16), s)
    f = s.float()
    c = torch.where(f > 0, ((x - m) / torch.where(f > 0, f, 1.0)).round().clamp(0, 15), 0.0)
    return c.to(torch.uint8), s, m.half()


def _pack(k, v):
    """Tiles [..., 2, 10 d] (uint8) of fp16 K and V rows [..., 16, d]."""
    lead, d = k.shape[:-2], k.shape[-1]
    G = d // 32
    n = len(lead)
    out = []
    for x, is_k in ((k, True), (v, False)):
        c, s, m = _quantise(x)  # [..., 16, G, 32], [..., 16, G, 1]
        s, m = s.squeeze(-1), m.squeeze(-1)
        at = list(range(n))
        if is_k:  # [16, G, t, b, 2] -> [16, t, G, b]
            c = c.unflatten(-1, (4, 4, 2)).permute(*at, n, n + 2, n + 1, n + 3, n + 4)
        else:  # [j / 8, t, j % 2, G, u, b, 2] -> [j / 8, u, t, G, j % 2, b]
            c = c.unflatten(n, (2, 4, 2)).unflatten(-1, (8, 2, 2))
            c = c.permute(*at, n, n + 4, n + 1, n + 3, n + 2, n + 5, n + 6)
        c = (c[..., 0] | (c[..., 1] << 4)).reshape(*lead, 8 * d)

        def by_quarter(y):  # [j / 8, t, j % 2, G] -> [t, G, j / 8, j % 2]
            return y.unflatten(n, (2, 4, 2)).permute(*at, n + 1, n + 3, n, n + 2).reshape(*lead, 16 * G)

        p = torch.cat([by_quarter(s), m.reshape(*lead, 16 * G) if is_k else by_quarter(m)], -1)
        out.append(torch.cat([c, p.contiguous().view(torch.uint8)], -1))
    return torch.stack(out, -2)


def prepare(case, seed):
    past, new = _lengths(case)
    H, Hk, d, B = case["heads"], case["kv_heads"], case["head_dim"], case["batch"]
    rng = torch.Generator(device=DEV).manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, device=DEV, generator=rng)

    def ints(x):
        return torch.tensor(x, dtype=torch.int32, device=DEV)

    total = [p + n for p, n in zip(past, new)]
    need = [-(-t // 16) for t in total]
    blocks = sum(need) + sum(need) // 10 + 1
    order = torch.randperm(blocks, device=DEV, generator=rng).int()
    width = max(max(need), 1)
    have = ints(need)
    col = torch.arange(width, device=DEV)
    ahead = (have.cumsum(0) - have).long()
    table = torch.where(col < have[:, None],
                        order[(ahead[:, None] + col).clamp(max=blocks - 1)], -1).int()
    # K with a few channels of large values, as attention layers have them
    gain = torch.where(torch.rand(Hk, d, device=DEV, generator=rng) < 0.03, 4.0, 1.0)
    pool = torch.zeros(1, blocks, Hk, 2, 10 * d, dtype=torch.uint8, device=DEV)
    if case["kind"] != "store":
        step = max(1, (1 << 27) // (Hk * 16 * d))
        for b in range(0, blocks, step):
            n = min(step, blocks - b)
            k = (normal(n, Hk, 16, d) * gain[:, None]).half()
            pool[0, b:b + n] = _pack(k, normal(n, Hk, 16, d).half())
    st = dict(case=case, pool=pool, table=table, lengths=ints(total), handles={})
    T = sum(new)
    if T:
        st["q"] = normal(T, H, d).half()
        st["out"] = torch.empty_like(st["q"])
    if case["kind"] == "prefill":
        st["cu_q"] = ints([sum(new[:i]) for i in range(B + 1)])
        st["cu_k"] = ints([sum(total[:i]) for i in range(B + 1)])
        st["max_new"] = max(new)
        st["used_blocks"] = sum(need)
    if case["kind"] == "store":
        st["k"] = (normal(T, Hk, d) * gain).half()
        st["v"] = normal(T, Hk, d).half()
        seq = torch.repeat_interleave(torch.arange(B, device=DEV), ints(new))
        start = ints(new).cumsum(0) - ints(new)
        pos = ints(past)[seq] + torch.arange(T, device=DEV) - start[seq]
        st["pos"] = pos.int()
        st["slots"] = (table[seq, pos // 16] * 16 + pos % 16).int()
        ang = torch.arange(max(total), device=DEV, dtype=torch.float64)[:, None] / 10000.0 ** (
            torch.arange(0, d, 2, device=DEV, dtype=torch.float64) / d)
        st["rope"] = torch.stack([ang.cos(), ang.sin()], -1).float()
        st["first"], st["lengths"] = ints(past), ints(new)
    if case["kind"] in ("store", "read"):
        rows = sum(new) if case["kind"] == "store" else sum(total)
        st["row_starts"] = (st["lengths"].cumsum(0) - st["lengths"]).int()
        st["k_out"] = torch.empty(rows, Hk, d, dtype=torch.float16, device=DEV)
        st["v_out"] = torch.empty(rows, Hk, d, dtype=torch.float16, device=DEV)
    return st


# ------------------------------------------------------------------ plain form

def _unpack(tiles, kv):
    """fp32 values m + s c, [..., 16, d], of the K (kv 0) or V (kv 1) tiles of [..., 2, 10 d]."""
    x = tiles[..., kv, :]
    lead, n, d = x.shape[:-1], x.dim() - 1, x.shape[-1] // 10
    G = d // 32
    at = list(range(n))
    c = torch.stack([x[..., :8 * d] & 15, x[..., :8 * d] >> 4], -1)
    if kv == 0:
        c = c.reshape(*lead, 16, 4, G, 4, 2).permute(*at, n, n + 2, n + 1, n + 3, n + 4)
    else:
        c = c.reshape(*lead, 2, 8, 4, G, 2, 2, 2)
        c = c.permute(*at, n, n + 2, n + 4, n + 3, n + 1, n + 5, n + 6)
    c = c.reshape(*lead, 16, G, 32).float()
    p = x[..., 8 * d:].contiguous().view(torch.float16).float().reshape(*lead, 2, 16 * G)

    def by_token(y):
        return y.reshape(*lead, 4, G, 2, 2).permute(*at, n + 2, n, n + 3, n + 1).reshape(*lead, 16, G)

    s = by_token(p[..., 0, :])
    m = p[..., 1, :].reshape(*lead, 16, G) if kv == 0 else by_token(p[..., 1, :])
    return (s[..., None] * c + m[..., None]).reshape(*lead, 16, d)


def _history(st, kv):
    """fp32 rows [B, Hk, width * 16, d] of every sequence, padded."""
    tiles = st["pool"][0][st["table"].clamp(min=0).long()]  # [B, width, Hk, 2, 10 d]
    return _unpack(tiles, kv).permute(0, 2, 1, 3, 4).flatten(2, 3)


def _fp16_rows(x):
    """Rounded to fp16, saturated."""
    return x.clamp(-65504.0, 65504.0).half()


def _attend(q, k, v, ok):
    """q [B, Hk, n, d], k and v [B, Hk, N, d], ok [B, 1, n or 1, N]: softmax(q k^T / sqrt(d)) v."""
    x = torch.matmul(q * (1.0 / math.sqrt(q.shape[-1])), k.transpose(-1, -2))
    x = torch.where(ok, x, -math.inf)
    x = torch.exp(x - x.amax(-1, keepdim=True))
    return torch.matmul(x, v) / x.sum(-1, keepdim=True)


def _plain(st):
    case = st["case"]
    H, Hk, d, B = case["heads"], case["kv_heads"], case["head_dim"], case["batch"]
    g = H // Hk
    if case["kind"] == "decode":
        k, v = _history(st, 0), _history(st, 1)
        ok = torch.arange(k.shape[2], device=DEV) < st["lengths"][:, None]
        o = _attend(st["q"].float().view(B, Hk, g, d), k, v, ok[:, None, None])
        return {"out": o.reshape(B, H, d).half()}
    if case["kind"] == "read":
        rows = torch.arange(st["table"].shape[1] * 16, device=DEV) < st["lengths"][:, None]
        return {"k": _fp16_rows(_history(st, 0).transpose(1, 2)[rows]),
                "v": _fp16_rows(_history(st, 1).transpose(1, 2)[rows])}
    if case["kind"] == "store":
        cs = st["rope"][st["pos"].long()][:, None]  # [T, 1, d / 2, 2]
        c, s = cs[..., 0], cs[..., 1]

        def rotate(x):
            x = x.float().unflatten(-1, (-1, 2))
            a, b = x[..., 0], x[..., 1]
            return torch.stack([a * c - b * s, a * s + b * c], -1).flatten(-2).half()

        def there_and_back(x):
            y, s, m = _quantise(x)
            return _fp16_rows((s.float() * y.float() + m.float()).flatten(-2))

        return {"q": rotate(st["q"]), "k": there_and_back(rotate(st["k"])),
                "v": there_and_back(st["v"])}
    # prefill: query i of a sequence sees its first past + i + 1 tokens; K and V as read back
    k, v = _fp16_rows(_history(st, 0)).float(), _fp16_rows(_history(st, 1)).float()
    n = st["cu_q"][1:] - st["cu_q"][:-1]
    i = torch.arange(st["max_new"], device=DEV)
    real = i < n[:, None]  # [B, max_new]
    row = torch.where(real, st["cu_q"][:-1, None] + i, 0).long()
    q = st["q"][row].float().unflatten(2, (Hk, g)).permute(0, 2, 3, 1, 4).flatten(2, 3)
    last = st["lengths"][:, None] - n[:, None] + i
    ok = torch.arange(k.shape[2], device=DEV) <= last[..., None]  # [B, max_new, N]
    ok = ok.repeat(1, g, 1)[:, None]
    o = _attend(q, k, v, ok).unflatten(2, (g, -1)).permute(0, 3, 1, 2, 4).flatten(2, 3)
    return {"out": o[real].half()}


def _handles(st):
    """What a user's program makes once: the pool's descriptor and the workspaces."""
    from paged_kv_gqa_rope_gb300 import pa
    case, h = st["case"], st["handles"]
    H, Hk, d, B = case["heads"], case["kv_heads"], case["head_dim"], case["batch"]
    if not h:
        h["cache"] = pa.CacheI4(1, st["pool"].shape[1], Hk, d, buffer=st["pool"].view(-1))
        if case["kind"] == "decode":
            h["ws"] = pa.decode_i4_workspace(B, H, Hk, d)
        if case["kind"] == "prefill":
            h["ws"] = pa.prefill_i4_workspace(st["used_blocks"], B, st["table"].shape[1], Hk, d)
    return pa, h


def run(st):
    if not own:
        return _plain(st)
    pa, h = _handles(st)
    case = st["case"]
    if case["kind"] == "decode":
        return {"out": pa.decode_i4(st["q"], h["cache"], st["table"], st["lengths"], h["ws"],
                                    case["kv_heads"], out=st["out"])}
    if case["kind"] == "prefill":
        return {"out": pa.prefill_varlen_i4(st["q"], h["cache"], st["cu_q"], st["cu_k"],
                                            st["table"], st["max_new"], case["kv_heads"], h["ws"],
                                            out=st["out"])}
    got = {}
    if case["kind"] == "store":
        got["q"] = pa.rope_kv_write_i4(st["q"], st["k"], st["v"], st["pos"], st["slots"],
                                       st["rope"], h["cache"], q_out=st["out"])
    got["k"], got["v"] = pa.kv_read_i4(h["cache"], st["table"], st["lengths"], st["row_starts"],
                                       st["k_out"], st["v_out"], first_tokens=st.get("first"))
    return got


# ------------------------------------------------------------------ 64 bits

def _places(d, kv):
    """Byte offset and shift of every code [16, d], and fp16 places of step and least value [16, d]."""
    G = d // 32
    j = torch.arange(16, device=DEV)[:, None]
    x = torch.arange(d, device=DEV)[None, :]
    g, y = x // 32, x % 32
    step = 4 * (G * (j % 8 // 2) + g) + 2 * (j // 8) + j % 2
    if kv == 0:
        byte = j * (d // 2) + y // 8 * 4 * G + 4 * g + y % 8 // 2
        least = 16 * G + G * j + g
    else:
        byte = 2 * (2 * (G * (4 * (8 * (j // 8) + y // 4) + j % 8 // 2) + g) + j % 2) + y % 4 // 2
        least = 16 * G + step
    return byte, 4 * (y % 2) + 0 * byte, step + 0 * byte, least + 0 * byte


def _exact_rows(st, s, n, kv):
    """The first n cached rows [n, Hk, d] of sequence s, in 64 bits."""
    d = st["case"]["head_dim"]
    byte, shift, step, least = _places(d, kv)
    tile = st["pool"][0, st["table"][s, :-(-n // 16)].long(), :, kv]  # [blocks, Hk, 10 d]
    par = tile[..., 8 * d:].contiguous().view(torch.float16).double()
    c = (tile[..., byte].int() >> shift) & 15
    return (par[..., least] + par[..., step] * c.double()).transpose(1, 2).flatten(0, 1)[:n]


def _exact_codes(x):
    """The values, in 64 bits, that the codes of rows [T, Hk, d] stand for."""
    x = x.double().unflatten(-1, (-1, 32))
    m, top = x.amin(-1, keepdim=True), x.amax(-1, keepdim=True)
    r = (top - m) / torch.full_like(m, 15.0)
    s = r.half().double()
    e = torch.floor(torch.log2(r.clamp(min=2.0 ** -14)))
    s = torch.where(s < r, s + 2.0 ** (e - 10), s)
    c = torch.where(s > 0, torch.round((x - m) / torch.where(s > 0, s, 1.0)).clamp(0, 15), 0.0)
    return (m + s * c).flatten(-2)


def exact(case, seed):
    st = prepare(case, seed)
    past, new = _lengths(case)
    H, Hk, d, B = case["heads"], case["kv_heads"], case["head_dim"], case["batch"]
    g = H // Hk
    if case["kind"] == "store":
        ang = st["rope"].double()[st["pos"].long()]
        turn = torch.complex(ang[..., 0], ang[..., 1])[:, None]

        def rotated(x):
            z = torch.view_as_complex(x.double().unflatten(-1, (-1, 2)).contiguous())
            return torch.view_as_real(z * turn).flatten(-2)

        return {"q": rotated(st["q"]), "k": _exact_codes(rotated(st["k"]).half()),
                "v": _exact_codes(st["v"])}
    if case["kind"] == "read":
        return {"k": torch.cat([_exact_rows(st, s, past[s], 0) for s in range(B)]),
                "v": torch.cat([_exact_rows(st, s, past[s], 1) for s in range(B)])}
    out, at = [], 0
    for s in range(B):
        n, p = new[s], past[s]
        k, v = (_exact_rows(st, s, p + n, kv).transpose(0, 1) for kv in (0, 1))
        if case["kind"] == "prefill":
            k, v = k.half().double(), v.half().double()
        q = st["q"][at:at + n].double().transpose(0, 1).unflatten(0, (Hk, g))  # [Hk, g, n, d]
        for lo in range(0, n, 256):
            x = q[:, :, lo:lo + 256] @ k[:, None].transpose(-1, -2) / math.sqrt(d)
            i = torch.arange(lo, lo + x.shape[2], device=DEV)
            x.masked_fill_(torch.arange(p + n, device=DEV) > p + i[:, None], -math.inf)
            o = torch.softmax(x, -1) @ v[:, None]
            out.append(o.flatten(0, 1).transpose(0, 1))
        at += n
    return {"out": torch.cat(out)}
