"""Cases of the operators of long contexts over the fp16 paged cache: decode
attention of sequences that share a prefix, decode attention that accumulates
each cached token's attention weight, eviction of the tokens with the least
weight, and the append with other rotary layouts.

`run` computes a case with elementary torch operations in 32 bits (`own` false)
or with the library's entry points (`own` true); `exact` computes it in 64 bits
from the definition.

The pool is [2 (K, V)][layers][blocks][16][KV heads][d] fp16; token t of
sequence s is row t % 16 of block block_tables[s][t / 16].  Q head h reads KV
head h / (heads / KV heads).  With x_h = q_h K^T / sqrt(d) over the cached
tokens:
    shared   out_h = softmax(x_h) V; the sequences of a group name the same first
             blocks
    weights  the same (nothing shared), and
             weight[kv head][token] += sum over its Q heads of softmax(x_h)[token]
    evict    of a sequence's n tokens, for each KV head: the first `sinks`, the
             last `recent`, and of the others those of the largest weight (of
             equal ones the first), `budget` in all, in their order; all if
             n <= budget.  K and V rows and weights move together; weights of
             the places that fall free become zero
    rope     the first `rotary` values of every Q and K row turned pairwise by
             angle(position, i), i < rotary / 2: values 2i and 2i + 1
             (interleaved) or i and i + rotary / 2 (half); K and V appended
"""

import math
import random

import torch

own = False

DEV = "cuda"
HEADS = [(4, 2, 64), (14, 2, 64), (32, 4, 64), (12, 4, 128), (16, 8, 128), (8, 1, 128),
         (32, 8, 128), (64, 8, 128), (32, 32, 128), (40, 40, 128)]  # (Q heads, KV heads, d)


def listed():
    def case(name, kind, heads, kv_heads, d, batch, past, mix, **more):
        return dict(name=name, kind=kind, heads=heads, kv_heads=kv_heads, head_dim=d, batch=batch,
                    past_lo=past[0], past_hi=past[1], mix=mix, **more)

    return [
        # decode with a shared prefix: `past` is what a sequence has of its own behind it.
        # Four samples of one short prompt, a small model (latency alone)
        case("shared_small", "shared", 4, 2, 64, 4, (1, 9), 1, groups=1, pre_lo=80, pre_hi=80),
        # a serving batch under one long system prompt: grouped heads, one KV head per Q head
        case("shared_gqa", "shared", 64, 8, 128, 32, (16, 512), 2, groups=1, pre_lo=8192, pre_hi=8192),
        case("shared_mha", "shared", 32, 32, 128, 32, (16, 512), 3, groups=1, pre_lo=2048, pre_hi=2048),
        # several documents in one batch, each with questions about it
        case("shared_groups", "shared", 32, 8, 128, 64, (16, 1000), 4, groups=6, pre_lo=100, pre_hi=16384),
        # decode that accumulates weights: three short sequences, a serving batch,
        # histories from 16 to 16384 tokens side by side
        case("weights_small", "weights", 4, 2, 64, 3, (3, 9), 5),
        case("weights_gqa", "weights", 64, 8, 128, 32, (4097, 4097), 6),
        case("weights_ragged", "weights", 32, 8, 128, 64, (16, 16384), 7),
        # eviction: a small model's sequences, a serving batch cut to a quarter, one
        # long document cut to an eighth
        case("evict_small", "evict", 32, 4, 64, 7, (200, 700), 8, budget=256, sinks=4, recent=64),
        case("evict_batch", "evict", 32, 8, 128, 32, (1000, 5000), 9, budget=1024, sinks=4, recent=256),
        case("evict_one_long", "evict", 64, 8, 128, 1, (32767, 32767), 10, budget=4096, sinks=4,
             recent=1024),
        # the append: one decode step's tokens (half layout, whole heads), a batch of
        # prompts (half layout, half of each head, positions far out)
        case("rope_step", "rope", 32, 8, 128, 256, (16, 1000), 11, new_lo=1, new_hi=1, rotary=128,
             half=True),
        case("rope_prompts", "rope", 64, 8, 128, 16, (0, 100000), 12, new_lo=128, new_hi=2048,
             rotary=64, half=True),
    ]


def _between(rng, lo, hi):
    """A whole number, uniform over its logarithm."""
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["shared", "shared", "weights", "weights", "evict", "rope"])
    heads, kv_heads, d = rng.choice(HEADS)
    c = dict(kind=kind, heads=heads, kv_heads=kv_heads, head_dim=d, mix=rng.randrange(1 << 20),
             past_lo=1)
    if kind == "rope":
        c["new_hi"] = rng.choice([1, _between(rng, 1, 2048)])
        most = 2e8 / ((heads + kv_heads) * d * c["new_hi"])
        c["batch"] = _between(rng, 1, max(1, min(256, int(most))))
        c["new_lo"] = _between(rng, 1, c["new_hi"])
        c["past_lo"], c["past_hi"] = 0, rng.choice([0, _between(rng, 1, 100000)])
        c["rotary"] = d * rng.choice([2, 1, 3, 4, 4, 4]) // 4
        c["half"] = rng.random() < 0.6
        return c
    size = {"shared": 6e7, "weights": 1.3e8, "evict": 1.2e8}[kind] / (kv_heads * d)  # padded tokens
    if kind == "shared":
        c["past_hi"] = _between(rng, 1, 2000)
        c["batch"] = _between(rng, 2, max(2, min(200, int(size / c["past_hi"]))))
        c["groups"] = _between(rng, 1, min(8, c["batch"]))
        rows = c["batch"] * heads  # (padded scores of a group's rows)
        c["pre_hi"] = _between(rng, 16, max(16, min(32768, int(min(size, 2e8 / rows)) // c["groups"])))
        c["pre_lo"] = _between(rng, 1, c["pre_hi"])
    else:
        c["past_hi"] = _between(rng, 1, 32767)
        c["batch"] = _between(rng, 1, max(1, min(200, int(size / c["past_hi"]))))
    c["past_lo"] = _between(rng, 1, c["past_hi"])
    if kind == "evict":
        c["budget"] = _between(rng, 1, 1 + c["past_hi"])
        c["sinks"] = rng.choice([0, min(4, c["budget"])])
        c["recent"] = rng.choice([0, (c["budget"] - c["sinks"]) // 4, c["budget"] - c["sinks"]])
    return c


def _some(rng, lo, hi, n):
    if lo == hi:
        return [lo] * n
    return [min(hi, max(lo, _between(rng, max(lo, 1), hi))) if lo or rng.random() < 0.8 else 0
            for _ in range(n)]


def _lengths(case):
    """By the case alone: each sequence's own cached tokens; each group's sequences and
    shared blocks, or each sequence's new tokens."""
    rng = random.Random(case["mix"])
    past = _some(rng, case["past_lo"], case["past_hi"], case["batch"])
    if case["kind"] == "shared":
        cuts = sorted(rng.sample(range(1, case["batch"]), case["groups"] - 1))
        sizes = [b - a for a, b in zip([0] + cuts, cuts + [case["batch"]])]
        return past, sizes, [p // 16 for p in _some(rng, case["pre_lo"], case["pre_hi"], case["groups"])]
    if case["kind"] == "rope":
        return past, _some(rng, case["new_lo"], case["new_hi"], case["batch"])
    return (past,)


def _totals(case):
    """Cached tokens that each sequence attends to (or evicts from), and the tokens that
    the cache holds for them."""
    if case["kind"] == "shared":
        past, sizes, pre = _lengths(case)
        first = [16 * p for n, p in zip(sizes, pre) for _ in range(n)]
        return [f + p for f, p in zip(first, past)], 16 * sum(pre) + sum(past)
    past = _lengths(case)[0]
    return past, sum(past)


def work(case):
    H, Hk, d, B = case["heads"], case["kv_heads"], case["head_dim"], case["batch"]
    if case["kind"] == "rope":
        T = sum(_lengths(case)[1])
        # Q in and out, K and V in and appended, a row of the table, position and slot
        return dict(bytes=T * (4 * H * d + 8 * Hk * d + 4 * case["rotary"] + 8),
                    flops=T * 3 * (H + Hk) * case["rotary"])
    total, held = _totals(case)
    if case["kind"] == "evict":
        kept = sum(min(n, case["budget"]) for n in total)
        # the kept rows in and out, all weights in, the weights' places out
        return dict(bytes=8 * kept * Hk * d + 8 * held * Hk, flops=held * Hk)
    more = 8 * held * Hk if case["kind"] == "weights" else 0
    return dict(bytes=4 * held * Hk * d + 4 * B * H * d + held / 4 + more,
                flops=4 * H * d * sum(total))


# ------------------------------------------------------------------ inputs

def prepare(case, seed):
    H, Hk, d, B = case["heads"], case["kv_heads"], case["head_dim"], case["batch"]
    rng = torch.Generator(device=DEV).manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, device=DEV, generator=rng)

    def ints(x):
        return torch.tensor(x, dtype=torch.int32, device=DEV)

    def tables(need, order):
        """Rows of blocks, taken one after another from `order`; -1 behind them."""
        have, col = ints(need), torch.arange(max(max(need), 1), device=DEV)
        at = ((have.cumsum(0) - have).long()[:, None] + col).clamp(max=max(len(order) - 1, 0))
        return torch.where(col < have[:, None], order[at], -1).int()

    st = dict(case=case, handles={})
    # K with a few channels of large values, as attention layers have them
    gain = torch.where(torch.rand(Hk, d, device=DEV, generator=rng) < 0.03, 4.0, 1.0)

    if case["kind"] == "rope":
        past, new = _lengths(case)
        T = sum(new)
        seq = torch.repeat_interleave(torch.arange(B, device=DEV), ints(new))
        pos = ints(past)[seq] + torch.arange(T, device=DEV) - (ints(new).cumsum(0) - ints(new))[seq]
        # the blocks that the new tokens fall into
        first = [p // 16 for p in past]
        need = [-(-(p + n) // 16) - f for p, n, f in zip(past, new, first)]
        blocks = sum(need) + sum(need) // 10 + 1
        table = tables(need, torch.randperm(blocks, device=DEV, generator=rng))
        st["slots"] = (table[seq, (pos // 16 - ints(first)[seq]).long()] * 16 + pos % 16).int()
        st["pos"] = pos.int()
        st["q"], st["v"] = normal(T, H, d).half(), normal(T, Hk, d).half()
        st["k"] = (normal(T, Hk, d) * gain).half()
        st["out"] = torch.empty_like(st["q"])
        st["rope"] = _angles(case, max(p + n for p, n in zip(past, new)))
        st["rope"] = torch.stack([st["rope"].cos(), st["rope"].sin()], -1).float()
        st["pool"] = torch.zeros(2, 1, blocks, 16, Hk, d, dtype=torch.float16, device=DEV)
        return st

    total, _ = _totals(case)
    st["lengths"] = ints(total)
    need = [-(-n // 16) for n in total]
    if case["kind"] == "shared":
        past, sizes, pre = _lengths(case)
        mine = [-(-n // 16) for n in past]
        count = sum(pre) + sum(mine)
        order = torch.randperm(count + count // 10 + 1, device=DEV, generator=rng)
        group = torch.repeat_interleave(torch.arange(len(sizes), device=DEV), ints(sizes))
        col = torch.arange(max(need), device=DEV)
        ahead, behind = tables(pre, order[:sum(pre)] if sum(pre) else order[:1]), tables(mine, order[sum(pre):])
        lead = ints(pre)[group][:, None]
        own_col = (col - lead).clamp(0, behind.shape[1] - 1).long()
        pre_col = col.clamp(max=ahead.shape[1] - 1).expand(B, -1)
        table = torch.where(col < lead, ahead[group].gather(1, pre_col), behind.gather(1, own_col))
        st["table"] = torch.where(col < ints(need)[:, None], table, -1).int()
        st["starts"] = ints([sum(sizes[:i]) for i in range(len(sizes) + 1)])
        st["shared"], st["group"] = ints(pre), group
        st["most"] = (max(sizes), max(pre), max(past))
        blocks = len(order)
    else:
        blocks = sum(need) + sum(need) // 10 + 1
        st["table"] = tables(need, torch.randperm(blocks, device=DEV, generator=rng))
    if case["kind"] == "evict":
        kept = [min(n, case["budget"]) for n in total]
        fresh = [-(-n // 16) for n in kept]
        st["held"] = blocks
        st["to"] = tables(fresh, blocks + torch.randperm(sum(fresh), device=DEV, generator=rng))
        st["to_lengths"] = torch.zeros_like(st["lengths"])
        blocks += sum(fresh)
    pool = torch.zeros(2, 1, blocks, 16, Hk, d, dtype=torch.float16, device=DEV)
    step = max(1, (1 << 27) // (Hk * 16 * d))
    for b in range(0, st.get("held", blocks), step):
        n = min(step, st.get("held", blocks) - b)
        pool[0, 0, b:b + n] = (normal(n, 16, Hk, d) * gain).half()
        pool[1, 0, b:b + n] = normal(n, 16, Hk, d).half()
    st["pool"] = pool
    if case["kind"] != "evict":
        st["q"] = normal(B, H, d).half()
        st["out"] = torch.empty_like(st["q"])
    if case["kind"] != "shared":
        # what earlier steps left: most weights small, a few large, some never touched
        n = 16 * st["table"].shape[1]
        w = torch.rand(B, Hk, n, device=DEV, generator=rng).clamp(min=1e-3) ** 4
        w = torch.where(torch.rand(B, Hk, n, device=DEV, generator=rng) < 0.1, 0.0, w)
        st["weights"] = torch.where(torch.arange(n, device=DEV) < st["lengths"][:, None, None], w, 0.0)
        st["weights_out"] = torch.zeros_like(st["weights"])
    return st


def _angles(case, positions):
    """position * 10000^(-2i / rotary), slowed for long contexts: frequencies whose wave is
    longer than 4096 positions by 8, those shorter than 1024 not, in between in proportion."""
    i = torch.arange(0, case["rotary"], 2, device=DEV, dtype=torch.float64)
    f = 10000.0 ** (-i / case["rotary"])
    keep = ((4096 * f / (2 * math.pi) - 1) / (4 - 1)).clamp(0, 1)
    f = f * keep + f / 8 * (1 - keep)
    return torch.arange(positions, device=DEV, dtype=torch.float64)[:, None] * f


# ------------------------------------------------------------------ plain form

def _rows(st, kv, table, tokens):
    """fp32 rows [n, Hk, width, d] of the tokens [n, width] of the table's sequences."""
    block = table.gather(1, (tokens // 16).clamp(max=table.shape[1] - 1)).clamp(min=0).long()
    return st["pool"][kv, 0][block, tokens % 16].float().transpose(1, 2)


def _history(st, kv):
    """fp32 rows [B, Hk, width * 16, d] of every sequence, padded."""
    x = st["pool"][kv, 0][st["table"].clamp(min=0).long()]  # [B, width, 16, Hk, d]
    return x.flatten(1, 2).transpose(1, 2).float()


def _plain_shared(st):
    case = st["case"]
    H, Hk, d, B = case["heads"], case["kv_heads"], case["head_dim"], case["batch"]
    g, (most, pre, past) = H // Hk, st["most"]
    q = st["q"].float().view(B, Hk, g, d) * (1.0 / math.sqrt(d))
    # behind the prefix, each sequence by itself
    lead = 16 * st["shared"].long()[st["group"]][:, None]
    tokens = lead + torch.arange(past, device=DEV)
    have = tokens < st["lengths"][:, None]
    tokens = torch.where(have, tokens, 0)
    x = torch.matmul(q, _rows(st, 0, st["table"], tokens).transpose(-1, -2))
    x = torch.where(have[:, None, None], x, -math.inf)
    v = _rows(st, 1, st["table"], tokens)
    if pre == 0:
        e = torch.exp(x - x.amax(-1, keepdim=True))
        return {"out": (torch.matmul(e, v) / e.sum(-1, keepdim=True)).reshape(B, H, d).half()}
    # the prefix, once for a group: the queries of its sequences stacked
    start = st["starts"][:-1].long()
    member = torch.arange(B, device=DEV) - start[st["group"]]
    seq = (start[:, None] + torch.arange(most, device=DEV)).clamp(max=B - 1)
    stacked = q[seq].permute(0, 2, 1, 3, 4).flatten(2, 3)  # [G, Hk, most * g, d]
    tokens = torch.arange(16 * pre, device=DEV).expand(len(start), -1)
    have = tokens < 16 * st["shared"][:, None]
    tokens = torch.where(have, tokens, 0)
    table = st["table"][start]
    y = torch.matmul(stacked, _rows(st, 0, table, tokens).transpose(-1, -2))
    y = torch.where(have[:, None, None], y, -math.inf)

    def of_sequences(z):  # [G, Hk, most * g, ...] -> [B, Hk, g, ...]
        return z.unflatten(2, (most, g))[st["group"], :, member]

    m = torch.maximum(x.amax(-1, keepdim=True), of_sequences(y.amax(-1, keepdim=True)))
    e = torch.exp(x - m)
    top = m[seq].permute(0, 2, 1, 3, 4).flatten(2, 3)
    f = torch.exp(y - top)
    o = torch.matmul(e, v) + of_sequences(torch.matmul(f, _rows(st, 1, table, tokens)))
    s = e.sum(-1, keepdim=True) + of_sequences(f.sum(-1, keepdim=True))
    return {"out": (o / s).reshape(B, H, d).half()}


def _plain_weights(st):
    case = st["case"]
    H, Hk, d, B = case["heads"], case["kv_heads"], case["head_dim"], case["batch"]
    k = _history(st, 0)
    q = st["q"].float().view(B, Hk, H // Hk, d) * (1.0 / math.sqrt(d))
    x = torch.matmul(q, k.transpose(-1, -2))
    have = torch.arange(k.shape[2], device=DEV) < st["lengths"][:, None]
    x = torch.where(have[:, None, None], x, -math.inf)
    x = torch.exp(x - x.amax(-1, keepdim=True))
    x = x / x.sum(-1, keepdim=True)
    o = torch.matmul(x, _history(st, 1))
    return {"out": o.reshape(B, H, d).half(),
            "weights": torch.where(have[:, None], st["weights"] + x.sum(2), 0.0)}


def _plain_evict(st):
    case, w = st["case"], st["weights"]
    B, Hk, n = w.shape
    at = torch.arange(n, device=DEV)
    length = st["lengths"].long()[:, None, None]
    keep = st["lengths"].clamp(max=case["budget"])
    # the first and the last tokens ahead of every weight, places behind the length after it
    rank = torch.where((at < case["sinks"]) | (at >= length - case["recent"]), math.inf, w)
    rank = torch.where(at < length, rank, -math.inf)
    order = torch.sort(rank, dim=-1, descending=True, stable=True).indices[..., :case["budget"]]
    col = torch.arange(order.shape[-1], device=DEV)
    chosen = col < keep[:, None, None]
    order = torch.sort(torch.where(chosen, order, n)).values  # [B, Hk, budget], in order
    chosen = order < n
    order = torch.where(chosen, order, 0)
    moved = torch.zeros_like(w)
    moved[..., :order.shape[-1]] = torch.where(chosen, w.gather(-1, order), 0.0)
    b, h, i = chosen.nonzero(as_tuple=True)
    src = order[b, h, i]
    block, to = st["table"][b, src // 16].long(), st["to"][b, i // 16].long()
    for kv in (0, 1):
        st["pool"][kv, 0][to, i % 16, h] = st["pool"][kv, 0][block, src % 16, h]
    return {"k": st["pool"][0, 0, st["held"]:], "v": st["pool"][1, 0, st["held"]:],
            "weights": moved, "lengths": keep}


def _plain_rope(st):
    case = st["case"]
    r = case["rotary"]
    cs = st["rope"][st["pos"].long()][:, None]  # [T, 1, r / 2, 2]
    c, s = cs[..., 0], cs[..., 1]

    def turn(x):
        x = x.float()
        y = x[..., :r].unflatten(-1, (2, -1) if case["half"] else (-1, 2))
        a, b = y.unbind(-2 if case["half"] else -1)
        y = torch.stack([a * c - b * s, a * s + b * c], -2 if case["half"] else -1).flatten(-2)
        return torch.cat([y, x[..., r:]], -1).half()

    block, row = (st["slots"] // 16).long(), (st["slots"] % 16).long()
    st["pool"][0, 0, block, row] = turn(st["k"])
    st["pool"][1, 0, block, row] = st["v"]
    return {"q": turn(st["q"]), "k": st["pool"][0], "v": st["pool"][1]}


# ------------------------------------------------------------------ the library's calls

def _handles(st):
    """What a user's program makes once: the pool's descriptor and the workspaces."""
    from paged_kv_gqa_rope_gb300 import pa
    case, h = st["case"], st["handles"]
    H, Hk, d, B = case["heads"], case["kv_heads"], case["head_dim"], case["batch"]
    if not h:
        h["cache"] = pa.Cache(1, st["pool"].shape[2], Hk, d, tensor=st["pool"])
        if case["kind"] == "shared":
            h["ws"] = pa.decode_shared_workspace(B, H, Hk, d)
        if case["kind"] == "weights":
            blocks = sum(-(-n // 16) for n in _totals(case)[0])
            h["ws"] = pa.decode_weights_workspace(B, H, Hk, d, blocks)
        if case["kind"] == "evict":
            h["ws"] = pa.kv_evict_workspace(B, Hk, case["budget"])
    return pa, h


def run(st):
    case = st["case"]
    if not own:
        return dict(shared=_plain_shared, weights=_plain_weights, evict=_plain_evict,
                    rope=_plain_rope)[case["kind"]](st)
    pa, h = _handles(st)
    if case["kind"] == "shared":
        return {"out": pa.decode_shared(st["q"], h["cache"], st["table"], st["lengths"],
                                        st["starts"], st["shared"], h["ws"], case["kv_heads"],
                                        out=st["out"])}
    if case["kind"] == "weights":
        out, weights = pa.decode_weights(st["q"], h["cache"], st["table"], st["lengths"],
                                         st["weights"], h["ws"], case["kv_heads"],
                                         weights_out=st["weights_out"], out=st["out"])
        return {"out": out, "weights": weights}
    if case["kind"] == "evict":
        weights, lengths = pa.kv_evict(h["cache"], st["table"], st["lengths"], st["weights"],
                                       case["budget"], h["ws"], sinks=case["sinks"],
                                       recent=case["recent"], out_block_tables=st["to"],
                                       out_context_lens=st["to_lengths"],
                                       weights_out=st["weights_out"])
        return {"k": st["pool"][0, 0, st["held"]:], "v": st["pool"][1, 0, st["held"]:],
                "weights": weights, "lengths": lengths}
    q = pa.rope_kv_write_layout(st["q"], st["k"], st["v"], st["pos"], st["slots"], st["rope"],
                                h["cache"], "half" if case["half"] else "interleaved",
                                q_out=st["out"])
    return {"q": q, "k": st["pool"][0], "v": st["pool"][1]}


# ------------------------------------------------------------------ 64 bits

def _cached(st, s, n, kv):
    """The first n cached rows [Hk, n, d] of sequence s, in 64 bits."""
    x = st["pool"][kv, 0][st["table"][s, :-(-n // 16)].long()].flatten(0, 1)[:n]
    return x.double().transpose(0, 1)


def exact(case, seed):
    st = prepare(case, seed)
    H, Hk, d, B = case["heads"], case["kv_heads"], case["head_dim"], case["batch"]
    if case["kind"] == "rope":
        r = case["rotary"]
        i = torch.arange(r // 2, device=DEV)
        first, second = (i, i + r // 2) if case["half"] else (2 * i, 2 * i + 1)
        cs = st["rope"].double()[st["pos"].long()][:, None]
        turn = torch.complex(cs[..., 0], cs[..., 1])

        def turned(x):
            x = x.double()
            z = torch.complex(x[..., first], x[..., second]) * turn
            x[..., first], x[..., second] = z.real, z.imag
            return x

        k, v = st["pool"].double()[:, 0].flatten(1, 2)
        k[st["slots"].long()], v[st["slots"].long()] = turned(st["k"]), st["v"].double()
        return {"q": turned(st["q"]), "k": k.view(st["pool"].shape[1:]),
                "v": v.view(st["pool"].shape[1:])}
    total, _ = _totals(case)
    if case["kind"] == "evict":
        w = st["weights"].double().cpu().numpy()
        moved = torch.zeros(w.shape, dtype=torch.float64)
        k, v = (st["pool"][kv, 0].double() for kv in (0, 1))
        for s, n in enumerate(total):
            last = max(n - case["recent"], 0)
            for h in range(Hk):
                def before(t):  # the order in which tokens are kept
                    return (not (t < case["sinks"] or t >= last), -w[s, h, t], t)
                kept = sorted(sorted(range(n), key=before)[:case["budget"]])
                moved[s, h, :len(kept)] = torch.from_numpy(w[s, h, kept])
                src, i = torch.tensor(kept, device=DEV), torch.arange(len(kept), device=DEV)
                block, to = st["table"][s, src // 16].long(), st["to"][s, i // 16].long()
                for x in (k, v):
                    x[to, i % 16, h] = x[block, src % 16, h]
        return {"k": k[st["held"]:], "v": v[st["held"]:], "weights": moved.to(DEV),
                "lengths": st["lengths"].clamp(max=case["budget"])}
    out, weights = [], torch.zeros(B, Hk, 16 * st["table"].shape[1], dtype=torch.float64, device=DEV)
    for s, n in enumerate(total):
        q = st["q"][s].double().unflatten(0, (Hk, H // Hk))
        p = torch.softmax(q @ _cached(st, s, n, 0).transpose(-1, -2) / math.sqrt(d), -1)
        out.append((p @ _cached(st, s, n, 1)).flatten(0, 1))
        if case["kind"] == "weights":
            weights[s, :, :n] = st["weights"][s, :, :n].double() + p.sum(1)
    if case["kind"] == "shared":
        return {"out": torch.stack(out)}
    return {"out": torch.stack(out), "weights": weights}
