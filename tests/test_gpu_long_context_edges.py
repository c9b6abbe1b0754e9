"""Calls of the long-context operators that their documentation allows beside those of
test_gpu_long_context.py: values that must come back as they are, workspaces that hold
anything, tables far wider than the contexts."""

import math

import numpy as np
import pytest
import torch

from oracle import reference as orc
from paged_kv_gqa_rope_gb300 import pa
from tests.gpu_helpers import assert_attention_close, bits, half_ulp16
from tests.test_gpu_long_context import (SHARED, EvictBatch, SharedBatch, WeightBatch, dev, ints,
                                         normal16)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib(libpa):
    assert torch.cuda.is_available()
    assert pa.check_device() == pa.PA_OK
    return libpa


# An average of equal values is the value.  P is fp16 in the product with V (of the
# shared prefixes), so that holds only if the sum that it is divided by adds the same fp16
# values.  Here one key of
# score 0 stands beside keys whose P is 0.9 of half a step above a power of two: each loses
# 0.9 * 2^-11 of itself to its rounding, while the values, 2047 / 1024 by powers of two,
# have a half step of 2^-12 of themselves.  Beside that rounding stand fp32 ones alone: a row
# has at most 300 blocks, 38 tiles of 8 products or 300 of one, each of which cuts its sum by
# 2^-22 at most, 300 * 2^-22 < 2^-13 together; the sums of P add 2^-24 a value of a thread's
# chain, at most 38 * 32 of them, less than 2^-13.
SCALE = (1 - math.log2(1 + 0.9 * 2.0 ** -11)) / math.log2(math.e)


def equal_values(b, seed):
    """Every token of the batch gets the same V row a KV head; the output that then is due."""
    rng = np.random.default_rng(seed)
    row = (2047 / 1024 * 2.0 ** rng.integers(-2, 2, (b.Hk, b.d)) * rng.choice([-1, 1], (b.Hk, b.d)))
    written = ~np.isnan(b.pool[1])
    b.pool[1] = np.where(written, row.astype(np.float16), b.pool[1])
    b.pool[0] = np.where(written, np.float16(0), b.pool[0])
    b.pool[0, ..., 0] = np.where(written[..., 0], np.float16(-1), b.pool[0, ..., 0])
    for s in range(len(b.ctx)):
        b.pool[0, b.layer, b.bt[s, 0], 0] = 0
    b.q[:] = 1
    return np.repeat(row, b.H // b.Hk, 0).astype(np.float16) + np.zeros(b.q.shape, np.float16)


@pytest.mark.parametrize("H,Hk,d", [(4, 2, 64), (14, 2, 64), (8, 1, 128), (12, 4, 128), (6, 6, 128)])
@pytest.mark.parametrize("groups", range(len(SHARED)))
def test_shared_gives_equal_values_back(H, Hk, d, groups):
    b = SharedBatch(groups, H, Hk, d, SHARED[groups])
    want = equal_values(b, groups)
    assert np.array_equal(bits(b.run(scale=SCALE)), bits(want))


@pytest.mark.parametrize("H,Hk,d", [(4, 2, 64), (14, 2, 64), (8, 1, 128), (12, 4, 128), (6, 6, 128)])
@pytest.mark.parametrize("lens", [[1], [16, 2, 17], [300, 5, 33, 64], [4800], [3] * 70])
def test_weights_give_equal_values_back(H, Hk, d, lens):
    b = WeightBatch(len(lens), H, Hk, d, lens)
    want = equal_values(b, len(lens))
    b.w[:] = 0
    out, got = b.run(scale=SCALE)
    assert np.array_equal(bits(out), bits(want))
    # The weights are those of the scores, not of P: n - 1 tokens of p beside one of 1.
    # Off by a sum of at most 80 blocks a warp, each step 2^-24 (2^-17.6), and a handful of
    # roundings of 2^-22.
    g, p, got = H // Hk, 2.0 ** -(SCALE * math.log2(math.e)), got.cpu().numpy()
    for s, n in enumerate(lens):
        w = np.full(n, g * p / (1 + p * (n - 1)))
        w[0] = g / (1 + p * (n - 1))
        assert np.abs(got[s, :, :n] / w - 1).max() <= 2.0 ** -17


@pytest.mark.parametrize("value", [np.inf, -np.inf, np.nan])
def test_infinite_values_stay_in_their_columns(value):
    """An infinite V of one token makes its column infinite, whatever P's rounding leaves for
    a second product; a NaN makes it NaN.  The other columns and heads are as before."""
    lens = [300, 5, 64, 2000]
    w = WeightBatch(9, 8, 2, 64, lens)
    b = SharedBatch(9, 8, 2, 64, [(20, [3, 40, 1]), (0, [77])])
    for x, run in ((w, lambda: w.run()[0]), (b, b.run)):
        want = x.want() if x is b else x.out()
        x.pool[1, 0, x.bt[0, 0], 0, 1, 7] = value  # the first sequence's, KV head 1, column 7
        got = run().float().cpu().numpy()
        hit = np.zeros(got.shape, bool)
        hit[:3 if x is b else 1, 4:, 7] = True  # (a shared block's: all who share it)
        assert np.isnan(got[hit]).all() if np.isnan(value) else (got[hit] == value).all()
        got[hit] = want[hit] = 0
        assert_attention_close(got.astype(np.float64), want)


@pytest.mark.parametrize("H,Hk,d", [(8, 1, 128), (32, 4, 64), (6, 6, 128)])
def test_weights_output_keeps_what_the_rounding_of_p_leaves(H, Hk, d):
    """The first key's P is 1 and its V -(n - 1) / 2, the n - 1 others' P is 0.9 * 2^-11 of
    itself above 1 / 2 and their V 1: what a single fp16 half keeps of P cancels."""
    b = WeightBatch(11, H, Hk, d, [3, 65, 1001, 3001])
    equal_values(b, 0)
    b.pool[1] = np.where(np.isnan(b.pool[1]), b.pool[1], np.float16(1))
    for s, n in enumerate(b.ctx):
        b.pool[1, 0, b.bt[s, 0], 0] = -(n - 1) / 2
    out = b.run(scale=SCALE)[0].double().cpu().numpy()
    p = 2.0 ** -(SCALE * math.log2(math.e))
    for s, n in enumerate(b.ctx):
        want = np.full((H, d), (n - 1) * (p - 0.5) / (1 + (n - 1) * p))  # 2.2e-4 to 4.4e-4
        # at most 47 blocks a warp, each cutting the sums of products of size n / 2 by 2^-22
        # of them, which are divided by more than n / 2; an exponent's roundings, 2^-21 of P
        assert (np.abs(out[s] - want) <= half_ulp16(want) + 50 * 2.0 ** -22).all()


# ------------------------------------------------------------------ workspaces

@pytest.mark.parametrize("byte", [0xFF, 0x7F, 0x3C])
def test_workspaces_hold_anything_before_the_first_call(byte):
    """Bytes that read as NaN, as negative or as large numbers: the same bits come out as
    from a cleared workspace, for sequences in order and those left out."""
    for groups in SHARED + [[(20, [3, 9, 1]), (12, [5, 5]), (9, [2, 300, 4])]]:
        b = SharedBatch(1, 8, 2, 128, groups)
        if len(groups) == 3:
            b.ctx[1] = 0  # left out
        B, outs = len(b.ctx), []
        for fill in (0, byte):
            ws = pa.decode_shared_workspace(B, 8, 2, 128).fill_(fill)
            status, out = pa.new_status(), torch.full(b.q.shape, 7.0).half().cuda()
            b.run(ws=ws, out=out, status=status)
            outs.append((out, int(status.item())))
        assert torch.equal(outs[0][0], outs[1][0]) and outs[0][1] == outs[1][1]
    for lens, blocks in (([1], 1), ([3000, 2, 77], 194), ([40] * 70, 210), ([300, 0, 9, 500], 24)):
        w = WeightBatch(2, 8, 2, 128, lens)  # (the last: one left out, one with no room)
        outs = []
        for fill in (0, byte):
            ws = pa.decode_weights_workspace(len(lens), 8, 2, 128, blocks).fill_(fill)
            status, out = pa.new_status(), torch.full(w.q.shape, 7.0).half().cuda()
            _, got = w.run(ws=ws, out=out, status=status)
            outs.append((out, got, int(status.item())))
        assert all(torch.equal(x, y) for x, y in zip(outs[0][:2], outs[1][:2]))
        assert outs[0][2] == outs[1][2]
        assert outs[0][2] == (pa.PA_DEV_BAD_LENGTH | pa.PA_DEV_WORKSPACE if 0 in lens else 0)


def test_half_a_million_pairs():
    """4096 sequences of 128 KV heads, 5 tokens behind 4 blocks that 64 of them share: with
    equal values in a head every output is the value, and the weights of a KV head's only Q
    head sum to 1."""
    B, H, d, pre, n = 4096, 128, 64, 4, 69
    rng = np.random.default_rng(3)
    row = rng.uniform(0.25, 4, (H, d)).astype(np.float16)
    cache = pa.Cache(1, 40, H, d)
    cache.tensor[0] = dev(normal16(rng, 1, 40, 16, H, d))
    cache.tensor[1] = dev(row)
    bt = np.empty((B, pre + 1), np.int32)
    for r in range(B // 64):
        bt[64 * r:64 * r + 64, :pre] = rng.permutation(40)[:pre]
    bt[:, pre] = rng.integers(0, 40, B)
    q, ctx = dev(normal16(rng, B, H, d)), ints([n] * B)
    status = pa.new_status()
    out = pa.decode_shared(q, cache, dev(bt), ctx, ints(list(range(0, B + 1, 64))),
                           ints([pre] * (B // 64)), pa.decode_shared_workspace(B, H, H, d), H,
                           status=status)
    assert int(status.item()) == 0 and torch.equal(out, dev(row).expand_as(out))
    w = torch.zeros(B, H, 80, device="cuda")
    out, _ = pa.decode_weights(q, cache, dev(bt), ctx, w,
                               pa.decode_weights_workspace(B, H, H, d, B * (pre + 1)), H,
                               status=status)
    assert int(status.item()) == 0 and torch.equal(out, dev(row).expand_as(out))
    # (69 weights, each with the roundings of an exponent below 16 and of a sum)
    assert (w.sum(-1) - 1).abs().max() <= 2.0 ** -16 and not w[..., n:].any()


# ------------------------------------------------------------------ wide tables

@pytest.mark.parametrize("width", [16383, 16384, 17000, 70000])
@pytest.mark.parametrize("lens", [[33000, 700], [70000, 20, 100, 5000, 3]])
def test_evict_with_tables_far_wider_than_the_contexts(width, lens):
    """Tables of 262128 tokens and more: clusters give way to one CTA a list, which reads
    what is past its registers again.  In place, weights beside, and into other blocks."""
    def widen(b):
        b.bt = np.concatenate([b.bt, np.full((len(lens), width - b.bt.shape[1]), -1, np.int32)], 1)
        return b

    for budget, sinks, recent in ((3000, 4, 256), (200, 0, 0)):
        widen(EvictBatch(1, 2, 2, 64, lens)).check(budget, sinks, recent)
    b = widen(EvictBatch(2, 2, 2, 64, lens, layers=2, layer=1))
    b.w[0, 0, :lens[0]] = 0.5  # (ties among what is read again)
    pool, want = b.pool.copy(), b.w.copy()
    n = orc.evict(pool, 1, b.bt, b.ctx, want, 1500, 4, 64, b.bt)
    for s, k in enumerate(lens):
        want[s, :, k:] = 5
    beside, status = torch.full(b.w.shape, 5.0, device="cuda"), pa.new_status()
    got, lens_out = b.run(1500, 4, 64, weights_out=beside, status=status)
    assert int(status.item()) == 0 and np.array_equal(lens_out.cpu().numpy(), n)
    assert np.array_equal(got.cpu().numpy(), want) and np.array_equal(bits(b.cache.tensor), bits(pool))
    b = widen(EvictBatch(3, 2, 2, 64, lens))
    more = -(-1500 // 16) * len(lens)
    b.pool = np.concatenate([b.pool, np.full_like(b.pool[:, :, :more], 7)], 2)
    to = np.arange(b.NB, b.NB + more, dtype=np.int32).reshape(len(lens), -1)
    b.NB += more
    b.check(1500, 4, 64, to)


def test_decodes_with_tables_far_wider_than_the_contexts():
    b = SharedBatch(4, 8, 2, 64, [(20, [3, 40]), (0, [17])])
    w = WeightBatch(5, 8, 2, 64, [300, 2, 64])
    for x in (b, w):
        x.bt = np.concatenate([x.bt, np.full((3, 70000), -1, np.int32)], 1)
    assert_attention_close(b.run(), b.want())
    out, got = w.run()
    assert_attention_close(out, w.out())
    want, tol = w.want()
    assert (np.abs(got.cpu().numpy() - want) <= tol).all()


# ------------------------------------------------------------------ layers

@pytest.mark.parametrize("inplace", [True, False])
def test_evict_every_layer_from_the_old_lengths(inplace):
    """Layers one after another, each with its own weights, through one workspace; then
    decode with weights over each, with the lengths that the last call wrote."""
    L, H, Hk, d = 3, 8, 2, 64
    b = EvictBatch(4, H, Hk, d, [500, 30, 129], layers=L)
    rng = np.random.default_rng(5)
    more = 7 * 3
    b.pool = normal16(rng, 2, L, b.NB + more, 16, Hk, d)
    to = b.bt if inplace else np.arange(b.NB, b.NB + more, dtype=np.int32).reshape(3, 7)
    w = np.stack([rng.random(b.w.shape, dtype=np.float32) for _ in range(L)])
    for s, n in enumerate(b.ctx):
        w[:, s, :, n:] = 0
    cache = pa.Cache(L, b.NB + more, Hk, d, tensor=dev(b.pool))
    bt, tod, ctx, wd = dev(b.bt), dev(to), dev(b.ctx), dev(w)
    new, ws, status = torch.zeros_like(ctx), pa.kv_evict_workspace(3, Hk, 100), pa.new_status()
    for layer in range(L):
        pa.kv_evict(cache, bt, ctx, wd[layer], 100, ws, sinks=4, recent=20, out_block_tables=tod,
                    out_context_lens=new, layer=layer, status=status)
    lens = [orc.evict(b.pool, layer, b.bt, b.ctx, w[layer], 100, 4, 20, to) for layer in range(L)][0]
    assert int(status.item()) == 0 and new.tolist() == lens.tolist() == [100, 30, 100]
    assert np.array_equal(wd.cpu().numpy(), w) and np.array_equal(bits(cache.tensor), bits(b.pool))
    q = normal16(rng, 3, H, d)
    for layer in range(L):
        out, _ = pa.decode_weights(dev(q), cache, tod, new, wd[layer],
                                   pa.decode_weights_workspace(3, H, Hk, d, 7 * 3), Hk, layer=layer,
                                   status=status)
        assert_attention_close(out, orc.attention_decode(q, b.pool, layer, to, lens, H, Hk))
    assert int(status.item()) == 0


# ------------------------------------------------------------------ largest sizes

@pytest.mark.parametrize("half", [False, True])
def test_append_of_more_tokens_than_a_grid_has_rows(half):
    """70000 tokens: past 65535, and past what is stored to stay in L2."""
    T, H, Hk, d, rotary = 70000, 4, 2, 128, 96
    rng = np.random.default_rng(6)
    q, k, v = (normal16(rng, 64, n, d) for n in (H, Hk, Hk))
    pos = rng.integers(0, 500, T).astype(np.int32)
    table = orc.rope_scaled_table(500, rotary)
    pick = np.arange(T) % 64  # (rows again and again, at other positions)
    NB = T // 16 + 2
    slots = rng.permutation(NB * 16)[:T].astype(np.int32)
    cache, status = pa.Cache(1, NB, Hk, d), pa.new_status()
    cache.tensor.zero_()
    out = pa.rope_kv_write_layout(dev(q[pick]), dev(k[pick]), dev(v[pick]), dev(pos), dev(slots),
                                  dev(table), cache, "half" if half else "interleaved",
                                  status=status)
    assert int(status.item()) == 0
    assert np.array_equal(bits(out), bits(orc.rope_layout_pinned(q[pick], pos, table, half)))
    pool = np.zeros((2, 1, NB, 16, Hk, d), np.float16)
    orc.kv_write(pool, 0, orc.rope_layout_pinned(k[pick], pos, table, half), v[pick], slots)
    assert np.array_equal(bits(cache.tensor), bits(pool))


def test_a_line_of_more_places_than_32_bits_plan():
    """4096 KV heads over 32768 shared tokens: 2.1 million places, which the plan divides in
    64 bits; against pa_decode, whose own rounding of P stands beside."""
    H, d, pre, B = 4096, 64, 2048, 2
    cache = pa.Cache(1, pre + 2 * B, H, d)
    gen = torch.Generator(device="cuda").manual_seed(1)
    for part in cache.tensor.view(-1).split(2**30):
        part.normal_(generator=gen)
    bt = torch.arange(pre + 2, dtype=torch.int32).repeat(B, 1)
    bt[1, pre:] += 2
    ctx = ints([16 * pre + 9, 16 * pre + 32])
    q = torch.randn(B, H, d, device="cuda", generator=gen).half()
    status = pa.new_status()
    out = pa.decode_shared(q, cache, bt.cuda(), ctx, ints([0, B]), ints([pre]),
                           pa.decode_shared_workspace(B, H, H, d), H, status=status)
    want = pa.decode(q, cache, bt.cuda(), ctx, pa.decode_workspace(B, H, H, d), H)
    assert int(status.item()) == 0
    # (each within the library's 1e-3 of the exact output)
    assert torch.linalg.norm(out.float() - want.float()) <= 2e-3 * torch.linalg.norm(want.float())
    assert (out.float() - want.float()).abs().max() <= 2e-3


def test_most_kv_heads():
    """65535 KV heads, as many as a grid has rows: weights and an eviction by them."""
    H, d, n, budget = 65535, 64, 20, 10
    cache = pa.Cache(1, 2, H, d)
    gen = torch.Generator(device="cuda").manual_seed(2)
    cache.tensor.normal_(generator=gen)
    before = cache.tensor.clone()
    bt, ctx = ints([[1, 0]]), ints([n])
    q = torch.randn(1, H, d, device="cuda", generator=gen).half()
    w = torch.zeros(1, H, 32, device="cuda")
    status = pa.new_status()
    out, _ = pa.decode_weights(q, cache, bt, ctx, w, pa.decode_weights_workspace(1, H, H, d, 2), H,
                               status=status)
    K, V = (before[i, 0, [1, 0]].reshape(32, H, d)[:n].float() for i in range(2))
    p = torch.softmax(torch.einsum("hd,thd->ht", q[0].float(), K) / d ** 0.5, -1)
    assert int(status.item()) == 0
    assert (w[0, :, :n] - p).abs().max() <= 1e-5 and not w[..., n:].any()
    want = torch.einsum("ht,thd->hd", p, V)
    assert (out[0].float() - want).abs().max() <= 2e-3
    kept = w[0, :, :n].topk(budget).indices.sort().values.T  # [budget, H]
    old = w.clone()
    pa.kv_evict(cache, bt, ctx, w, budget, pa.kv_evict_workspace(1, H, budget), status=status)
    assert int(status.item()) == 0 and ctx.tolist() == [budget]
    for i, rows in enumerate((K, V)):
        got = cache.tensor[i, 0, 1, :budget].float()
        assert torch.equal(got, rows.gather(0, kept[..., None].expand(-1, -1, d)))
    assert torch.equal(w[0, :, :budget], old[0].gather(1, kept.T)) and not w[..., budget:].any()
