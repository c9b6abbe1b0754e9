"""The long-context operators at their edges of size and use: thousands of sequences,
pools and weights past 32 bits, two streams at once, workspaces that serve several
shapes, calls on a stream of the caller's."""

import numpy as np
import pytest
import torch

from oracle import reference as orc
from paged_kv_gqa_rope_gb300 import pa
from tests.gpu_helpers import assert_attention_close, bits
from tests.test_gpu_long_context import (EvictBatch, SharedBatch, WeightBatch, cache_of, dev, ints,
                                         normal16)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib(libpa):
    assert torch.cuda.is_available()
    assert pa.check_device() == pa.PA_OK
    return libpa


@pytest.mark.parametrize("H,Hk", [(1, 1), (3, 1)])
def test_shared_thousands_of_groups(H, Hk):
    """4096 sequences in 2048 groups of two: many groups in every CTA's range, lines of
    groups longer than a warp."""
    rng = np.random.default_rng(1)
    groups = [(int(rng.integers(8, 20)), [int(x) for x in rng.integers(0, 20, 2)]) for _ in range(2048)]
    b = SharedBatch(3, H, Hk, 64, groups)
    status = pa.new_status()
    out = b.run(status=status)
    assert int(status.item()) == 0
    assert_attention_close(out, b.want())


def test_shared_one_group_of_thousands():
    b = SharedBatch(4, 2, 1, 64, [(20, [1 + i % 3 for i in range(4096)])])
    assert_attention_close(b.run(), b.want())


def test_weights_and_eviction_of_thousands():
    lens = [1 + (i * 37) % 60 for i in range(4096)]
    b = WeightBatch(5, 2, 1, 64, lens)
    status = pa.new_status()
    out, got = b.run(status=status)
    assert int(status.item()) == 0
    assert_attention_close(out, b.out())
    want, tol = b.want()
    assert (np.abs(got.cpu().numpy() - want) <= tol).all()
    EvictBatch(6, 1, 1, 64, lens).check(20, 2, 5)


class FarPool:
    """A pool of more than 2^32 elements a plane whose last blocks alone are used."""

    def __init__(self, small):
        _, L, n, bs, Hk, d = small.shape
        self.n = n
        blocks = 2**32 // (bs * Hk * d) + n + 3
        self.at = blocks - n
        self.cache = pa.Cache(L, blocks, Hk, d)
        self.cache.tensor[:, :, self.at:].copy_(torch.from_numpy(small))

    def table(self, bt):
        return dev(np.where(bt >= 0, bt + self.at, bt).astype(np.int32))

    def used(self):
        return self.cache.tensor[:, :, self.at:]


def test_pools_past_32_bits():
    H, Hk, d = 32, 32, 128
    b = SharedBatch(7, H, Hk, d, [(20, [3, 40]), (0, [17])])
    far = FarPool(b.pool)
    out = pa.decode_shared(dev(b.q), far.cache, far.table(b.bt), dev(b.ctx), dev(b.starts),
                           dev(b.shared), pa.decode_shared_workspace(3, H, Hk, d), Hk)
    assert_attention_close(out, b.want())
    w = dev(np.zeros((3, Hk, 16 * b.bt.shape[1]), np.float32))
    out, w = pa.decode_weights(dev(b.q), far.cache, far.table(b.bt), dev(b.ctx), w,
                               pa.decode_weights_workspace(3, H, Hk, d, 100), Hk)
    assert_attention_close(out, b.want())
    for s, x in enumerate(orc.decode_weights(b.q, b.pool, 0, b.bt, b.ctx, H, Hk)):
        assert np.abs(w[s, :, :b.ctx[s]].cpu().numpy() - x).max() <= 1e-4
    # append to and evict from the same far blocks
    rng = np.random.default_rng(1)
    T = 40
    q, k, v = normal16(rng, T, H, d), normal16(rng, T, Hk, d), normal16(rng, T, Hk, d)
    slots = rng.permutation(b.NB * 16)[:T].astype(np.int32)
    pos = np.arange(T, dtype=np.int32)
    table = orc.rope_scaled_table(T, 64)
    pa.rope_kv_write_layout(dev(q), dev(k), dev(v), dev(pos), dev(slots + 16 * far.at), dev(table),
                            far.cache, "half")
    orc.kv_write(b.pool, 0, orc.rope_layout_pinned(k, pos, table, True), v, slots)
    assert np.array_equal(bits(far.used()), bits(b.pool))
    e = EvictBatch(8, Hk, Hk, d, [300, 40])
    del far
    far = FarPool(e.pool)
    lens, w = dev(e.ctx), dev(e.w)
    pa.kv_evict(far.cache, far.table(e.bt), lens, w, 64, pa.kv_evict_workspace(2, Hk, 64), sinks=4,
                recent=16)
    assert orc.evict(e.pool, 0, e.bt, e.ctx, e.w, 64, 4, 16, e.bt).tolist() == lens.tolist()
    assert np.array_equal(w.cpu().numpy(), e.w) and np.array_equal(bits(far.used()), bits(e.pool))


def test_weights_past_32_bits():
    """Rows of weights 2^30 floats apart."""
    b = EvictBatch(9, 4, 2, 64, [200, 90])
    stride = 2**30 + 5
    w = torch.zeros(2, 2, stride, device="cuda")
    small = b.w.shape[-1]
    w[..., :small] = dev(b.w)
    want, tol = b.want()
    ws = pa.decode_weights_workspace(2, 4, 2, 64, b.blocks)
    cache = cache_of(b.pool)
    pa.decode_weights(dev(b.q), cache, dev(b.bt), dev(b.ctx), w, ws, 2)
    got = w[..., :small].cpu().numpy()
    assert (np.abs(got - want) <= tol).all()
    lens = dev(b.ctx)
    pa.kv_evict(cache, dev(b.bt), lens, w, 50, pa.kv_evict_workspace(2, 2, 50), recent=9)
    pool = b.pool.copy()
    orc.evict(pool, 0, b.bt, b.ctx, got, 50, 0, 9, b.bt)
    assert np.array_equal(w[..., :small].cpu().numpy(), got)
    assert np.array_equal(bits(cache.tensor), bits(pool))


def test_two_streams_at_once():
    """The same calls on two streams, each with its own workspace, many times over."""
    one = SharedBatch(21, 8, 2, 128, [(60, [30, 5, 70, 1])])
    two = SharedBatch(22, 8, 2, 128, [(9, [300, 5]), (33, [8, 8])])
    wa, wb = WeightBatch(23, 8, 2, 128, [700, 3, 64]), WeightBatch(24, 8, 2, 128, [90] * 9)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    jobs = []
    for b, w, st in ((one, wa, streams[0]), (two, wb, streams[1])):
        B, n = len(b.ctx), len(w.ctx)
        jobs.append((st, [dev(b.q), cache_of(b.pool), dev(b.bt), dev(b.ctx), dev(b.starts), dev(b.shared),
                          pa.decode_shared_workspace(B, 8, 2, 128), 2],
                     [dev(w.q), cache_of(w.pool), dev(w.bt), dev(w.ctx), dev(w.w),
                      pa.decode_weights_workspace(n, 8, 2, 128, w.blocks), 2], b, w))
    torch.cuda.synchronize()
    got = []
    for _ in range(20):
        for st, shared, weights, _, w in jobs:
            out = pa.decode_shared(*shared, stream=st)
            with torch.cuda.stream(st):
                apart = torch.zeros_like(weights[4])
            o, x = pa.decode_weights(*weights, weights_out=apart, stream=st)
            got.append((out, o, x))
    torch.cuda.synchronize()
    wants = [(b.want(), w.out(), *w.want()) for _, _, _, b, w in jobs]
    for i, (out, o, x) in enumerate(got):
        want, want_o, want_x, tol = wants[i % 2]
        assert torch.equal(out, got[i % 2][0]) and torch.equal(o, got[i % 2][1])
        assert torch.equal(x, got[i % 2][2])
        if i < 2:
            assert_attention_close(out, want)
            assert_attention_close(o, want_o)
            x = x.cpu().numpy()
            for s, n in enumerate(jobs[i][4].ctx):
                assert (np.abs(x - want_x)[s, :, :n] <= tol[s, :, :n]).all()


def test_one_workspace_for_several_shapes():
    ws_s = pa.decode_shared_workspace(64, 8, 8, 128)
    ws_w = pa.decode_weights_workspace(64, 8, 8, 128, 800)
    for seed, (H, Hk, d, lens) in enumerate([(8, 8, 128, [40] * 64), (8, 1, 64, [3000, 5]),
                                             (4, 2, 128, [100] * 30), (8, 8, 128, [33] * 64),
                                             (7, 1, 128, [5000]), (8, 8, 64, [70] * 64)]):
        b = WeightBatch(seed, H, Hk, d, lens)
        out, got = b.run(ws=ws_w)
        assert_attention_close(out, b.out())
        want, tol = b.want()
        assert (np.abs(got.cpu().numpy() - want) <= tol).all()
        c = SharedBatch(seed, H, Hk, d, [(12, [n % 100 for n in lens])])
        assert_attention_close(c.run(ws=ws_s), c.want())


def test_calls_on_another_stream():
    side = torch.cuda.Stream()
    e = EvictBatch(31, 4, 4, 64, [500, 130, 77])
    pool, want = e.pool.copy(), e.w.copy()
    n = orc.evict(pool, 0, e.bt, e.ctx, want, 100, 4, 20, e.bt)
    cache, w, lens, bt, ws = cache_of(e.pool), dev(e.w), dev(e.ctx), dev(e.bt), pa.kv_evict_workspace(3, 4, 100)
    torch.cuda.synchronize()
    pa.kv_evict(cache, bt, lens, w, 100, ws, sinks=4, recent=20, stream=side)
    side.synchronize()
    assert np.array_equal(w.cpu().numpy(), want) and lens.tolist() == n.tolist()
    assert np.array_equal(bits(cache.tensor), bits(pool))
    # decode right behind the eviction, with the lengths that it writes
    lens, w, cache = dev(e.ctx), dev(e.w), cache_of(e.pool)
    rng = np.random.default_rng(2)
    q = normal16(rng, 3, 8, 64)
    qd, dws = dev(q), pa.decode_workspace(3, 8, 4, 64)
    torch.cuda.synchronize()
    for _ in range(5):
        lens.copy_(dev(e.ctx))
        cache.tensor.copy_(dev(e.pool))
        w.copy_(dev(e.w))
        pa.kv_evict(cache, bt, lens, w, 100, ws, sinks=4, recent=20)
        out = pa.decode(qd, cache, bt, lens, dws, 4)
        assert_attention_close(out, orc.attention_decode(q, pool, 0, e.bt, n, 8, 4))
    table = pa.rope_table_scaled(100, 64, scaling="linear", factor=2.0, stream=side)
    assert np.array_equal(table.cpu().numpy(), orc.rope_scaled_table(100, 64, scaling="linear", factor=2.0))
    with pytest.raises(ValueError):
        pa.rope_table_scaled(100, 64, device="cpu", stream=side)


def test_empty_batches():
    cache = pa.Cache(1, 4, 2, 64)
    none = torch.empty(0, 4, 64, dtype=torch.float16, device="cuda")
    kv, i0 = none[:, :2].contiguous(), torch.empty(0, dtype=torch.int32, device="cuda")
    bt, w = torch.empty(0, 3, dtype=torch.int32, device="cuda"), torch.empty(0, 2, 48, device="cuda")
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    assert pa.decode_shared(none, cache, bt, i0, ints([0]), i0, ws, 2).shape == (0, 4, 64)
    assert pa.decode_weights(none, cache, bt, i0, w, ws, 2)[0].shape == (0, 4, 64)
    pa.kv_evict(cache, bt, i0, w, 8, ws)
    pa.rope_kv_write_layout(none, kv, kv, i0, i0, pa.rope_table(4, 64), cache, "half")


def test_lengths_written_just_before():
    """Lengths and groups changed by a copy, by an eviction, or by either with an append
    in between, right before the decodes that read them ahead of their wait."""
    H, Hk, d = 8, 2, 128
    b = SharedBatch(31, H, Hk, d, [(40, [30, 5, 70, 9]), (12, [50, 33])])
    pool, bt, q = cache_of(b.pool), dev(b.bt), dev(b.q)
    B = len(b.ctx)
    variants = [(b.ctx, b.starts, b.shared), (b.ctx - 3, b.starts, np.array([25, 12], np.int32)),
                (b.ctx - 2, np.array([0, 6, 6], np.int32), np.zeros(2, np.int32))]
    variants = [tuple(dev(x.astype(np.int32)) for x in v) for v in variants]
    ctx, starts, shared = (torch.empty_like(x) for x in variants[0])
    ws = pa.decode_shared_workspace(B, H, Hk, d)
    blocks = int(sum(-(-b.ctx // 16)))
    ww = pa.decode_weights_workspace(B, H, Hk, d, blocks)
    w0 = dev(np.random.default_rng(2).random((B, Hk, 16 * b.bt.shape[1])).astype(np.float32))
    # an append elsewhere: it lets the next kernel start at once
    other = pa.Cache(1, 2, Hk, d)
    oq, ok = torch.zeros(3, H, d).half().cuda(), torch.zeros(3, Hk, d).half().cuda()
    table = pa.rope_table(16, d)
    pos = slots = torch.arange(3, dtype=torch.int32).cuda()

    def step(v, wait, append):
        for x, y in zip((ctx, starts, shared), variants[v]):
            x.copy_(y)
        w = w0.clone()
        if append:
            pa.rope_kv_write_layout(oq, ok, ok, pos, slots, table, other, "half")
        if wait:
            torch.cuda.synchronize()
        out = pa.decode_shared(q, pool, bt, ctx, starts, shared, ws, Hk)
        o, w = pa.decode_weights(q, pool, bt, ctx, w, ww, Hk)
        return out, o, w

    want = [step(v, True, False) for v in range(3)]
    got = [(i % 3, step(i % 3, False, i % 2 == 0)) for i in range(60)]
    torch.cuda.synchronize()
    for v, outs in got:
        for x, y in zip(outs, want[v]):
            assert torch.equal(x, y)

    # lengths that an eviction in place leaves
    e = WeightBatch(33, H, Hk, d, [300, 77, 1000, 64])
    first, n = dev(e.pool), len(e.ctx)
    epool, ebt, eq = torch.empty_like(first), dev(e.bt), dev(e.q)
    cache = pa.Cache(1, e.NB, Hk, d, tensor=epool)
    ew = pa.decode_weights_workspace(n, H, Hk, d, e.blocks)
    es = pa.kv_evict_workspace(n, Hk, 128)
    elen, weights = dev(e.ctx), dev(e.w)

    def evict(wait, append):
        epool.copy_(first)
        elen.copy_(dev(e.ctx))
        weights.copy_(dev(e.w))
        pa.kv_evict(cache, ebt, elen, weights, 128, es, sinks=4, recent=16)
        if append:
            pa.rope_kv_write_layout(oq, ok, ok, pos, slots, table, other, "half")
        if wait:
            torch.cuda.synchronize()
        o, w = pa.decode_weights(eq, cache, ebt, elen, weights, ew, Hk)
        return o, w.clone(), elen.clone()

    want = evict(True, False)
    assert want[2].tolist() == [128, 77, 128, 64]
    got = [evict(False, i % 2 == 0) for i in range(20)]
    torch.cuda.synchronize()
    for outs in got:
        for x, y in zip(outs, want):
            assert torch.equal(x, y)
