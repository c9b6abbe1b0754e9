"""The long-context operators on the GPU against the oracle: the append with other
rotary layouts, decode with shared prefixes, decode that accumulates attention weights,
eviction by them, and a run of them together."""

import math

import numpy as np
import pytest
import torch

from oracle import reference as orc
from paged_kv_gqa_rope_gb300 import pa
from tests.gpu_helpers import assert_attention_close, bits, half_ulp16

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib(libpa):
    assert torch.cuda.is_available()
    assert pa.check_device() == pa.PA_OK
    return libpa


def dev(x):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def normal16(rng, *shape, std=1.0):
    return (rng.standard_normal(shape) * std).astype(np.float16)


def cache_of(pool):
    return pa.Cache(pool.shape[1], pool.shape[2], pool.shape[4], pool.shape[5], tensor=dev(pool))


# ------------------------------------------------------------------ the append

ROPE_SHAPES = [(4, 2, 64, 1), (32, 8, 128, 7), (14, 2, 64, 33), (5, 5, 128, 300), (64, 8, 128, 2000),
               (8, 1, 64, 1300)]


@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("H,Hk,d,T", ROPE_SHAPES)
def test_append_bit_exact(H, Hk, d, T, half):
    rng = np.random.default_rng(H * 1000 + T)
    for rotary in sorted({16, d // 2, 3 * d // 4, d}):
        q, k, v = normal16(rng, T, H, d), normal16(rng, T, Hk, d, std=3), normal16(rng, T, Hk, d)
        pos = rng.integers(0, 5000, T).astype(np.int32)
        NB = -(-T // 16) + 3
        slots = rng.permutation(NB * 16)[:T].astype(np.int32)
        if T > 4:
            slots[3] = -1  # a padding token
        pool = normal16(rng, 2, 2, NB, 16, Hk, d)
        cache, status = cache_of(pool), pa.new_status()
        table = orc.rope_scaled_table(5000, rotary)
        qd, kd, vd = dev(q), dev(k), dev(v)
        out = torch.zeros_like(qd) if rotary < d else None  # (and in place)
        got = pa.rope_kv_write_layout(qd, kd, vd, dev(pos), dev(slots), dev(table), cache,
                                      "half" if half else "interleaved", layer=1, q_out=out,
                                      status=status)
        assert got is (qd if out is None else out) and int(status.item()) == 0
        assert np.array_equal(bits(got), bits(orc.rope_layout_pinned(q, pos, table, half)))
        if out is not None:
            assert np.array_equal(bits(qd), bits(q))
        assert np.array_equal(bits(kd), bits(k)) and np.array_equal(bits(vd), bits(v))
        orc.kv_write(pool, 1, orc.rope_layout_pinned(k, pos, table, half), v, slots)
        assert np.array_equal(bits(cache.tensor), bits(pool))


def test_append_whole_interleaved_heads_is_rope_kv_write():
    rng = np.random.default_rng(5)
    for T in (3, 3000):
        H, Hk, d, NB = 8, 4, 128, T // 16 + 1
        q, k, v = (dev(normal16(rng, T, n, d)) for n in (H, Hk, Hk))
        pos, slots = dev(rng.integers(0, 900, T).astype(np.int32)), ints(list(range(T)))
        table = pa.rope_table(900, d)
        pool = np.zeros((2, 1, NB, 16, Hk, d), np.float16)
        one, two = cache_of(pool), cache_of(pool)
        out = pa.rope_kv_write_layout(q, k, v, pos, slots, table, one, "interleaved",
                                      q_out=torch.empty_like(q))
        pa.rope_kv_write(q, k, v, pos, slots, table, two)
        assert torch.equal(out, q) and torch.equal(one.tensor, two.tensor)


@pytest.mark.parametrize("T", [6, 2000])
def test_append_reports_bad_positions_and_slots(T):
    rng = np.random.default_rng(12)
    H, Hk, d, NB = 8, 2, 128, T // 16 + 2
    q, k, v = normal16(rng, T, H, d), normal16(rng, T, Hk, d), normal16(rng, T, Hk, d)
    pos = rng.integers(0, 50, T).astype(np.int32)
    slots = rng.permutation(NB * 16)[:T].astype(np.int32)
    good = slots.copy()
    pos[1], pos[2] = -1, 50
    slots[4] = NB * 16
    good[[1, 2, 4]] = -1
    pool = normal16(rng, 2, 1, NB, 16, Hk, d)
    cache, status = cache_of(pool), pa.new_status()
    out = torch.full((T, H, d), 7.0).half().cuda()
    table = orc.rope_scaled_table(50, 64)
    pa.rope_kv_write_layout(dev(q), dev(k), dev(v), dev(pos), dev(slots), dev(table), cache, "half",
                            q_out=out, status=status)
    assert int(status.item()) == pa.PA_DEV_BAD_POSITION | pa.PA_DEV_BAD_SLOT
    safe = np.clip(pos, 0, 49)
    want = orc.rope_layout_pinned(q, safe, table, True)
    want[[1, 2]] = 7
    assert np.array_equal(bits(out), bits(want))
    orc.kv_write(pool, 0, orc.rope_layout_pinned(k, safe, table, True), v, good)
    assert np.array_equal(bits(cache.tensor), bits(pool))


@pytest.mark.parametrize("kw", [
    dict(), dict(scaling="linear", factor=4.0), dict(scaling="ntk", factor=8.0),
    dict(scaling="yarn", factor=16.0, original_positions=4096, high=32.0),
    dict(scaling="yarn", factor=4.0, original_positions=64, high=32.0, attention=1.5),
    dict(scaling="bands", factor=8.0, original_positions=8192, theta=5e5),
    dict(scaling="linear", factor=1.0, attention=0.5)])
@pytest.mark.parametrize("rotary", [16, 96, 128])
def test_scaled_tables(rotary, kw):
    got = pa.rope_table_scaled(3000, rotary, **kw).cpu().numpy()
    want = orc.rope_scaled_table(3000, rotary, **{**dict(high=4.0), **kw})
    # an angle below 3000 after frequencies that agree to a few 2^-53, and one rounding
    # to fp32 of a value of at most 1.5
    assert got.shape == (3000, rotary // 2, 2)
    assert np.abs(got.astype(np.float64) - want).max() <= 1.5 * 2.0 ** -23
    if not kw:
        assert np.array_equal(got, pa.rope_table(3000, rotary).cpu().numpy())


# ------------------------------------------------------------------ shared prefixes

class SharedBatch:
    """Groups (shared blocks, own tokens of each sequence) over one pool; values of
    places that no sequence has written are NaN."""

    def __init__(self, seed, H, Hk, d, groups, layers=1, layer=0, std=1.0):
        rng = np.random.default_rng(seed)
        self.H, self.Hk, self.d = H, Hk, d
        tails = [t for _, own in groups for t in own]
        pre = [b for b, own in groups for _ in own]
        need = sum(b for b, _ in groups) + sum(-(-t // 16) for t in tails)
        self.NB = need + 3
        order = rng.permutation(self.NB)
        width = max(max(b + -(-t // 16) for b, t in zip(pre, tails)), 1)
        self.bt = np.full((len(tails), width), -1, np.int32)
        self.pool = np.full((2, layers, self.NB, 16, Hk, d), np.nan, np.float16)
        at, s = 0, 0
        for b, own in groups:
            head = order[at:at + b]
            at += b
            self.pool[:, layer, head] = normal16(rng, 2, b, 16, Hk, d, std=std)
            for t in own:
                n = -(-t // 16)
                mine = order[at:at + n]
                at += n
                self.bt[s, :b], self.bt[s, b:b + n] = head, mine
                rows = normal16(rng, 2, n, 16, Hk, d, std=std).reshape(2, n * 16, Hk, d)
                rows[:, t:] = np.nan
                self.pool[:, layer, mine] = rows.reshape(2, n, 16, Hk, d)
                s += 1
        self.ctx = np.array([16 * b + t for b, t in zip(pre, tails)], np.int32)
        sizes = [len(own) for _, own in groups]
        self.starts = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
        self.shared = np.array([b for b, _ in groups], np.int32)
        self.q = normal16(rng, len(tails), H, d)
        self.layer = layer

    def run(self, ws=None, out=None, status=None, **kw):
        B = len(self.ctx)
        ws = pa.decode_shared_workspace(B, self.H, self.Hk, self.d) if ws is None else ws
        return pa.decode_shared(dev(self.q), cache_of(self.pool), dev(self.bt), dev(self.ctx),
                                dev(self.starts), dev(self.shared), ws, self.Hk, layer=self.layer,
                                out=out, status=status, **kw)

    def want(self, **kw):
        with np.errstate(invalid="ignore"):
            return orc.attention_decode(self.q, self.pool, self.layer, self.bt, self.ctx, self.H,
                                        self.Hk, **kw)


SHARED = [
    [(5, [3, 9, 1, 17])],
    [(8, [1, 16])],
    [(9, [0, 5, 0])],                        # nothing of one's own
    [(0, [5, 40]), (20, [7]), (33, [1] * 3)],  # nothing shared, one sequence, three
    [(1, [2] * 12), (2, [33] * 2), (17, list(range(1, 20)))],
    [(64, [1 + i % 30 for i in range(40)])],   # more sequences than a unit takes
    [(300, [5, 300])],                        # long: cut among many CTAs
    [(130, [0] * 5), (7, [100] * 3), (130, [64, 1])],
]


@pytest.mark.parametrize("H,Hk,d", [(4, 2, 64), (14, 2, 64), (8, 1, 128), (12, 4, 128), (6, 6, 128),
                                    (40, 8, 64)])
@pytest.mark.parametrize("groups", range(len(SHARED)))
def test_shared_matches_oracle(H, Hk, d, groups):
    b = SharedBatch(groups, H, Hk, d, SHARED[groups])
    status = pa.new_status()
    out = b.run(status=status)
    assert int(status.item()) == 0
    assert_attention_close(out, b.want())


def test_shared_large_batch():
    """More sequences of a group than fit two tiles, for 1 and 8 Q heads a KV head."""
    for H, Hk in ((2, 2), (8, 1)):
        b = SharedBatch(1, H, Hk, 128, [(40, [1 + i % 5 for i in range(300)]), (3, [1] * 9)])
        assert_attention_close(b.run(), b.want())


@pytest.mark.parametrize("H,Hk,d", [(1, 1, 64), (8, 1, 128), (6, 2, 128)])
@pytest.mark.parametrize("blocks", [list(range(1, 13)), [9, 8, 1], [40, 2, 70], [3] * 90, [900, 1]])
def test_shared_tails_in_pieces(H, Hk, d, blocks):
    """Tails cut into one piece (a block a CTA where there are few) up to many: those
    that the join takes from the CTAs' records, and those merged before it; alone ones
    beside them.  The workspace has held other shapes; twice the same bits."""
    ws = pa.decode_shared_workspace(128, H, Hk, d)
    SharedBatch(7, H, Hk, d, [(20, [1 + 37 * i % 90 for i in range(100)])]).run(ws=ws)
    b = SharedBatch(len(blocks), H, Hk, d, [(10, [16 * n - n % 3 for n in blocks]), (0, [50, 130])])
    status = pa.new_status()
    out = b.run(ws=ws, status=status)
    assert int(status.item()) == 0
    assert_attention_close(out, b.want())
    assert torch.equal(out, b.run(ws=ws))


def test_shared_scale_layer_and_large_scores():
    b = SharedBatch(3, 8, 2, 128, [(40, [9, 30, 1])], layers=3, layer=2, std=8.0)
    assert_attention_close(b.run(), b.want())
    assert_attention_close(b.run(scale=0.01), b.want(scale=0.01))


def test_shared_many_groups():
    """Hundreds of groups, empty ones among them, a workspace used for batches of
    several shapes."""
    rng = np.random.default_rng(9)
    groups = [(int(rng.integers(0, 12)), [int(x) for x in rng.integers(1, 30, rng.integers(1, 4))])
              for _ in range(150)]
    b = SharedBatch(2, 4, 2, 64, groups)
    starts = np.sort(np.concatenate([b.starts, rng.choice(b.starts, 20)])).astype(np.int32)
    shared = np.array([b.shared[np.searchsorted(b.starts, s)] if e > s else 10**6
                       for s, e in zip(starts, starts[1:])], np.int32)
    b.starts, b.shared = starts, shared
    ws = pa.decode_shared_workspace(400, 4, 2, 64)
    want = b.want()
    for _ in range(2):
        assert_attention_close(b.run(ws=ws), want)
        c = SharedBatch(7, 4, 2, 64, [(50, [4, 4, 4])])
        assert_attention_close(c.run(ws=ws), c.want())


@pytest.mark.parametrize("sink", [0.5, 0.9, 0.99])
def test_shared_beside_a_dominant_key(sink):
    """One key of value zero has `sink` of the weight, the others the rest: each is a
    probability near 1e-6 of the largest."""
    H, Hk, d, n = 8, 1, 128, 512  # blocks
    b = SharedBatch(5, H, Hk, d, [(n, [40, 40])], std=0.1)
    N = 16 * n + 40
    b.q[:] = 1
    gap = math.log(sink * N / (1 - sink)) * math.sqrt(d) / d
    b.pool[0] = 0
    b.pool[0, 0, b.bt[0, 0], 0] = gap
    b.pool[1, 0, b.bt[0, 0], 0] = 0
    got, want = b.run().double().cpu().numpy(), b.want()
    # three roundings of 2^-11 of values whose errors are independent, beside the output's
    # own rounding: at 0.99 it is near 0.01 * 0.1 / sqrt(8232) = 1.1e-5, below fp16's least
    # normal number, where half a step (2^-25) is 2.7e-3 of it
    beyond = np.maximum(np.abs(got - want) - half_ulp16(want), 0)
    rel = np.linalg.norm(beyond) / np.linalg.norm(want)
    assert rel <= 1e-3, rel


def test_shared_leaves_out_what_is_out_of_order():
    groups = [(20, [3, 9, 1]), (12, [5, 5]), (9, [2, 3, 4])]
    for change in ("length", "first", "short", "blocks", "negative", "starts", "tail block"):
        b = SharedBatch(11, 8, 2, 64, groups)
        want, bad, bit = b.want(), [], pa.PA_DEV_BAD_LENGTH
        if change == "length":
            b.ctx[1], bad = 16 * b.bt.shape[1] + 1, [1]
        if change == "first":  # a padded place: its table is not read
            b.ctx[0], b.bt[0], bad = 0, 10**6, [0]
        if change == "short":
            b.ctx[4], bad = 16 * 12 - 1, [4]
        if change == "blocks":
            b.shared[1], bad = b.bt.shape[1] + 1, [3, 4]
        if change == "negative":
            b.shared[2], bad = -1, [5, 6, 7]
        if change == "starts":
            b.starts[1], bad = 6, list(range(8))
            b.starts[2] = 3
        if change == "tail block":
            bit, b.bt[3, 12] = pa.PA_DEV_BAD_BLOCK, b.NB
            w = SharedBatch(11, 8, 2, 64, groups)  # its 5 tokens drop out
            w.ctx[3] = 16 * 12
            want = w.want()
        status, out = pa.new_status(), torch.full(b.q.shape, 7.0).half().cuda()
        ws = pa.decode_shared_workspace(8, 8, 2, 64)
        b.run(ws=ws, out=out, status=status)
        assert int(status.item()) == bit, change
        good = [s for s in range(8) if s not in bad]
        assert (out[bad] == 7).all(), change
        if good:
            assert_attention_close(out[good], want[good])
        b = SharedBatch(12, 8, 2, 64, groups)  # the workspace is as it was
        assert_attention_close(b.run(ws=ws), b.want())


def test_shared_block_out_of_range_drops_out():
    b = SharedBatch(13, 8, 2, 128, [(30, [3, 9, 1])])
    b.bt[:, 7], b.bt[:, 20] = -1, b.NB
    status = pa.new_status()
    out = b.run(status=status)
    assert int(status.item()) == pa.PA_DEV_BAD_BLOCK
    cut = SharedBatch(13, 8, 2, 128, [(30, [3, 9, 1])])
    cut.bt = np.delete(cut.bt, [7, 20], axis=1)
    cut.ctx -= 32
    assert_attention_close(out, cut.want())


def test_shared_in_a_graph_and_on_a_stream():
    b = SharedBatch(14, 8, 2, 128, [(40, [9, 30, 1]), (16, [50, 2])])
    want = b.want()
    args = [dev(b.q), cache_of(b.pool), dev(b.bt), dev(b.ctx), dev(b.starts), dev(b.shared)]
    ws, out = pa.decode_shared_workspace(5, 8, 2, 128), torch.empty_like(args[0])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = pa.decode_shared(*args, ws, 2, stream=side)
    side.synchronize()
    assert_attention_close(got, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pa.decode_shared(*args, ws, 2, out=out)
    for _ in range(3):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, got)  # the same bits each time
    args[4].copy_(ints([0, 5, 5]))  # other groups between replays: none shares
    args[5].zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert_attention_close(out, want)


def test_shared_flat_history():
    """65536 keys of equal weight and values of one sign, whose sums grow as they can."""
    b = SharedBatch(17, 8, 1, 128, [(4096, [5, 40])])
    b.pool[0] = 0
    b.pool[1] = 0.5 + 0.01 * b.pool[1].astype(np.float32)
    assert_attention_close(b.run(), b.want())


@pytest.mark.parametrize("value", [65504, -65504])
def test_values_at_the_end_of_the_range(value):
    """Averages of finite values stay finite: within a rounding of P (2^-11) of V's."""
    b = SharedBatch(16, 8, 2, 128, [(40, [9, 300, 0]), (0, [77])], std=3.0)
    b.pool[1] = value
    w = WeightBatch(16, 8, 2, 128, [300, 9], std=3.0)
    w.pool[1] = value
    for out in (b.run(), w.run()[0]):
        out = out.float().cpu().numpy()
        assert np.isfinite(out).all() and np.abs(out - value).max() <= 65504 * 2.0 ** -11 + 16


def test_shared_nan_reaches_its_own_rows_alone():
    b = SharedBatch(15, 4, 2, 64, [(20, [3, 9, 1])])
    b.q[1, 3, 5] = np.nan
    out = b.run()
    nan = torch.isnan(out).flatten(1)
    assert nan[1].view(4, 64)[3].all() and int(nan.sum()) == 64
    keep = torch.ones(3, 4, dtype=torch.bool)
    keep[1, 3] = False
    assert_attention_close(out.cpu()[keep].float().numpy().astype(np.float64), b.want()[keep.numpy()])


# ------------------------------------------------------------------ accumulated weights

class WeightBatch:
    def __init__(self, seed, H, Hk, d, lens, layers=1, layer=0, std=1.0):
        rng = np.random.default_rng(seed)
        self.H, self.Hk, self.d, self.layer = H, Hk, d, layer
        self.ctx = np.array(lens, np.int32)
        need = [-(-n // 16) for n in lens]
        self.NB = sum(need) + 2
        order = rng.permutation(self.NB).astype(np.int32)
        self.bt = np.full((len(lens), max(max(need), 1)), -1, np.int32)
        self.pool = np.full((2, layers, self.NB, 16, Hk, d), np.nan, np.float16)
        at = 0
        for s, n in enumerate(lens):
            mine = order[at:at + need[s]]
            at += need[s]
            self.bt[s, :need[s]] = mine
            rows = normal16(rng, 2, need[s] * 16, Hk, d, std=std)
            rows[:, n:] = np.nan
            self.pool[:, layer, mine] = rows.reshape(2, need[s], 16, Hk, d)
        self.q = normal16(rng, len(lens), H, d)
        self.stride = 16 * self.bt.shape[1] + 3
        self.w = rng.random((len(lens), Hk, self.stride)).astype(np.float32)
        for s, n in enumerate(lens):
            self.w[s, :, n:] = 0
        self.blocks = sum(need)

    def want(self):
        """The weights, and how far fp32 may take them."""
        with np.errstate(invalid="ignore"):
            p = orc.decode_weights(self.q, self.pool, self.layer, self.bt, self.ctx, self.H, self.Hk)
        w, tol = self.w.astype(np.float64), np.zeros(self.w.shape)
        g = self.H // self.Hk
        for s, n in enumerate(self.ctx):
            K, _ = orc.gather_kv(self.pool, self.layer, self.bt[s], int(n))
            size = max(np.abs(self.q[s, h].astype(np.float64)) @ np.abs(K[:, h // g]).T.max(-1)
                       for h in range(self.H))
            w[s, :, :n] += p[s]
            # a score is a sum of d products, cut or rounded by 2^-23 of the sum of their
            # sizes at each; twice that in the exponent (the row's sum too), then a
            # handful of roundings, and those of g + 1 additions
            rel = np.expm1(2 * self.d * 2.0 ** -23 * size / math.sqrt(self.d)) + 16 * 2.0 ** -23
            tol[s, :, :n] = p[s] * rel + (g + 1) * 2.0 ** -24 * w[s, :, :n]
        return w, tol

    def run(self, weights="in", ws=None, **kw):
        ws = ws if ws is not None else pa.decode_weights_workspace(len(self.ctx), self.H, self.Hk,
                                                                   self.d, self.blocks)
        w = dev(self.w) if weights == "in" else weights
        return pa.decode_weights(dev(self.q), cache_of(self.pool), dev(self.bt), dev(self.ctx), w, ws,
                                 self.Hk, layer=self.layer, **kw)

    def out(self):
        with np.errstate(invalid="ignore"):
            return orc.attention_decode(self.q, self.pool, self.layer, self.bt, self.ctx, self.H,
                                        self.Hk)


@pytest.mark.parametrize("H,Hk,d", [(4, 2, 64), (14, 2, 64), (8, 1, 128), (12, 4, 128), (6, 6, 128),
                                    (10, 2, 128), (40, 8, 64), (6, 1, 64)])
@pytest.mark.parametrize("lens", [[1], [16, 1, 17], [300, 5, 33, 64], [5000], [1] * 70])
def test_weights_match_oracle(H, Hk, d, lens):
    b = WeightBatch(len(lens), H, Hk, d, lens)
    status = pa.new_status()
    out, got = b.run(status=status)
    assert int(status.item()) == 0
    assert_attention_close(out, b.out())
    want, tol = b.want()
    got = got.cpu().numpy()
    assert (np.abs(got - want) <= tol).all()
    for s, n in enumerate(lens):
        assert (got[s, :, n:] == 0).all()


def test_weights_from_nothing_and_beside():
    b = WeightBatch(3, 8, 2, 128, [100, 7, 40], layers=2, layer=1)
    want, tol = b.want()
    zero = dev(np.full_like(b.w, 7.0))
    _, got = b.run(weights=None, weights_out=zero)
    assert got is zero
    got, before = got.cpu().numpy(), dev(b.w)
    for s, n in enumerate(b.ctx):
        fresh = want[s, :, :n] - b.w[s, :, :n]
        assert (np.abs(got[s, :, :n] - fresh) <= tol[s, :, :n] + 2.0 ** -24).all()
        assert (got[s, :, n:] == 7).all()  # places behind the context stay
    _, apart = b.run(weights=before, weights_out=dev(np.zeros_like(b.w)))
    assert np.array_equal(before.cpu().numpy(), b.w)
    assert (np.abs(apart.cpu().numpy() - want) <= tol).all()


@pytest.mark.parametrize("g", range(1, 9))
def test_weights_one_workspace_again(g):
    """Batches of several shapes by turns in one workspace, whose scores' lines the
    second kernel gives up: pairs in one to many pieces, padded blocks, odd groups."""
    batches = [WeightBatch(g, 2 * g, 2, 64, lens)
               for lens in ([128, 16 * 9 + 1, 7, 33], [40] * 30 + [1], [3000, 2], list(range(1, 180, 9)))]
    ws = pa.decode_weights_workspace(31, 2 * g, 2, 64, max(b.blocks for b in batches))
    for b in batches + batches[::-1]:
        status = pa.new_status()
        out, got = b.run(ws=ws, status=status)
        assert int(status.item()) == 0
        assert_attention_close(out, b.out())
        want, tol = b.want()
        assert (np.abs(got.cpu().numpy() - want) <= tol).all()


def test_weights_sum_to_the_heads():
    """Every row's weights sum to the group's size, over lengths of all sorts."""
    b = WeightBatch(4, 32, 4, 64, [1, 2, 15, 16, 17, 1000, 4097, 31])
    _, got = b.run(weights=None, weights_out=dev(np.zeros_like(b.w)))
    total = got.double().sum(-1).cpu().numpy()
    assert np.abs(total - 8).max() <= 8 * 2e-5


def test_weights_bad_lengths_blocks_and_little_room():
    lens = [100, 30, 50, 64]
    b = WeightBatch(5, 8, 2, 64, lens)
    want, tol = b.want()
    out_want = b.out()
    b.ctx[1] = 0
    status, out = pa.new_status(), torch.full(b.q.shape, 7.0).half().cuda()
    _, got = b.run(out=out, status=status)
    assert int(status.item()) == pa.PA_DEV_BAD_LENGTH
    got = got.cpu().numpy()
    ok = [0, 2, 3]
    assert (out[1] == 7).all() and np.array_equal(got[1], b.w[1])
    assert_attention_close(out[ok], out_want[ok])
    assert (np.abs(got - want)[ok] <= tol[ok]).all()
    # a context longer than the rows of weights
    b = WeightBatch(5, 8, 2, 64, lens)
    b.w = np.ascontiguousarray(b.w[..., :99])
    status, out = pa.new_status(), torch.full(b.q.shape, 7.0).half().cuda()
    _, got = b.run(out=out, status=status)
    assert int(status.item()) == pa.PA_DEV_BAD_LENGTH and (out[0] == 7).all()
    assert np.array_equal(got[0].cpu().numpy(), b.w[0])
    assert (np.abs(got.cpu().numpy()[1:] - want[1:, :, :99]) <= tol[1:, :, :99]).all()
    # scores for the first two sequences alone: 7 + 2 blocks of 7 + 2 + 4 + 4
    b = WeightBatch(5, 8, 2, 64, lens)
    ws = pa.decode_weights_workspace(4, 8, 2, 64, 10)
    status = pa.new_status()
    out, got = b.run(ws=ws, status=status)
    assert int(status.item()) == pa.PA_DEV_WORKSPACE
    assert_attention_close(out, out_want)
    got = got.cpu().numpy()
    assert (np.abs(got - want)[:2] <= tol[:2]).all() and np.array_equal(got[2:], b.w[2:])
    # a block out of range drops out of the attention, and gets no weight
    b = WeightBatch(5, 8, 2, 64, lens)
    b.bt[0, 2] = b.NB
    status = pa.new_status()
    _, got = b.run(status=status)
    assert int(status.item()) == pa.PA_DEV_BAD_BLOCK
    got = got.cpu().numpy()
    assert np.array_equal(got[0, :, 32:48], b.w[0, :, 32:48])
    assert np.abs((got - b.w)[0].sum(-1) - 4).max() <= 4e-5


def test_weights_in_a_graph_accumulate():
    b = WeightBatch(6, 8, 2, 128, [100, 7, 1000])
    want, tol = b.want()
    args = [dev(b.q), cache_of(b.pool), dev(b.bt), dev(b.ctx), dev(np.zeros_like(b.w))]
    ws, out = pa.decode_weights_workspace(3, 8, 2, 128, b.blocks), torch.empty_like(args[0])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    pa.decode_weights(*args, ws, 2, out=out, stream=side)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pa.decode_weights(*args, ws, 2, out=out)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    got = args[4].cpu().numpy()
    fresh = want - b.w
    assert (np.abs(got - 4 * fresh) <= 4 * tol + 2.0 ** -22 * got).all()


# ------------------------------------------------------------------ eviction

class EvictBatch(WeightBatch):
    def run(self, budget, sinks=0, recent=0, to=None, **kw):
        self.cache = cache_of(self.pool)
        ws = pa.kv_evict_workspace(len(self.ctx), self.Hk, budget)
        return pa.kv_evict(self.cache, dev(self.bt), dev(self.ctx), dev(self.w), budget, ws,
                           sinks=sinks, recent=recent, layer=self.layer,
                           out_block_tables=None if to is None else dev(to), **kw)

    def check(self, budget, sinks=0, recent=0, to=None):
        pool, w = self.pool.copy(), self.w.copy()
        n = orc.evict(pool, self.layer, self.bt, self.ctx, w, budget, sinks, recent,
                      self.bt if to is None else to)
        status = pa.new_status()
        got_w, got_n = self.run(budget, sinks, recent, to, status=status)
        assert int(status.item()) == 0
        assert np.array_equal(got_n.cpu().numpy(), n)
        assert np.array_equal(got_w.cpu().numpy().view(np.uint32), w.view(np.uint32))
        assert np.array_equal(bits(self.cache.tensor), bits(pool))


EVICT = [([1], 1, 0, 0), ([40, 0, 1, 33], 16, 2, 5), ([700, 200, 256, 257], 256, 4, 64),
         ([9000, 100], 1000, 4, 256), ([300], 299, 0, 299), ([300, 5000], 300, 300, 0),
         ([5000], 4999, 0, 0), ([20000], 1, 0, 0), ([4096, 4097, 8192], 2048, 1, 1), ([64] * 50, 10, 0, 3),
         ([70000], 3000, 0, 7), ([40000] + [20] * 79, 500, 4, 64)]


@pytest.mark.parametrize("H,Hk,d", [(2, 2, 64), (8, 8, 128), (1, 1, 128)])
@pytest.mark.parametrize("case", range(len(EVICT)))
def test_evict_in_place(H, Hk, d, case):
    lens, budget, sinks, recent = EVICT[case]
    EvictBatch(case, H, Hk, d, lens, layers=2, layer=1).check(budget, sinks, recent)


@pytest.mark.parametrize("values", ["equal", "few", "zeros", "signs", "nan", "tiny", "ordered"])
def test_evict_ties_and_odd_weights(values):
    for n, budget in ((100, 37), (6000, 1500), (5000, 4)):
        b = EvictBatch(1, 2, 2, 64, [n])
        rng = np.random.default_rng(n)
        shape = b.w[..., :n].shape
        w = {"equal": lambda: np.full(shape, 0.25), "zeros": lambda: np.zeros(shape),
             "few": lambda: rng.integers(0, 3, shape) / 2,
             "signs": lambda: rng.choice([-1.5, -0.0, 0.0, 1.5, np.inf, -np.inf], shape),
             "nan": lambda: np.where(rng.random(shape) < 0.9, np.nan, rng.random(shape)),
             "tiny": lambda: rng.integers(0, 50, shape) * 2.0 ** -149,
             "ordered": lambda: np.broadcast_to(np.arange(n)[::-1], shape)}[values]()
        b.w[..., :n] = w
        b.check(budget)
        b.check(budget, 2, min(budget - 3, 40))


def test_evict_into_other_blocks():
    """Wholly, and only the first blocks (a shared prefix): the old rows stay."""
    for whole in (True, False):
        b = EvictBatch(2, 4, 4, 128, [500, 130, 77])
        spare = np.setdiff1d(np.arange(b.NB), b.bt)
        more = 30
        b.pool = np.concatenate([b.pool, np.full_like(b.pool[:, :, :more], 7)], 2)
        fresh = np.concatenate([spare, np.arange(b.NB, b.NB + more)]).astype(np.int32)
        b.NB += more
        to = b.bt.copy() if not whole else np.full((3, 8), -1, np.int32)
        at = 0
        for s in range(3):
            n = 7 if whole else 3
            to[s, :n] = fresh[at:at + n]
            at += n
        b.check(100, 4, 20, to)
        old = b.bt[0, :3]
        assert np.array_equal(bits(b.cache.tensor[:, 0, dev(old).long()]), bits(b.pool[:, 0, old]))


def test_evict_leaves_out_what_is_out_of_order():
    b = EvictBatch(3, 2, 2, 64, [200, 300, 100, 250])
    pool, w = b.pool.copy(), b.w.copy()
    ctx = b.ctx.copy()
    b.ctx[:] = [-1, 16 * b.bt.shape[1] + 1, 100, 250]
    lens = torch.full((4,), 99, dtype=torch.int32, device="cuda")
    to = b.bt[:, :4].copy()  # room for 64 tokens
    status = pa.new_status()
    got, n = b.run(80, to=to, status=status, out_context_lens=lens)
    assert int(status.item()) == pa.PA_DEV_BAD_LENGTH
    assert n is lens and n.tolist() == [99] * 4  # (80 tokens do not fit four blocks)
    assert np.array_equal(bits(b.cache.tensor), bits(pool)) and np.array_equal(got.cpu().numpy(), w)
    # a block out of range: its rows stay, the others move
    b.ctx = ctx
    b.bt[0, 3] = b.NB
    status = pa.new_status()
    _, n = b.run(80, status=status)
    assert int(status.item()) == pa.PA_DEV_BAD_BLOCK and n.tolist() == [80] * 4
    want_w = b.w.copy()
    orc_bt = b.bt.copy()
    orc_bt[0, 3] = 0
    orc.evict(pool, 0, orc_bt, ctx, want_w, 80, 0, 0, orc_bt)
    for s in (1, 2, 3):
        blocks = dev(b.bt[s, :-(-ctx[s] // 16)]).long()
        assert np.array_equal(bits(b.cache.tensor[:, 0, blocks]), bits(pool[:, 0, blocks.cpu().numpy()]))


def test_evict_weights_beside_and_graph():
    b = EvictBatch(4, 4, 4, 64, [500, 130, 77])
    pool, want = b.pool.copy(), b.w.copy()
    n = orc.evict(pool, 0, b.bt, b.ctx, want, 100, 4, 20, b.bt)
    want[:, :, max(b.ctx):] = 5
    for s in range(3):
        want[s, :, b.ctx[s]:] = 5
    cache, w, lens = cache_of(b.pool), dev(b.w), dev(b.ctx)
    out, out_lens = torch.full_like(w, 5.0), torch.zeros_like(lens)
    ws, bt = pa.kv_evict_workspace(3, 4, 100), dev(b.bt)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pa.kv_evict(cache, bt, lens, w, 100, ws, sinks=4, recent=20, weights_out=out,
                    out_context_lens=out_lens)
    graph.replay()
    torch.cuda.synchronize()
    assert np.array_equal(out.cpu().numpy(), want) and np.array_equal(out_lens.cpu().numpy(), n)
    assert np.array_equal(w.cpu().numpy(), b.w) and np.array_equal(lens.cpu().numpy(), b.ctx)
    assert np.array_equal(bits(cache.tensor), bits(pool))


# ------------------------------------------------------------------ together

def test_binding_refusals():
    b = WeightBatch(1, 4, 2, 64, [20, 3])
    q, bt, ctx, w = dev(b.q), dev(b.bt), dev(b.ctx), dev(b.w)
    cache, i4 = cache_of(b.pool), pa.CacheI4(1, 4, 2, 64)
    ws = pa.decode_weights_workspace(2, 4, 2, 64, 3)
    starts, shared = ints([0, 2]), ints([0])
    ws_s, ws_e = pa.decode_shared_workspace(2, 4, 2, 64), pa.kv_evict_workspace(2, 2, 8)
    with pytest.raises(TypeError):
        pa.decode_weights(q, i4, bt, ctx, w, ws, 2)
    with pytest.raises(ValueError):
        pa.decode_weights(q, cache, bt, ctx, w[:, :1].contiguous(), ws, 2)
    with pytest.raises(TypeError):
        pa.decode_weights(q, cache, bt, ctx, w.double(), ws, 2)
    with pytest.raises(TypeError):
        pa.decode_weights(q, cache, bt, ctx, w[..., ::2], ws, 2)
    with pytest.raises(pa.PAError):
        pa.decode_weights(q, cache, bt, ctx, w, ws[:256], 2)
    with pytest.raises(ValueError):
        pa.decode_shared(q, cache, bt, ctx, ints([0, 1, 2]), shared, ws_s, 2)
    with pytest.raises(ValueError):
        pa.decode_shared(q, cache, bt, ctx, starts, shared, ws_s, 2, layer=2**32)
    with pytest.raises(pa.PAError):
        pa.decode_shared(q, cache, bt, ctx, starts[:1], shared[:0], ws_s, 2)
    with pytest.raises(ValueError):
        pa.kv_evict(cache, bt, ctx, w, 2**32 + 8, ws_e)
    with pytest.raises(ValueError):
        pa.kv_evict(cache, bt, ctx[:1], w, 8, ws_e)
    with pytest.raises(pa.PAError):
        pa.kv_evict(cache, bt, ctx, w, 8, ws_e, sinks=5, recent=4)
    with pytest.raises(TypeError):
        pa.kv_evict(i4, bt, ctx, w, 8, ws_e)
    x = torch.zeros(2, 2, 64, dtype=torch.float16, device="cuda")
    with pytest.raises(ValueError):
        pa.rope_kv_write_layout(q, x, x, ctx, ctx, pa.rope_table(8, 64), cache, "other")
    with pytest.raises(pa.PAError):
        pa.rope_kv_write_layout(q, x, x, ctx, ctx, pa.rope_table(8, 24), cache, "half")
    with pytest.raises(ValueError):
        pa.Cache(1, b.NB, 2, 64, library_owned=True, tensor=dev(b.pool))
    with pytest.raises(ValueError):
        pa.Cache(1, b.NB + 1, 2, 64, tensor=dev(b.pool))


@pytest.mark.parametrize("H,Hk,d", [(8, 2, 64), (4, 4, 128)])
def test_serving_loop(H, Hk, d):
    """Prompts with a common beginning through the block manager: prefill in the half
    layout with a scaled table, decode with the prefix shared, decode that accumulates
    weights, eviction into fresh blocks, and decode on at the true positions."""
    rng = np.random.default_rng(8)
    B, common, NB = 3, 64, 96
    bm = pa.BlockManager(NB)
    prompts = [list(range(common)) + [100 * (i + 1) + j for j in range(5 + 7 * i)] for i in range(B)]
    scaling = dict(scaling="bands", factor=4.0, original_positions=64)
    table, host_table = pa.rope_table_scaled(400, d // 2, **scaling), None
    host_table = orc.rope_scaled_table(400, d // 2, **scaling)
    cache = pa.Cache(1, NB, Hk, d)
    cache.tensor.zero_()
    pool = np.zeros((2, 1, NB, 16, Hk, d), np.float16)
    width, status = 8, pa.new_status()
    bt = np.full((B, width), -1, np.int32)

    def append(q, k, v, pos, slots):
        out = pa.rope_kv_write_layout(dev(q), dev(k), dev(v), dev(pos), dev(slots), table, cache,
                                      "half", status=status)
        q_rot, k_rot = (orc.rope_layout_pinned(x, pos, host_table, True) for x in (q, k))
        orc.kv_write(pool, 0, k_rot, v, slots)
        assert np.array_equal(bits(out), bits(q_rot))
        return out, q_rot

    for i in range(B):
        cached = bm.allocate(i, prompts[i])
        assert cached == (common if i else 0)
        bt[i, :len(bm.block_table(i))] = bm.block_table(i)
        new = len(prompts[i]) - cached
        md = pa.prepare_prefill([cached], [new], bt[i:i + 1])
        q, k, v = normal16(rng, new, H, d), normal16(rng, new, Hk, d), normal16(rng, new, Hk, d)
        qr, q_rot = append(q, k, v, md["positions"], md["slot_mapping"])
        out = pa.prefill_varlen(qr, cache, dev(md["cu_seqlens_q"]), dev(md["cu_seqlens_k"]),
                                dev(bt[i:i + 1]), md["max_seqlen_q"], Hk, status=status)
        want = orc.attention_prefill(q_rot, pool, 0, md["cu_seqlens_q"], md["cu_seqlens_k"],
                                     bt[i:i + 1], H, Hk)
        assert_attention_close(out, want)
        bm.mark_computed(i, new)

    w = torch.zeros(B, Hk, width * 16, device="cuda")
    ws_s = pa.decode_shared_workspace(B, H, Hk, d)
    ws_w = pa.decode_weights_workspace(B, H, Hk, d, B * width)
    want_w = np.zeros((B, Hk, width * 16))
    ctx = np.array([bm.num_tokens(i) for i in range(B)], np.int32)
    true_pos = ctx.copy()
    slots = np.zeros(B, np.int32)
    ctx_d = None
    for step in range(14):
        for i in range(B):
            slots[i] = bm.append(i, step)
            t = bm.block_table(i)
            bt[i, :len(t)] = t
        q, k, v = normal16(rng, B, H, d), normal16(rng, B, Hk, d), normal16(rng, B, Hk, d)
        qr, q_rot = append(q, k, v, true_pos, slots)
        true_pos += 1
        ctx += 1
        want = orc.attention_decode(q_rot, pool, 0, bt, ctx, H, Hk)
        if step == 0:
            groups = pa.prepare_shared(bt, ctx)
            assert groups["group_starts"].tolist() == [0, 3] and groups["shared_blocks"].tolist() == [4]
            out = pa.decode_shared(qr, cache, dev(bt), dev(ctx), dev(groups["group_starts"]),
                                   dev(groups["shared_blocks"]), ws_s, Hk, status=status)
        else:
            out, _ = pa.decode_weights(qr, cache, dev(bt), dev(ctx), w, ws_w, Hk, status=status)
            for s, x in enumerate(orc.decode_weights(q_rot, pool, 0, bt, ctx, H, Hk)):
                want_w[s, :, :ctx[s]] += x
        assert_attention_close(out, want)
        assert np.abs(w.cpu().numpy() - want_w).max() <= 1e-4
        assert [bm.num_tokens(i) for i in range(B)] == ctx.tolist() or step == 3
        if step == 3:
            # the weights decide: what the GPU added up goes into the oracle's eviction
            to = np.full((B, width), -1, np.int32)
            for i in range(B):
                bm.evict_begin(i, 40)
                to[i, :3] = bm.block_table(i)
            host_w = w.cpu().numpy()
            ctx_d = dev(ctx)
            pa.kv_evict(cache, dev(bt), ctx_d, w, 40, pa.kv_evict_workspace(B, Hk, 40), sinks=4,
                        recent=8, out_block_tables=dev(to), status=status)
            ctx = orc.evict(pool, 0, bt, ctx, host_w, 40, 4, 8, to)
            for i in range(B):
                bm.evict_end(i)
            assert len(set(to[:, :3].ravel())) == 3 * B  # (nothing shared any more)
            assert ctx.tolist() == [40] * B and np.array_equal(ctx_d.cpu().numpy(), ctx)
            assert np.array_equal(w.cpu().numpy(), host_w)
            want_w = host_w.astype(np.float64)
            bt = to
            assert np.array_equal(bits(cache.tensor), bits(pool))
    assert int(status.item()) == 0
