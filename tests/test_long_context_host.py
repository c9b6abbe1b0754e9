"""The long-context operators without a GPU: the oracle's functions pinned, the host
metadata of shared prefixes, sizes and refusals of the library's entry points."""

import ctypes
import math

import numpy as np
import pytest
import torch

from oracle import reference as orc
from paged_kv_gqa_rope_gb300 import pa

# ---------------------------------------------------------------- the oracle


def test_layouts_turn_the_same_pairs():
    """The half layout is the interleaved one after a permutation of the rotated values;
    values behind the rotated part pass; rope_pinned is the interleaved whole head."""
    rng = np.random.default_rng(0)
    x = rng.standard_normal((5, 3, 64)).astype(np.float16)
    pos = np.array([0, 1, 7, 300, 999])
    table = orc.rope_scaled_table(1000, 32)
    inter = orc.rope_layout_pinned(x, pos, table, False)
    order = np.concatenate([np.arange(0, 32, 2), np.arange(1, 32, 2)])
    y = x.copy()
    y[..., :32] = x[..., order]
    half = orc.rope_layout_pinned(y, pos, table, True)
    assert np.array_equal(half[..., :32], inter[..., order])
    assert np.array_equal(inter[..., 32:], x[..., 32:]) and np.array_equal(inter[0], x[0])
    whole = orc.rope_layout_pinned(x, pos, orc.rope_scaled_table(1000, 64), False)
    assert np.array_equal(whole, orc.rope_pinned(x, pos, 64))


def test_scaled_frequencies():
    plain, a = orc.rope_scaled_frequencies(64)
    assert a == 1 and np.allclose(plain, 10000.0 ** (-np.arange(32) / 32), rtol=1e-15)
    assert orc.rope_scaled_frequencies(64, scaling="linear", factor=4.0)[0] == [x / 4 for x in plain]
    f, _ = orc.rope_scaled_frequencies(64, scaling="ntk", factor=4.0)
    assert f[0] == 1 and math.isclose(f[-1], plain[-1] / 4)  # fastest kept, slowest slowed
    for kind, high in (("yarn", 32.0), ("bands", 4.0)):
        f, a = orc.rope_scaled_frequencies(128, theta=5e5, scaling=kind, factor=8.0,
                                           original_positions=8192, low=1.0, high=high)
        p, _ = orc.rope_scaled_frequencies(128, theta=5e5)
        ratio = np.array(f) / np.array(p)
        turns = 8192 * np.array(p) / (2 * math.pi)
        assert np.all(np.diff(ratio) <= 1e-15) and np.allclose(ratio[turns < 0.9], 1 / 8)
        assert np.all(ratio[turns > high * 1.3] == 1)
        assert a == (0.1 * math.log(8) + 1 if kind == "yarn" else 1)
    # bands, by hand: a pair that turns 2.5 times of (1, 4) is half kept
    L = 2 * math.pi * 2.5
    f, _ = orc.rope_scaled_frequencies(16, scaling="bands", factor=3.0, original_positions=L)
    assert math.isclose(f[0], 0.5 + 0.5 / 3)


def test_decode_weights_sum_and_give_the_output():
    rng = np.random.default_rng(1)
    cache = rng.standard_normal((2, 1, 5, 16, 2, 64)).astype(np.float16)
    q = rng.standard_normal((2, 6, 64)).astype(np.float16)
    bt = np.array([[0, 2, 4], [1, 3, 3]])
    w = orc.decode_weights(q, cache, 0, bt, [40, 1], 6, 2)
    assert np.allclose(w[0].sum(-1), 3) and np.allclose(w[1], 3)
    # one Q head a KV head: the weights times V are the output
    w = orc.decode_weights(q[:, :2], cache, 0, bt, [40, 17], 2, 2)
    out = orc.attention_decode(q[:, :2], cache, 0, bt, [40, 17], 2, 2)
    for s, n in enumerate((40, 17)):
        _, V = orc.gather_kv(cache, 0, bt[s], n)
        assert np.allclose(np.einsum("ht,thd->hd", w[s], V), out[s], atol=1e-12)


def test_evict_keep_worked_examples():
    w = np.array([0.1, 5.0, 0.3, 0.3, 0.0, 0.3, 2.0, 0.0])
    assert orc.evict_keep(w, 3, 0, 0) == [1, 2, 6]  # of the equal 0.3 the first
    assert orc.evict_keep(w, 4, 1, 1) == [0, 1, 6, 7]
    assert orc.evict_keep(w, 4, 0, 4) == [4, 5, 6, 7]
    assert orc.evict_keep(w, 8, 1, 1) == list(range(8))
    w[1] = np.nan
    assert orc.evict_keep(w, 1, 0, 0) == [6] and orc.evict_keep(w, 7, 0, 0) == [0, 2, 3, 4, 5, 6, 7]


# ---------------------------------------------------------------- metadata of shared prefixes


def saved(bt, ctx, starts, shared, bs=16):
    """Block reads saved, after checking that the groups are what they claim to be."""
    assert starts[0] == 0 and starts[-1] == len(ctx) and np.all(np.diff(starts) > 0)
    total = 0
    for a, b, n in zip(starts, starts[1:], shared):
        for s in range(a, b):
            assert n * bs <= ctx[s] and np.array_equal(bt[s, :n], bt[a, :n])
        assert n == 0 or b - a > 1
        total += (b - a - 1) * n
    return total


def test_prepare_shared_worked_example(libpa):
    bt = np.array([[1, 2, 3, 4], [1, 2, 3, 5], [1, 2, 6, -1], [7, 8, -1, -1], [7, 9, -1, -1],
                   [10, -1, -1, -1]], np.int32)
    got = pa.prepare_shared(bt, np.array([60, 64, 40, 20, 31, 5], np.int32))
    # 3 blocks of two sequences (3 saved) or 2 of three (4 saved)
    assert got["group_starts"].tolist() == [0, 3, 5, 6] and got["shared_blocks"].tolist() == [2, 1, 0]
    # a block that is not full in every sequence is not shared
    got = pa.prepare_shared(bt[:2], np.array([40, 33], np.int32))
    assert got["shared_blocks"].tolist() == [2]
    got = pa.prepare_shared(bt[:2], np.array([15, 64], np.int32))
    assert got["group_starts"].tolist() == [0, 1, 2] and got["shared_blocks"].tolist() == [0, 0]
    got = pa.prepare_shared(np.zeros((0, 3), np.int32), np.zeros(0, np.int32))
    assert got["group_starts"].tolist() == [0] and len(got["shared_blocks"]) == 0


def test_prepare_shared_random_batches(libpa):
    rng = np.random.default_rng(4)
    for _ in range(200):
        B, width = int(rng.integers(1, 12)), int(rng.integers(1, 7))
        bt = np.sort(rng.integers(0, 3, (B, width)), axis=0).astype(np.int32)
        ctx = rng.integers(0, 16 * width + 1, B).astype(np.int32)
        got = pa.prepare_shared(bt, ctx)
        total = saved(bt, ctx, got["group_starts"], got["shared_blocks"])
        pairs = [next((i for i in range(width) if bt[s, i] != bt[s - 1, i]), width)
                 for s in range(1, B)]
        most = [min(p, ctx[s] // 16, ctx[s - 1] // 16) for s, p in zip(range(1, B), pairs)]
        assert (total == 0) == (not any(m > 0 for m in most))


def test_prepare_shared_from_the_block_manager(libpa):
    bm = pa.BlockManager(64)
    prompt = list(range(100))
    for i in range(3):
        bm.allocate(i, prompt + [1000 + i] * (10 + i))
    tables = [bm.block_table(i) for i in range(3)]
    bt = np.full((3, 8), -1, np.int32)
    for i, t in enumerate(tables):
        bt[i, :len(t)] = t
    got = pa.prepare_shared(bt, np.array([bm.num_tokens(i) for i in range(3)], np.int32))
    assert got["group_starts"].tolist() == [0, 3] and got["shared_blocks"].tolist() == [6]


def test_prepare_shared_refusals(libpa):
    bt, ctx = np.zeros((2, 2), np.int32), np.array([3, 33], np.int32)
    with pytest.raises(pa.PAError):
        pa.prepare_shared(bt, ctx)  # 33 tokens in two blocks
    with pytest.raises(pa.PAError):
        pa.prepare_shared(bt, np.array([-1, 3], np.int32))
    with pytest.raises(ValueError):
        pa.prepare_shared(bt, np.zeros(3, np.int32))
    n = ctypes.c_int(7)
    out = np.full(4, 7, np.int32)
    p = out.ctypes.data_as(ctypes.c_void_p)
    call = libpa.pa_prepare_shared
    good = bt.ctypes.data_as(ctypes.c_void_p)
    assert call(1, None, 2, good, 16, p, p, ctypes.byref(n)) == pa.PA_ERR_INVALID
    assert call(1, good, 2, good, 0, p, p, ctypes.byref(n)) == pa.PA_ERR_INVALID
    assert call(-1, good, 2, good, 16, p, p, ctypes.byref(n)) == pa.PA_ERR_INVALID
    assert call(1, good, 2, good, 16, p, p, None) == pa.PA_ERR_INVALID
    assert (out == 7).all() and n.value == 7


# ---------------------------------------------------------------- the block manager


def test_block_manager_evicts(libpa):
    bm = pa.BlockManager(20)
    prompt = list(range(64))
    bm.allocate(1, prompt + [1] * 20)  # 6 blocks
    bm.allocate(2, prompt + [2] * 40)  # 7, the first 4 shared
    for s, n in ((1, 84), (2, 40)):
        bm.mark_computed(s, n)
    old = {s: bm.block_table(s).tolist() for s in (1, 2)}
    assert old[1][:4] == old[2][:4] and bm.num_free() == 20 - 9
    bm.evict_begin(2, 70)  # 5 blocks: 4 fresh ones for the shared, its own fifth
    new = bm.block_table(2).tolist()
    assert new[4] == old[2][4] and not set(new[:4]) & set(old[1] + old[2])
    assert bm.num_tokens(2) == 70 and bm.num_free() == 11 - 4  # what it leaves stays taken
    with pytest.raises(pa.PAError):
        bm.append(2, 7)
    with pytest.raises(pa.PAError):
        bm.evict_begin(2, 60)
    bm.evict_end(2)
    assert bm.num_free() == 7 + 2 and bm.block_table(1).tolist() == old[1]
    with pytest.raises(pa.PAError):
        bm.evict_end(2)
    # on with its own slots; what fills is not matched, what it had of its own neither
    slots = [bm.append(2, 5) for _ in range(26)]
    assert slots[0] == new[4] * 16 + 6 and bm.num_tokens(2) == 96
    free = bm.num_free()
    assert bm.allocate(3, prompt + [2] * 40) == 64  # the shared prefix alone: sequence 1's
    assert bm.block_table(3).tolist()[:4] == old[1][:4] and bm.num_free() == free - 3
    bm.free(3)
    # sequence 1 in place: its blocks are matched no longer
    bm.evict_begin(1, 33)
    assert bm.block_table(1).tolist() == old[1][:3]
    bm.evict_end(1)
    bm.free(1)
    assert bm.allocate(4, prompt) == 0
    for s in (2, 4):
        bm.free(s)
    assert bm.num_free() == 20


def test_block_manager_evict_refusals(libpa):
    bm = pa.BlockManager(8)
    with pytest.raises(pa.PAError):
        bm.evict_begin(1, 4)
    bm.allocate(1, list(range(100)))
    with pytest.raises(pa.PAError):
        bm.evict_begin(1, 40)  # its prompt is not computed
    bm.mark_computed(1, 100)
    with pytest.raises(pa.PAError):
        bm.evict_begin(1, 0)
    bm.evict_begin(1, 100)  # nothing goes
    bm.evict_end(1)
    assert bm.num_tokens(1) == 100 and len(bm.block_table(1)) == 7
    bm.allocate(2, list(range(112)))
    bm.mark_computed(2, bm.num_tokens(2) - 96)
    table = bm.block_table(2).tolist()
    with pytest.raises(pa.PAError) as e:  # six shared blocks, no free one
        bm.evict_begin(2, 90)
    assert e.value.code == pa.PA_ERR_WORKSPACE and bm.block_table(2).tolist() == table
    bm.free(1)  # (between begin and end: blocks left behind are given back too)
    bm.evict_begin(2, 20)
    bm.free(2)
    assert bm.num_free() == 8


# ---------------------------------------------------------------- sizes and refusals

BUF = ctypes.c_void_p(1 << 24)
APART = ctypes.c_void_p(1 << 30)
ODD = ctypes.c_void_p((1 << 30) + 8)
INT_MAX = 2**31 - 1


@pytest.fixture
def desc(libpa):
    d = pa.PaCache()
    assert libpa.pa_alloc_cache(ctypes.byref(d), 1, 64, 16, 2, 64, ctypes.c_void_p(1 << 20)) == 0
    return ctypes.byref(d)


def test_workspace_sizes(libpa):
    assert libpa.pa_decode_shared_workspace_bytes(4, 8, 2, 64) >= 2 * 4 * 8 * 68 * 4
    assert libpa.pa_decode_shared_workspace_bytes(0, 8, 2, 64) == 0
    one = libpa.pa_decode_weights_workspace_bytes(4, 8, 2, 64, 1)
    assert one > 16 * 8 * 4
    assert libpa.pa_decode_weights_workspace_bytes(4, 8, 2, 64, 11) == one + 10 * 16 * 8 * 4
    assert libpa.pa_decode_weights_workspace_bytes(4, 8, 2, 64, 0) == 0
    assert libpa.pa_decode_weights_workspace_bytes(4, 8, 2, 64, 2**60) == 0  # past 64 bits
    assert libpa.pa_decode_weights_workspace_bytes(INT_MAX, INT_MAX, 2, 64, 1) == 0
    assert libpa.pa_decode_shared_workspace_bytes(INT_MAX, INT_MAX, 2, 64) == 0
    assert libpa.pa_decode_shared_workspace_bytes(INT_MAX, 8, 2, INT_MAX) == 0
    assert libpa.pa_kv_evict_workspace_bytes(3, 2, 100) >= 3 * 2 * 100 * 8
    assert libpa.pa_kv_evict_workspace_bytes(3, 2, 0) == 0
    assert libpa.pa_kv_evict_workspace_bytes(INT_MAX, INT_MAX, INT_MAX) == 0


def test_rope_layout_refusals(libpa, desc):
    def call(q=BUF, q_out=BUF, k=APART, v=APART, pos=BUF, slots=BUF, T=4, H=4, Hk=2, d=64, layout=1,
             r=32, table=BUF, maxpos=8, cache=desc, layer=0):
        return libpa.pa_rope_kv_write_layout(q, q_out, k, v, pos, slots, T, H, Hk, d, layout, r,
                                             table, maxpos, cache, layer, None, None)

    assert call(T=0, q=None, k=None) == pa.PA_OK
    assert call(d=96) == pa.PA_ERR_UNSUPPORTED
    assert call(r=24) == pa.PA_ERR_UNSUPPORTED
    for bad in (dict(T=-1), dict(H=5), dict(Hk=4), dict(layer=1), dict(layer=-1), dict(maxpos=0),
                dict(cache=None), dict(q=None), dict(q_out=None), dict(k=None), dict(v=None),
                dict(pos=None), dict(slots=None), dict(table=None), dict(q=ODD), dict(q_out=ODD),
                dict(k=ODD), dict(v=ODD), dict(table=ODD), dict(layout=2), dict(layout=-1),
                dict(r=0), dict(r=80), dict(r=-16), dict(T=INT_MAX, H=2**30), dict(T=1, H=2**30),
                dict(q_out=ctypes.c_void_p((1 << 24) + 16)), dict(q_out=APART)):
        assert call(**bad) == pa.PA_ERR_INVALID, bad


def test_table_refusals(libpa):
    def call(table=BUF, n=8, r=64, theta=1e4, null=False, **sc):
        s = pa.PaRopeScaling(**sc)
        return libpa.pa_rope_table_init_scaled(table, n, r, theta,
                                               None if null else ctypes.byref(s), None)

    assert call(r=24) == pa.PA_ERR_UNSUPPORTED and call(r=144) == pa.PA_ERR_UNSUPPORTED
    yarn = dict(kind=3, factor=2.0, original_positions=64, low=1.0, high=4.0)
    for bad in (dict(table=None), dict(table=ODD), dict(n=0), dict(theta=1.0), dict(theta=math.inf),
                dict(theta=math.nan, null=True), dict(kind=5, factor=2.0), dict(kind=-1, factor=2.0),
                dict(kind=1, factor=0.5), dict(kind=1, factor=math.nan), dict(kind=2, factor=math.inf),
                dict(attention=-1.0), dict(attention=math.nan), {**yarn, "original_positions": 0},
                {**yarn, "low": 0.0}, {**yarn, "high": 1.0}, {**yarn, "high": math.inf},
                {**yarn, "kind": 4, "low": 5.0}):
        assert call(**bad) == pa.PA_ERR_INVALID, bad
    for bad in (dict(scaling="dynamic"), dict(device="cpu")):
        with pytest.raises(ValueError):
            pa.rope_table_scaled(8, 64, **bad)


def test_shared_refusals(libpa, desc):
    def call(q=BUF, cache=desc, layer=0, bt=BUF, maxb=4, ctx=BUF, B=2, starts=BUF, shared=BUF, n=1,
             H=4, Hk=2, d=64, scale=0.0, ws=BUF, wsb=1 << 30, out=BUF):
        return libpa.pa_decode_shared(q, cache, layer, bt, maxb, ctx, B, starts, shared, n, H, Hk, d,
                                      scale, ws, wsb, out, None, None)

    assert call(B=0, q=None, ws=None, n=0) == pa.PA_OK
    for bad in (dict(d=96), dict(H=32), dict(B=4097), dict(n=4097)):
        assert call(**bad) == pa.PA_ERR_UNSUPPORTED, bad
    need = libpa.pa_decode_shared_workspace_bytes(2, 4, 2, 64)
    assert call(wsb=need - 1) == pa.PA_ERR_WORKSPACE
    for bad in (dict(B=-1), dict(H=5), dict(Hk=4), dict(layer=1), dict(maxb=0), dict(n=0), dict(n=-1),
                dict(maxb=INT_MAX // 16 + 1), dict(scale=-1.0), dict(scale=math.nan),
                dict(cache=None), dict(q=None), dict(bt=None), dict(ctx=None), dict(ws=None),
                dict(out=None), dict(starts=None), dict(shared=None), dict(q=ODD), dict(out=ODD),
                dict(ws=ctypes.c_void_p((1 << 24) + 128))):
        assert call(**bad) == pa.PA_ERR_INVALID, bad


def test_weights_refusals(libpa, desc):
    def call(q=BUF, cache=desc, layer=0, bt=BUF, maxb=4, ctx=BUF, B=2, H=4, Hk=2, d=64, scale=0.0,
             w=BUF, w_out=BUF, stride=64, ws=BUF, wsb=1 << 30, out=BUF):
        return libpa.pa_decode_weights(q, cache, layer, bt, maxb, ctx, B, H, Hk, d, scale, w, w_out,
                                       stride, ws, wsb, out, None, None)

    assert call(B=0, q=None, ws=None) == pa.PA_OK
    for bad in (dict(d=96), dict(H=32), dict(B=4097)):
        assert call(**bad) == pa.PA_ERR_UNSUPPORTED, bad
    assert call(wsb=libpa.pa_decode_weights_workspace_bytes(2, 4, 2, 64, 1) - 1) == pa.PA_ERR_WORKSPACE
    for bad in (dict(B=-1), dict(H=5), dict(Hk=4), dict(layer=1), dict(maxb=0), dict(stride=0),
                dict(stride=-1), dict(stride=2**62), dict(scale=-1.0), dict(cache=None), dict(q=None),
                dict(bt=None), dict(ctx=None), dict(ws=None), dict(out=None), dict(w_out=None),
                dict(q=ODD), dict(out=ODD), dict(ws=ctypes.c_void_p((1 << 24) + 128)),
                dict(w_out=ctypes.c_void_p((1 << 24) + 64))):  # overlaps, and is not, w
        assert call(**bad) == pa.PA_ERR_INVALID, bad


def test_evict_refusals(libpa, desc):
    def call(cache=desc, layer=0, bt=BUF, maxb=4, ctx=BUF, B=2, Hk=2, d=64, w=BUF, w_out=BUF,
             stride=64, budget=8, sinks=1, recent=2, to=BUF, to_maxb=4, to_ctx=BUF, ws=BUF,
             wsb=1 << 30):
        return libpa.pa_kv_evict(cache, layer, bt, maxb, ctx, B, Hk, d, w, w_out, stride, budget,
                                 sinks, recent, to, to_maxb, to_ctx, ws, wsb, None, None)

    assert call(B=0, w=None, ws=None) == pa.PA_OK
    for bad in (dict(d=96), dict(B=4097)):
        assert call(**bad) == pa.PA_ERR_UNSUPPORTED, bad
    assert call(wsb=libpa.pa_kv_evict_workspace_bytes(2, 2, 8) - 1) == pa.PA_ERR_WORKSPACE
    for bad in (dict(B=-1), dict(Hk=4), dict(Hk=0), dict(layer=1), dict(layer=-1), dict(maxb=0),
                dict(maxb=INT_MAX // 16 + 1), dict(to_maxb=0), dict(to_maxb=INT_MAX // 16 + 1),
                dict(stride=0), dict(stride=2**62), dict(budget=0), dict(sinks=-1), dict(recent=-1),
                dict(sinks=7), dict(sinks=INT_MAX, recent=INT_MAX), dict(cache=None), dict(bt=None),
                dict(ctx=None), dict(w=None), dict(w_out=None), dict(to=None), dict(to_ctx=None),
                dict(ws=None), dict(ws=ctypes.c_void_p((1 << 24) + 128)),
                dict(w_out=ctypes.c_void_p((1 << 24) + 64))):
        assert call(**bad) == pa.PA_ERR_INVALID, bad


def test_binding_refuses_host_tensors(libpa):
    x = torch.zeros(2, 4, 64, dtype=torch.float16)
    i, u = torch.zeros(2, 2, dtype=torch.int32), torch.zeros(8, dtype=torch.uint8)
    one = torch.zeros(1, dtype=torch.int32)
    w = torch.zeros(2, 2, 32)
    with pytest.raises(TypeError):
        pa.rope_kv_write_layout(x, x, x, one, one, torch.zeros(4, 16, 2), None, "half")
    with pytest.raises(TypeError):
        pa.decode_shared(x, None, i, one, one, one, u, 2)
    with pytest.raises(TypeError):
        pa.decode_weights(x, None, i, one, w, u, 2)
    with pytest.raises(TypeError):
        pa.decode_weights(x, None, i, one, None, u, 2)
    with pytest.raises(TypeError):
        pa.kv_evict(None, i, one, w, 4, u)
    with pytest.raises(TypeError):
        pa.Cache(1, 4, 2, 64, tensor=torch.zeros(2, 1, 4, 16, 2, 64, dtype=torch.float16))
    with pytest.raises(ValueError):
        pa.decode_weights_workspace(2, 4, 2, 64, 0, device="cpu")
    with pytest.raises(ValueError):
        pa.kv_evict_workspace(2, 2, 0, device="cpu")
    with pytest.raises(ValueError):
        pa.decode_shared_workspace(0, 4, 2, 64, device="cpu")
