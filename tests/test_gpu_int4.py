"""GPU parity of the 4-bit KV cache against the oracle: RoPE + quantised append
and read-back bit for bit; decode and prefill attention against the attention
formula, in 64 bits, on the values that the codes stand for; then the calls
together, as a serving loop makes them."""

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


def normal16(rng, *shape, std=1.0):
    return (rng.standard_normal(shape) * std).astype(np.float16)


def tables(rng, lens, spare=2):
    """Block tables of a shuffled pool; returns (table, blocks in the pool)."""
    need = [max(1, -(-int(n) // 16)) for n in lens]
    order = rng.permutation(sum(need) + spare).astype(np.int32)
    bt = np.full((len(lens), max(need)), -1, np.int32)
    at = 0
    for s, n in enumerate(need):
        bt[s, :n] = order[at:at + n]
        at += n
    return bt, sum(need) + spare


def cache_of(tiles):
    L, NB, Hk, _, n = tiles.shape
    c = pa.CacheI4(L, NB, Hk, n // 10)
    c.tiles.copy_(torch.from_numpy(tiles))
    return c


# ------------------------------------------------------------------ write

@pytest.mark.parametrize("H,Hk,d,T", [(1, 1, 64, 1), (1, 1, 128, 5), (33, 33, 128, 2),
                                      (4, 2, 64, 1), (4, 2, 64, 10), (32, 4, 64, 33),
                                      (8, 1, 128, 7), (32, 8, 128, 40), (64, 8, 128, 100),
                                      (5, 5, 128, 3), (14, 2, 64, 1500), (64, 8, 128, 1300)])
@pytest.mark.parametrize("in_place", [False, True])
def test_write_bit_exact(H, Hk, d, T, in_place):
    rng = np.random.default_rng(H * 1000 + T)
    q, k, v = normal16(rng, T, H, d), normal16(rng, T, Hk, d, std=3), normal16(rng, T, Hk, d)
    v[0, 0, :32] = 0.25  # a constant group
    k[T // 2, Hk - 1, 5] = np.inf
    v[T - 1, 0, 40] = np.nan
    pos = rng.integers(0, 5000, T).astype(np.int32)
    NB = -(-T // 16) + 3
    slots = rng.permutation(NB * 16)[:T].astype(np.int32)
    if T > 4:
        slots[3] = -1  # a padding token
    want = rng.integers(0, 256, (2, NB, Hk, 2, 10 * d)).astype(np.uint8)
    cache = cache_of(want)
    kd, vd, qd = dev(k), dev(v), dev(q)
    status = pa.new_status()
    out = None if in_place else torch.zeros_like(qd)
    got = pa.rope_kv_write_i4(qd, kd, vd, dev(pos), dev(slots), pa.rope_table(5000, d), cache,
                              layer=1, q_out=out, status=status)
    assert got is (qd if in_place else out)
    assert int(status.item()) == 0
    q_rot = orc.rope_pinned(q, pos, d)
    with np.errstate(invalid="ignore"):
        k_rot = orc.rope_pinned(k, pos, d)
        orc.kv_write_i4(want, 1, k_rot, v, slots)
    assert np.array_equal(bits(got), bits(q_rot))
    if not in_place:
        assert np.array_equal(bits(qd), bits(q))
    assert np.array_equal(bits(kd), bits(k)) and np.array_equal(bits(vd), bits(v))
    assert np.array_equal(cache.tiles.cpu().numpy(), want)


@pytest.mark.parametrize("std", [2e-7, 1e-5, 1e-2, 300.0, 2e4])
def test_write_bit_exact_at_every_magnitude(std):
    rng = np.random.default_rng(11)
    T, Hk, d = 64, 4, 128
    v = np.clip(rng.standard_normal((T, Hk, d)) * std, -65504, 65504).astype(np.float16)
    with np.errstate(over="ignore"):  # (an infinity now and then)
        v[:8] += np.float16(min(100 * std, 3e4))  # an offset far from zero
    k, q = normal16(rng, T, Hk, d), normal16(rng, T, Hk, d)
    cache = pa.CacheI4(1, 4, Hk, d)
    cache.buffer.zero_()
    slots, pos = np.arange(T, dtype=np.int32), np.zeros(T, np.int32)
    pa.rope_kv_write_i4(dev(q), dev(k), dev(v), dev(pos), dev(slots), pa.rope_table(1, d), cache)
    want = orc.new_cache_i4(1, 4, Hk, d)
    orc.kv_write_i4(want, 0, k, v, slots)
    assert np.array_equal(cache.tiles.cpu().numpy(), want)


@pytest.mark.parametrize("T", [6, 2000])
def test_write_reports_bad_positions_and_slots(T):
    rng = np.random.default_rng(12)
    H, Hk, d, NB = 8, 2, 128, T // 16 + 2
    q, k, v = normal16(rng, T, H, d), normal16(rng, T, Hk, d), normal16(rng, T, Hk, d)
    pos = rng.integers(0, 50, T).astype(np.int32)
    slots = rng.permutation(NB * 16)[:T].astype(np.int32)
    good_slots = slots.copy()
    pos[1], pos[2] = -1, 50
    slots[4] = NB * 16
    good_slots[[1, 2, 4]] = -1
    tiles = rng.integers(0, 256, (1, NB, Hk, 2, 10 * d)).astype(np.uint8)
    cache, status, out = cache_of(tiles), pa.new_status(), torch.full((T, H, d), 7.0).half().cuda()
    pa.rope_kv_write_i4(dev(q), dev(k), dev(v), dev(pos), dev(slots), pa.rope_table(50, d), cache,
                        q_out=out, status=status)
    assert int(status.item()) == pa.PA_DEV_BAD_POSITION | pa.PA_DEV_BAD_SLOT
    safe = np.clip(pos, 0, 49)
    want_q = orc.rope_pinned(q, safe, d)
    want_q[[1, 2]] = 7
    assert np.array_equal(bits(out), bits(want_q))
    orc.kv_write_i4(tiles, 0, orc.rope_pinned(k, safe, d), v, good_slots)
    assert np.array_equal(cache.tiles.cpu().numpy(), tiles)


# ------------------------------------------------------------------ read back

@pytest.mark.parametrize("Hk,d", [(2, 64), (4, 64), (1, 128), (8, 128), (5, 128)])
@pytest.mark.parametrize("first", [False, True])
def test_read_bit_exact(Hk, d, first):
    rng = np.random.default_rng(20 + Hk + d)
    lens = np.array([1, 0, 15, 16, 17, 200, 33, 0, 5], np.int32)
    f = rng.integers(0, 40, len(lens)).astype(np.int32) if first else np.zeros(len(lens), np.int32)
    bt, NB = tables(rng, lens + f)
    tiles = orc.pack_cache_i4(normal16(rng, 2, 2, NB, 16, Hk, d, std=2))
    vals = orc.read_rows_i4(orc.dequantize_cache_i4(tiles))
    cache = cache_of(tiles)
    gap = 3  # rows between the sequences that belong to none
    rows = (np.cumsum(lens + gap) - lens).astype(np.int32)
    total = int(rows[-1] + lens[-1]) + 4
    want = np.full((2, total, Hk, d), 9, np.float16)
    for s, n in enumerate(lens):
        for kv in (0, 1):
            flat = vals[kv, 1][bt[s][bt[s] >= 0]].reshape(-1, Hk, d)
            want[kv, rows[s]:rows[s] + n] = flat[f[s]:f[s] + n]
    for keep_k, keep_v in ((True, True), (True, False), (False, True)):
        ko, vo = (torch.full((total, Hk, d), 9.0).half().cuda() if x else None
                  for x in (keep_k, keep_v))
        status = pa.new_status()
        got = pa.kv_read_i4(cache, dev(bt), dev(lens), dev(rows), ko, vo,
                            first_tokens=dev(f) if first else None, layer=1, status=status)
        assert got[0] is ko and got[1] is vo and int(status.item()) == 0
        if keep_k:
            assert np.array_equal(bits(ko), bits(want[0]))
        if keep_v:
            assert np.array_equal(bits(vo), bits(want[1]))


def test_read_saturates_and_keeps_nan():
    x = np.zeros((2, 1, 1, 16, 1, 64), np.float16)
    x[:, 0, 0, 0, 0, :2] = [-65504, 65504]
    x[:, 0, 0, 1, 0, 40] = np.nan
    tiles = orc.pack_cache_i4(x)
    cache = cache_of(tiles)
    k, v = (torch.empty(16, 1, 64, dtype=torch.float16, device="cuda") for _ in range(2))
    one = dev(np.array([16], np.int32))
    pa.kv_read_i4(cache, dev(np.zeros((1, 1), np.int32)), one, one * 0, k, v)
    for t in (k.cpu(), v.cpu()):
        assert t[0, 0, 1] == 65504 and t[0, 0, 0] == -65504
        assert torch.isnan(t[1, 0, 32:]).all() and torch.isfinite(t[1, 0, :32]).all()


def test_read_reports_bad_lengths_rows_and_blocks():
    rng = np.random.default_rng(22)
    Hk, d = 2, 64
    lens = np.array([20, -1, 40, 33, 17, 18, 19], np.int32)
    bt, NB = tables(rng, np.full(7, 48))
    tiles = orc.pack_cache_i4(normal16(rng, 2, 1, NB, 16, Hk, d))
    vals = orc.read_rows_i4(orc.dequantize_cache_i4(tiles))[0, 0]
    first = np.array([0, 0, 10, 0, 0, -3, 0], np.int32)  # 2: past the table; 5: negative
    rows = np.array([0, 20, 20, 100, 40, 60, 200 - 18], np.int32)  # 6: one row too far
    bt[0, 1] = NB
    bt[4, 0] = -5
    out = torch.full((200, Hk, d), 9.0).half().cuda()
    status = pa.new_status()
    pa.kv_read_i4(cache_of(tiles), dev(bt), dev(lens), dev(rows), out, None,
                  first_tokens=dev(first), status=status)
    assert int(status.item()) == pa.PA_DEV_BAD_LENGTH | pa.PA_DEV_BAD_BLOCK
    want = np.full((200, Hk, d), 9, np.float16)
    want[0:16] = vals[bt[0, 0]]
    want[56] = vals[bt[4, 1]][0]
    want[100:133] = vals[bt[3]].reshape(-1, Hk, d)[:33]
    assert np.array_equal(bits(out), bits(want))


def test_read_padded_batch():
    """Sequences of length 0 read nothing and report nothing, whatever their
    other entries hold."""
    rng = np.random.default_rng(24)
    bt, NB = tables(rng, [20])
    tiles = orc.pack_cache_i4(normal16(rng, 2, 1, NB, 16, 2, 64))
    bt = np.concatenate([bt, np.full((3, 2), 1 << 30, np.int32)])
    out, status = torch.full((25, 2, 64), 9.0).half().cuda(), pa.new_status()
    i32 = lambda *x: dev(np.array(x, np.int32))  # noqa: E731
    pa.kv_read_i4(cache_of(tiles), dev(bt), i32(20, 0, 0, 0), i32(2, -7, 2**31 - 1, 0), out, None,
                  first_tokens=i32(0, -1, 2**31 - 1, 5), status=status)
    assert int(status.item()) == 0
    want = np.full((25, 2, 64), 9, np.float16)
    vals = orc.read_rows_i4(orc.dequantize_cache_i4(tiles))[0, 0]
    want[2:22] = vals[bt[0]].reshape(-1, 2, 64)[:20]
    assert np.array_equal(bits(out), bits(want))
    # nothing at all to read
    pa.kv_read_i4(cache_of(tiles), dev(bt), i32(0, 0, 0, 0), i32(0, 0, 0, 0), out, out, status=status)
    assert int(status.item()) == 0 and np.array_equal(bits(out), bits(want))


def test_read_many_sequences():
    rng = np.random.default_rng(23)
    B, Hk, d = 4096, 1, 64
    lens = rng.integers(0, 20, B).astype(np.int32)
    bt, NB = tables(rng, lens)
    tiles = orc.pack_cache_i4(normal16(rng, 2, 1, NB, 16, Hk, d))
    vals = orc.read_rows_i4(orc.dequantize_cache_i4(tiles))[1, 0]
    rows = (np.cumsum(lens) - lens).astype(np.int32)
    out = torch.empty(int(lens.sum()), Hk, d, dtype=torch.float16, device="cuda")
    pa.kv_read_i4(cache_of(tiles), dev(bt), dev(lens), dev(rows), None, out)
    want = np.concatenate([vals[bt[s]].reshape(-1, Hk, d)[:n] for s, n in enumerate(lens)])
    assert np.array_equal(bits(out), bits(want))


# ------------------------------------------------------------------ decode

def decode_want(q, tiles, layer, bt, ctx, Hk, scale=None):
    """The decode formula in 64 bits on m + s c, and for every output how far
    the kernel may be from it:
      - the output's own fp16 rounding, half a step;
      - each probability enters P V as an fp16 product with its group's step and
        is multiplied by c - 8, |c - 8| <= 8, and as an fp16 factor of the
        group's fp16 centre m + 8 s: 2^-11 p (8 s + 2 |m + 8 s|), and below
        fp16's normal range 2^-25 instead of the relative error (p is at least
        1/4 of its true size relative to the largest): 2^-25 (8 + |m + 8 s|) 4;
      - fp32 scores: 300 roundings of 2^-24 of the sum of the terms' sizes, so
        every probability is off by that, relatively, and 2^-21 for the
        exponential and the sums."""
    B, H, d = q.shape
    g = H // Hk
    scale = 1 / math.sqrt(d) if scale is None else scale
    vals = orc.dequantize_cache_i4(tiles[layer:layer + 1])[:, 0]
    _, _, step, least = orc.kv_i4_places(d, True)
    par = np.ascontiguousarray(tiles[layer, :, :, 1, 8 * d:]).view(np.float16).astype(np.float64)
    st = np.swapaxes(np.repeat(par[..., step], 32, -1), 1, 2)   # [NB, 16, Hk, d]
    mid = np.swapaxes(np.repeat(par[..., least], 32, -1), 1, 2) + 8 * st
    out, tol = np.zeros((B, H, d)), np.zeros((B, H, d))
    for s in range(B):
        n = int(ctx[s])
        rows = bt[s, :-(-n // 16)]
        K, V, S, Z = (x[rows].reshape(-1, Hk, d)[:n] for x in (vals[0], vals[1], st, mid))
        for h in range(H):
            qv = q[s, h].astype(np.float64)
            x = K[:, h // g] @ qv * scale
            big = np.abs(K[:, h // g]) @ np.abs(qv) * scale
            w = np.exp(x - x.max())
            v, sv, z = V[:, h // g], S[:, h // g], np.abs(Z[:, h // g])
            rel = (w * (big * 300 * 2.0 ** -24 * 4 + 2.0 ** -21)) @ np.abs(v)
            rnd = 2.0 ** -11 * (w @ (8 * sv + 2 * z)) + 2.0 ** -23 * (8 + z).sum(0)
            out[s, h] = w @ v / w.sum()
            tol[s, h] = (rel + rnd) / w.sum() + 2.0 ** -20 * np.abs(out[s, h])
    with np.errstate(invalid="ignore"):
        return out, tol + half_ulp16(out)


def decode_case(seed, H, Hk, d, ctxs, std_k=1.0, std_v=1.0, layers=1, offset=0.0):
    rng = np.random.default_rng(seed)
    ctx = np.array(ctxs, np.int32)
    bt, NB = tables(rng, ctx)
    pool = rng.standard_normal((2, layers, NB, 16, Hk, d))
    pool[0] *= std_k
    pool[1] = pool[1] * std_v + offset
    with np.errstate(over="ignore"):  # (an infinity now and then at the largest)
        pool = pool.astype(np.float16)
    return normal16(rng, len(ctxs), H, d), orc.pack_cache_i4(pool), bt, ctx


def run_decode(q, tiles, bt, ctx, Hk, layer=0, scale=0.0, ws=None, **kw):
    B, H, d = q.shape
    cache = tiles if isinstance(tiles, pa.CacheI4) else cache_of(tiles)
    ws = pa.decode_i4_workspace(B, H, Hk, d) if ws is None else ws
    status = pa.new_status()
    out = pa.decode_i4(dev(q), cache, dev(bt), dev(ctx), ws, Hk, layer=layer, scale=scale,
                       status=status, **kw)
    assert int(status.item()) == 0
    return out


def check_decode(q, tiles, bt, ctx, Hk, layer=0, scale=None, **kw):
    out = run_decode(q, tiles, bt, ctx, Hk, layer, scale or 0.0, **kw)
    want, tol = decode_want(q, tiles, layer, bt, ctx, Hk, scale)
    got = out.cpu().numpy().astype(np.float64)
    ok = ~np.isnan(want)  # (a group with an infinity or a NaN reads as NaN)
    assert np.array_equal(np.isfinite(got), ok)
    worst = np.max(np.abs(got - want)[ok] / tol[ok])
    assert worst <= 1, worst
    return out


@pytest.mark.parametrize("H,Hk,d", [(8, 8, 128), (32, 8, 128), (64, 8, 128), (16, 8, 64),
                                    (8, 1, 64), (8, 1, 128), (14, 2, 64), (6, 2, 128),
                                    (35, 7, 128), (1, 1, 128), (1, 1, 64)])
def test_decode_edge_lengths(H, Hk, d):
    ctxs = [1, 2, 7, 8, 9, 15, 16, 17, 31, 32, 33, 47, 48, 49, 255, 256, 257, 1000, 4100]
    check_decode(*decode_case(H + Hk + d, H, Hk, d, ctxs), Hk)


@pytest.mark.parametrize("ctxs", [[1], [3], [16], [17], [33], [100], [5000], [20000], [1] * 700,
                                  [40] * 300, [20000, 1, 1], [1, 20000], [3000, 17, 16, 2500]])
@pytest.mark.parametrize("H,Hk,d", [(16, 2, 128), (4, 4, 64)])
def test_decode_batches(ctxs, H, Hk, d):
    check_decode(*decode_case(len(ctxs) + ctxs[0], H, Hk, d, ctxs), Hk)


@pytest.mark.parametrize("std_k,std_v,offset", [(1e-3, 1.0, 0), (8.0, 1.0, 0), (60.0, 1.0, 0),
                                                (1.0, 1e-3, 0), (1.0, 1e-5, 0), (1.0, 2e4, 0), (1.0, 9e3, 0),
                                                (1.0, 1.0, 50.0), (0.0, 0.0, 1.0)])
def test_decode_magnitudes(std_k, std_v, offset):
    q, tiles, bt, ctx = decode_case(31, 16, 4, 128, [5, 300, 1200], std_k, std_v, offset=offset)
    check_decode(q, tiles, bt, ctx, 4)
    for factor in (2.0 ** -10, 2.0 ** -22, 100.0):  # and of the query
        check_decode((q.astype(np.float32) * factor).astype(np.float16), tiles, bt, ctx, 4)


def test_decode_layer_and_scale():
    q, tiles, bt, ctx = decode_case(32, 8, 2, 128, [70, 900], layers=3)
    for layer in (0, 2):
        check_decode(q, tiles, bt, ctx, 2, layer=layer)
    check_decode(q, tiles, bt, ctx, 2, layer=1, scale=0.31)


@pytest.mark.parametrize("d", [64, 128])
def test_decode_zero_query_averages(d):
    q, tiles, bt, ctx = decode_case(33, 8, 2, d, [1, 50, 333])
    q[:] = 0
    check_decode(q, tiles, bt, ctx, 2)


def test_decode_a_late_large_score_and_step():
    """The running maximum, and the largest step, are met late, in the last
    token: everything before it is rescaled."""
    rng = np.random.default_rng(34)
    n = 600
    pool = rng.standard_normal((2, 1, 40, 16, 1, 128)).astype(np.float16)
    bt = np.arange(40, dtype=np.int32)[None]
    q = normal16(rng, 1, 4, 128)
    last = pool[:, 0, (n - 1) // 16, (n - 1) % 16, 0]
    last[0] = q[0, 0]  # score |q|^2 / sqrt(d), about 11
    last[1] = normal16(rng, 128, std=5000)
    check_decode(q, orc.pack_cache_i4(pool), bt, np.array([n], np.int32), 1)


@pytest.mark.parametrize("d", [64, 128])
def test_decode_ignores_what_lies_past_the_context(d):
    q, tiles, bt, ctx = decode_case(35, 16, 4, d, [20, 300, 4, 47, 33])
    want = run_decode(q, tiles, bt, ctx, 4)
    for fill in (0xFF, 0x7C):  # NaN and huge parameters, every code 15
        bad = tiles.copy()
        for kv in (0, 1):
            byte, shift, step, least = orc.kv_i4_places(d, kv == 1)
            for s, n in enumerate(ctx):
                for j in range(int(n) % 16 or 16, 16):
                    t = bad[0, bt[s, (n - 1) // 16], :, kv]
                    t[:, byte[j][shift[j] == 0]] |= 0x0F
                    t[:, byte[j][shift[j] == 4]] |= 0xF0
                    for p in (*step[j], *least[j]):
                        t[:, 8 * d + 2 * p:8 * d + 2 * p + 2] = fill
        # blocks that no table names
        unused = np.setdiff1d(np.arange(tiles.shape[1]), bt)
        bad[:, unused] = 0xFF
        assert np.array_equal(bits(run_decode(q, bad, bt, ctx, 4)), bits(want))


def test_decode_nan_stays_in_its_group():
    q, tiles, bt, ctx = decode_case(36, 8, 2, 128, [100, 100])
    _, _, step, least = orc.kv_i4_places(128, True)
    v = tiles[0, bt[0, 2], 1, 1, 8 * 128:].view(np.float16)
    v[step[5, 2]], v[least[5, 2]] = 0, np.nan
    got = run_decode(q, tiles, bt, ctx, 2).float().cpu().numpy()
    nan = np.zeros((2, 8, 128), bool)
    nan[0, 4:, 64:96] = True
    assert np.array_equal(np.isnan(got), nan)


def test_decode_reports_bad_blocks_and_lengths():
    q, tiles, bt, ctx = decode_case(37, 16, 2, 128, [40, 64, 80, 90, 30])
    for value, bit in ((tiles.shape[1], pa.PA_DEV_BAD_BLOCK), (-1, pa.PA_DEV_BAD_BLOCK)):
        b = bt.copy()
        b[1, 2] = value
        status = pa.new_status()
        ws = pa.decode_i4_workspace(5, 16, 2, 128)
        out = pa.decode_i4(dev(q), cache_of(tiles), dev(b), dev(ctx), ws, 2, status=status)
        assert int(status.item()) == bit
        want, tol = decode_want(q, tiles, 0, bt, ctx, 2)
        keep = [0, 2, 3, 4]
        assert (np.abs(out.cpu().numpy() - want) <= tol)[keep].all()
        assert torch.isfinite(out).all()
    for bad in (0, -3, bt.shape[1] * 16 + 1):  # its rows stay as they were
        c = ctx.copy()
        c[2] = bad
        status, out = pa.new_status(), torch.full((5, 16, 128), 3.0).half().cuda()
        pa.decode_i4(dev(q), cache_of(tiles), dev(bt), dev(c), ws, 2, out=out, status=status)
        assert int(status.item()) == pa.PA_DEV_BAD_LENGTH
        got = out.cpu().numpy()
        assert (got[2] == 3).all()
        assert (np.abs(got - want) <= tol)[[0, 1, 3, 4]].all()


def test_decode_repeats_bit_for_bit_in_one_workspace():
    """Many calls of changing shapes through one workspace, left ready each time."""
    ws = pa.decode_i4_workspace(64, 64, 8, 128)
    cases = [decode_case(40 + i, H, Hk, 128, ctxs) for i, (H, Hk, ctxs) in enumerate(
        [(64, 8, [3000] * 3), (8, 8, [1, 700, 33]), (16, 4, [9000]), (32, 4, list(range(1, 60)))])]
    want = [check_decode(q, t, bt, ctx, t.shape[2], ws=ws) for q, t, bt, ctx in cases]
    caches = [cache_of(t) for _, t, _, _ in cases]
    for _ in range(10):
        for (q, t, bt, ctx), c, w in zip(cases, caches, want):
            assert torch.equal(run_decode(q, c, bt, ctx, t.shape[2], ws=ws), w)


def test_decode_on_another_stream():
    q, tiles, bt, ctx = decode_case(50, 32, 4, 128, [500, 1500, 17])
    want = run_decode(q, tiles, bt, ctx, 4)
    side = torch.cuda.Stream()
    ws, cache = pa.decode_i4_workspace(3, 32, 4, 128), cache_of(tiles)
    a = [dev(x) for x in (q, bt, ctx)]
    torch.cuda.synchronize()
    out = torch.zeros_like(want)
    torch.cuda.synchronize()
    for given in (True, False):
        out.zero_()
        torch.cuda.synchronize()
        with torch.cuda.stream(torch.cuda.current_stream() if given else side):
            pa.decode_i4(a[0], cache, a[1], a[2], ws, 4, out=out, stream=side if given else None)
        side.synchronize()
        assert torch.equal(out, want)


def test_decode_right_behind_new_lengths():
    """Lengths written by kernels and copies directly before the call."""
    H, Hk, d = 16, 2, 128
    q, tiles, bt, ctx = decode_case(42, H, Hk, d, [900, 17, 3000, 333] * 4)
    cache, qd, btd = cache_of(tiles), dev(q), dev(bt)
    lens = [dev(c) for c in (ctx, np.maximum(ctx // 3, 1).astype(np.int32), np.ones_like(ctx))]
    ws = pa.decode_i4_workspace(len(ctx), H, Hk, d)
    want = [run_decode(q, cache, bt, x.cpu().numpy(), Hk) for x in lens]
    live, got = lens[0].clone(), []
    for i in range(60):
        if i % 2:
            live.copy_(lens[i % 3])
        else:
            torch.add(lens[i % 3], 0, out=live)
        got.append(pa.decode_i4(qd, cache, btd, live, ws, Hk))
    for i, x in enumerate(got):
        assert torch.equal(x, want[i % 3])


def test_decode_two_streams_at_once():
    """Two calls in flight together, each with its own workspace."""
    cases = [decode_case(51 + i, 64, 8, 128, [2000 + 500 * i] * 4) for i in range(2)]
    want = [run_decode(q, t, bt, ctx, 8) for q, t, bt, ctx in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    ready = [([dev(x) for x in (q, bt, ctx)], cache_of(t), pa.decode_i4_workspace(4, 64, 8, 128),
              torch.zeros_like(w)) for (q, t, bt, ctx), w in zip(cases, want)]
    torch.cuda.synchronize()
    for _ in range(20):
        for ((q, bt, ctx), c, ws, out), st in zip(ready, streams):
            pa.decode_i4(q, c, bt, ctx, ws, 8, out=out, stream=st)
    torch.cuda.synchronize()
    for (_, _, _, out), w in zip(ready, want):
        assert torch.equal(out, w)


def test_decode_4096_sequences():
    rng = np.random.default_rng(57)
    ctxs = rng.integers(1, 40, 4096)
    ctxs[:5] = [1, 16, 17, 700, 1]
    check_decode(*decode_case(57, 2, 1, 64, ctxs), 1)


@pytest.mark.parametrize("H,Hk,d", [(8, 8, 64), (16, 4, 128)])
def test_decode_long_flat_sums(H, Hk, d):
    """Long histories that every key has a share in: the sums behind an output are
    hundreds of times the output.  Relative L2 error over all outputs: the fp16
    roundings of p s, of the centre's operands and of the output, each of an rms
    of at most 2^-10 / sqrt(12) of its value (a value rounded to fp16 is off by
    an even distribution over one step, at most 2^-10 of it)."""
    B, n = 64 // Hk * 2, 32768
    rng = torch.Generator(device="cuda").manual_seed(59)
    NB = B * n // 16
    cache = pa.CacheI4(1, NB, Hk, d)
    slots = torch.arange(n, dtype=torch.int32, device="cuda")
    table, pos = pa.rope_table(1, d), torch.zeros(n, dtype=torch.int32, device="cuda")
    for s in range(B):
        k, v = (torch.randn(n, Hk, d, device="cuda", generator=rng).half() for _ in range(2))
        q = torch.zeros(n, Hk, d, dtype=torch.float16, device="cuda")
        pa.rope_kv_write_i4(q, k, v, pos, slots + s * n, table, cache)
    q = torch.randn(B, H, d, device="cuda", generator=rng).half()
    bt = torch.arange(NB, dtype=torch.int32, device="cuda").view(B, -1)
    ctx = torch.full((B,), n - 5, dtype=torch.int32, device="cuda")
    out = pa.decode_i4(q, cache, bt, ctx, pa.decode_i4_workspace(B, H, Hk, d), Hk).double()
    err = norm = 0.0
    for s in range(0, B, 3):
        tiles = cache.tiles[0, bt[s].long()]  # [blocks, Hk, 2, 10 d]
        val = []
        for kv in (0, 1):
            byte, shift, step, least = (torch.from_numpy(x).cuda() for x in orc.kv_i4_places(d, kv == 1))
            x = tiles[:, :, kv]
            p = x[..., 8 * d:].contiguous().view(torch.float16).double()
            c = (x[..., byte].int() >> shift) & 15
            y = p[..., least].repeat_interleave(32, -1) + p[..., step].repeat_interleave(32, -1) * c
            val.append(y.transpose(0, 1).flatten(1, 2)[:, :n - 5])  # [Hk, n - 5, d]
        w = q[s].double().view(Hk, H // Hk, d) @ val[0].transpose(-1, -2) / math.sqrt(d)
        want = (torch.softmax(w, -1) @ val[1]).view(H, d)
        err += float((out[s] - want).square().sum())
        norm += float(want.square().sum())
    assert math.sqrt(err / norm) <= math.sqrt(3) * 2.0 ** -10 / math.sqrt(12), math.sqrt(err / norm)


@pytest.mark.parametrize("H,Hk,d", [(32, 8, 128), (8, 2, 64)])
def test_pool_past_32_bits(H, Hk, d):
    """Blocks whose bytes lie past 2^32 (and 2^33) of the pool, in a layer past the
    first: append, read back, prefill and decode."""
    rng = np.random.default_rng(58)
    NB = 9_000_000_000 // (2 * Hk * 20 * d)
    cache = pa.CacheI4(2, NB, Hk, d)
    assert cache.buffer.numel() > 2**33
    bt = np.array([[NB - 1, 3, NB - 2, NB // 2], [NB - 5, NB - 4, 0, NB - 3]], np.int32)
    n = np.array([60, 33], np.int32)
    md = pa.prepare_prefill([0, 0], n, bt)
    q, k, v = (normal16(rng, 93, h, d) for h in (H, Hk, Hk))
    qd, status = dev(q), pa.new_status()
    pa.rope_kv_write_i4(qd, dev(k), dev(v), dev(md["positions"]), dev(md["slot_mapping"]),
                        pa.rope_table(64, d), cache, layer=1, status=status)
    # the same rows in a small pool, on the host
    small = np.where(bt >= 0, np.arange(8).reshape(2, 4), -1).astype(np.int32)
    md2 = pa.prepare_prefill([0, 0], n, small)
    tiles = orc.new_cache_i4(1, 8, Hk, d)
    q_rot = orc.rope_pinned(q, md["positions"], d)
    orc.kv_write_i4(tiles, 0, orc.rope_pinned(k, md["positions"], d), v, md2["slot_mapping"])
    assert np.array_equal(cache.tiles[1][torch.from_numpy(bt.reshape(-1)).cuda().long()].cpu().numpy()
                          [:4].reshape(4, -1)[:3], tiles[0, :3].reshape(3, -1))
    ko, vo = (torch.empty(93, Hk, d, dtype=torch.float16, device="cuda") for _ in range(2))
    pa.kv_read_i4(cache, dev(bt), dev(n), dev(np.array([0, 60], np.int32)), ko, vo, layer=1,
                  status=status)
    vals = orc.read_rows_i4(orc.dequantize_cache_i4(tiles))[:, 0].reshape(2, 2, 64, Hk, d)
    for kv, got in enumerate((ko, vo)):
        want = np.concatenate([vals[kv, s][:m] for s, m in enumerate(n)])
        assert np.array_equal(bits(got), bits(want))
    ws = pa.prefill_i4_workspace(8, 2, 4, Hk, d)
    out = pa.prefill_varlen_i4(qd, cache, dev(md["cu_seqlens_q"]), dev(md["cu_seqlens_k"]), dev(bt),
                               60, Hk, ws, layer=1, status=status)
    assert_attention_close(out, prefill_want(q_rot, tiles, small,
                                             (md["cu_seqlens_q"], md["cu_seqlens_k"]), Hk))
    last = q_rot[[59, 92]]
    got = pa.decode_i4(dev(last), cache, dev(bt), dev(n), pa.decode_i4_workspace(2, H, Hk, d), Hk,
                       layer=1, status=status)
    want, tol = decode_want(last, tiles, 0, small, n, Hk)
    assert (np.abs(got.cpu().numpy() - want) <= tol).all()
    assert int(status.item()) == 0


# ------------------------------------------------------------------ prefill

def prefill_case(seed, H, Hk, d, past, new, layers=1):
    rng = np.random.default_rng(seed)
    past, new = np.array(past), np.array(new)
    bt, NB = tables(rng, past + new)
    tiles = orc.pack_cache_i4(normal16(rng, 2, layers, NB, 16, Hk, d))
    cu = [np.concatenate([[0], np.cumsum(x)]).astype(np.int32) for x in (new, past + new)]
    return normal16(rng, int(new.sum()), H, d), tiles, bt, cu


def prefill_want(q, tiles, bt, cu, Hk, layer=0, scale=None, seqs=None):
    vals = orc.read_rows_i4(orc.dequantize_cache_i4(tiles)).astype(np.float64)
    return orc.attention_prefill(q, vals, layer, cu[0], cu[1], bt, q.shape[1], Hk, scale=scale,
                                 seqs=seqs)


def run_prefill(q, tiles, bt, cu, Hk, layer=0, scale=0.0, blocks=None, max_new=None):
    B = len(cu[0]) - 1
    lens = np.diff(cu[1])
    blocks = int((-(-lens // 16)).sum()) if blocks is None else blocks
    ws = pa.prefill_i4_workspace(max(blocks, 1), B, bt.shape[1], Hk, q.shape[2])
    ws.fill_(0xFF)  # NaN everywhere: undefined contents must not show
    status = pa.new_status()
    out = pa.prefill_varlen_i4(dev(q), cache_of(tiles), dev(cu[0]), dev(cu[1]), dev(bt),
                               int(np.diff(cu[0]).max()) if max_new is None else max_new, Hk, ws,
                               layer=layer, scale=scale, status=status)
    return out, int(status.item())


@pytest.mark.parametrize("H,Hk,d", [(4, 2, 64), (8, 8, 128), (32, 4, 128), (14, 2, 64)])
def test_prefill_against_the_formula(H, Hk, d):
    past, new = [0, 5, 16, 0, 300, 31, 2], [3, 130, 1, 0, 257, 16, 40]
    q, tiles, bt, cu = prefill_case(60 + H, H, Hk, d, past, new, layers=2)
    for layer, scale in ((0, None), (1, 0.2)):
        out, status = run_prefill(q, tiles, bt, cu, Hk, layer, scale or 0.0)
        assert status == 0
        assert_attention_close(out, prefill_want(q, tiles, bt, cu, Hk, layer, scale))


def test_prefill_workspace_too_small_is_reported():
    q, tiles, bt, cu = prefill_case(70, 8, 2, 128, [0, 100, 0], [40, 30, 20])
    out, status = run_prefill(q, tiles, bt, cu, 2, blocks=4)  # 3 + 9 + 2 are needed
    assert status & pa.PA_DEV_WORKSPACE
    want = prefill_want(q, tiles, bt, cu, 2)
    assert_attention_close(out, want, rows=slice(0, 40))  # the sequence that fits


def test_prefill_sequences_without_new_tokens():
    """A batch in which some sequences have nothing new, or nothing at all."""
    q, tiles, bt, cu = prefill_case(73, 8, 2, 128, [50, 0, 7, 0], [0, 33, 1, 0])
    out, status = run_prefill(q, tiles, bt, cu, 2)
    assert status == 0
    assert_attention_close(out, prefill_want(q, tiles, bt, cu, 2))


def test_prefill_reports_bad_lengths():
    q, tiles, bt, cu = prefill_case(74, 8, 2, 128, [0, 10, 0], [40, 30, 20])
    good = prefill_want(q, tiles, bt, cu, 2)
    for k_of_1 in (20, bt.shape[1] * 16 + 1):  # fewer keys than queries; past the table
        k = np.diff(cu[1])
        k[1] = k_of_1
        bad = np.concatenate([[0], np.cumsum(k)]).astype(np.int32)
        out, status = run_prefill(q, tiles, bt, (cu[0], bad), 2)
        assert status == pa.PA_DEV_BAD_LENGTH
        assert_attention_close(out, good, rows=np.r_[0:40, 70:90])


def test_prefill_bad_block_is_reported():
    q, tiles, bt, cu = prefill_case(71, 8, 2, 64, [0, 0], [40, 30])
    bt[1, 1] = tiles.shape[1] + 3
    out, status = run_prefill(q, tiles, bt, cu, 2)
    assert status & pa.PA_DEV_BAD_BLOCK
    assert_attention_close(out, prefill_want(q, tiles, bt, cu, 2, seqs=[0]), rows=slice(0, 40))


def test_prefill_equals_read_back_and_fp16_prefill():
    """The same call made by hand: the rows read back into an fp16 pool, then
    pa_prefill_varlen over it, give the same bits."""
    q, tiles, bt, cu = prefill_case(72, 32, 8, 128, [200, 0, 33], [150, 300, 1])
    out, status = run_prefill(q, tiles, bt, cu, 8)
    assert status == 0
    lens = np.diff(cu[1]).astype(np.int32)
    need = -(-lens // 16)
    start = (np.cumsum(need) - need).astype(np.int32)
    pool = pa.Cache(1, int(need.sum()), 8, 128)
    rows = pool.tensor.view(2, -1, 8, 128)
    pa.kv_read_i4(cache_of(tiles), dev(bt), dev(lens), dev(16 * start), rows[0], rows[1])
    table = np.where(np.arange(bt.shape[1]) < need[:, None],
                     start[:, None] + np.arange(bt.shape[1]), -1).astype(np.int32)
    by_hand = pa.prefill_varlen(dev(q), pool, dev(cu[0]), dev(cu[1]), dev(table), 300, 8)
    assert torch.equal(out, by_hand)


# ------------------------------------------------------------------ together

@pytest.mark.parametrize("H,Hk,d", [(8, 2, 64), (16, 2, 128)])
def test_serving_loop(H, Hk, d):
    """Prompts in two chunks, then decode steps, through the block manager: the
    quantised append, prefill and decode of each against the oracle, and the
    whole history read back at the end."""
    rng = np.random.default_rng(80 + d)
    prompts, chunk, steps = [37, 5, 90], 40, 3
    NB, B = 24, len(prompts)
    bm = pa.BlockManager(NB)
    cache = pa.CacheI4(1, NB, Hk, d)
    cache.buffer.fill_(0xFF)
    tiles = cache.tiles.cpu().numpy().copy()
    table, status = pa.rope_table(256, d), pa.new_status()
    for s, n in enumerate(prompts):
        bm.allocate(s, rng.integers(0, 1000, n))

    def padded_tables():
        rows = [bm.block_table(s) for s in range(B)]
        w = max(len(r) for r in rows)
        return np.array([np.pad(r, (0, w - len(r)), constant_values=-1) for r in rows], np.int32)

    def store(md):
        T = len(md["positions"])
        q, k, v = (normal16(rng, T, h, d) for h in (H, Hk, Hk))
        qd = dev(q)
        pa.rope_kv_write_i4(qd, dev(k), dev(v), dev(md["positions"]), dev(md["slot_mapping"]),
                            table, cache, status=status)
        q_rot = orc.rope_pinned(q, md["positions"], d)
        orc.kv_write_i4(tiles, 0, orc.rope_pinned(k, md["positions"], d), v, md["slot_mapping"])
        assert np.array_equal(bits(qd), bits(q_rot))
        assert np.array_equal(cache.tiles.cpu().numpy(), tiles)
        return qd, q_rot

    for _ in range(3):
        spans = [bm.next_chunk(s, chunk) for s in range(B)]
        if not any(n for _, n in spans):
            break
        bt = padded_tables()
        md = pa.prepare_prefill([c for c, _ in spans], [n for _, n in spans], bt)
        qd, q_rot = store(md)
        ws = pa.prefill_i4_workspace(int((-(-np.diff(md["cu_seqlens_k"]) // 16)).sum()), B,
                                     bt.shape[1], Hk, d)
        out = pa.prefill_varlen_i4(qd, cache, dev(md["cu_seqlens_q"]), dev(md["cu_seqlens_k"]),
                                   dev(bt), md["max_seqlen_q"], Hk, ws, status=status)
        want = prefill_want(q_rot, tiles, bt, (md["cu_seqlens_q"], md["cu_seqlens_k"]), Hk)
        assert_attention_close(out, want)
        for s, (_, n) in enumerate(spans):
            bm.mark_computed(s, n)
    ws = pa.decode_i4_workspace(B, H, Hk, d)
    for _ in range(steps):
        cached = [bm.num_tokens(s) for s in range(B)]
        for s in range(B):
            bm.append(s, 7)
        bt = padded_tables()
        md = pa.prepare_decode(cached, bt)
        qd, q_rot = store(md)
        out = pa.decode_i4(qd, cache, dev(bt), dev(md["context_lens"]), ws, Hk, status=status)
        want, tol = decode_want(q_rot, tiles, 0, bt, md["context_lens"], Hk)
        assert (np.abs(out.cpu().numpy() - want) <= tol).all()
    lens = md["context_lens"]
    rows = (np.cumsum(lens) - lens).astype(np.int32)
    k, v = (torch.empty(int(lens.sum()), Hk, d, dtype=torch.float16, device="cuda")
            for _ in range(2))
    pa.kv_read_i4(cache, dev(bt), dev(lens), dev(rows), k, v, status=status)
    vals = orc.read_rows_i4(orc.dequantize_cache_i4(tiles))
    for kv, got in enumerate((k, v)):
        want = np.concatenate([vals[kv, 0][bt[s, :-(-n // 16)]].reshape(-1, Hk, d)[:n]
                               for s, n in enumerate(lens)])
        assert np.array_equal(bits(got), bits(want))
    assert int(status.item()) == 0


def test_captured_step_replays():
    """A decode step (append, then decode) captured once in a CUDA graph and
    replayed with other tokens, positions and lengths; a second graph that
    shares the workspace, replayed in turn."""
    H, Hk, d, NB = 16, 2, 128, 80
    rng = np.random.default_rng(90)
    tiles = orc.pack_cache_i4(normal16(rng, 2, 1, NB, 16, Hk, d))
    bt = rng.permutation(NB).astype(np.int32).reshape(2, NB // 2)
    ws, table = pa.decode_i4_workspace(2, H, Hk, d), pa.rope_table(NB * 8, d)
    cache, status = cache_of(tiles), pa.new_status()
    btd = dev(bt)
    graphs = []
    for _ in range(2):
        b = dict(q=torch.zeros(2, H, d), k=torch.zeros(2, Hk, d), v=torch.zeros(2, Hk, d))
        b = {n: t.half().cuda() for n, t in b.items()}
        b |= {n: torch.zeros(2, dtype=torch.int32, device="cuda") for n in ("pos", "slots", "ctx")}
        b["slots"].fill_(-1)
        b["ctx"].fill_(1)
        b["q_out"], b["out"] = torch.empty_like(b["q"]), torch.empty_like(b["q"])

        def step(b=b):
            pa.rope_kv_write_i4(b["q"], b["k"], b["v"], b["pos"], b["slots"], table, cache,
                                q_out=b["q_out"], status=status)
            pa.decode_i4(b["q_out"], cache, btd, b["ctx"], ws, Hk, out=b["out"], status=status)

        step()  # once outside the capture
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step()
        graphs.append((g, b))
    cached = np.array([3, 500])
    for i in range(6):
        g, b = graphs[i % 2]
        md = pa.prepare_decode(cached, bt)
        q, k, v = (normal16(rng, 2, h, d) for h in (H, Hk, Hk))
        for n, x in (("q", q), ("k", k), ("v", v), ("pos", md["positions"]),
                     ("slots", md["slot_mapping"]), ("ctx", md["context_lens"])):
            b[n].copy_(torch.from_numpy(x))
        g.replay()
        torch.cuda.synchronize()
        q_rot = orc.rope_pinned(q, md["positions"], d)
        orc.kv_write_i4(tiles, 0, orc.rope_pinned(k, md["positions"], d), v, md["slot_mapping"])
        assert np.array_equal(cache.tiles.cpu().numpy(), tiles)
        want, tol = decode_want(q_rot, tiles, 0, bt, md["context_lens"], Hk)
        assert (np.abs(b["out"].cpu().numpy() - want) <= tol).all()
        cached += 1 + 13 * (i % 3)
    assert int(status.item()) == 0


def test_binding_refuses_shapes_and_places():
    c = pa.CacheI4(1, 4, 2, 64)
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")  # noqa: E731
    f16 = lambda *s: torch.zeros(*s, dtype=torch.float16, device="cuda")  # noqa: E731
    with pytest.raises(ValueError):
        pa.kv_read_i4(c, i32(2, 4), i32(2), i32(2), f16(8, 2, 64), f16(9, 2, 64))
    with pytest.raises(ValueError):
        pa.kv_read_i4(c, i32(2, 4), i32(2), i32(2), f16(8, 3, 64))
    with pytest.raises(ValueError):
        pa.kv_read_i4(c, i32(2, 4), i32(3), i32(2), f16(8, 2, 64))
    with pytest.raises(TypeError):
        pa.decode_i4(f16(2, 64, 4).transpose(1, 2), c, i32(2, 4), i32(2),
                     pa.decode_i4_workspace(2, 4, 2, 64), 2)
    with pytest.raises(pa.PAError):
        pa.decode_i4(f16(2, 4, 64), c, i32(2, 4), i32(2), pa.decode_i4_workspace(2, 4, 2, 64), 4)
    with pytest.raises(ValueError):
        pa.CacheI4(1, 4, 2, 64, buffer=torch.empty(100, dtype=torch.uint8, device="cuda"))
    with pytest.raises(pa.PAError):
        n = pa.cache_i4_bytes(1, 4, 16, 2, 64)
        pa.CacheI4(1, 4, 2, 64, buffer=torch.empty(n + 16, dtype=torch.uint8, device="cuda")[16:])
    table, ws = pa.rope_table(4, 64), pa.decode_i4_workspace(2, 4, 2, 64)
    with pytest.raises(TypeError):
        pa.rope_kv_write_i4(f16(1, 4, 64), f16(1, 2, 64), f16(1, 2, 64).cpu(), i32(1), i32(1),
                            table, c)
    q, bt, ctx = f16(2, 4, 64), i32(2, 4), i32(2)
    for bad in (q.cpu(), q.float(), None, [1], q.permute(1, 0, 2)):
        with pytest.raises(TypeError):
            pa.decode_i4(bad, c, bt, ctx, ws, 2)
    for args in ((q[0], c, bt, ctx, ws, 2), (q, c, bt[0], ctx, ws, 2), (q, c, bt, ctx[:1], ws, 2),
                 (q, c, bt[:1], ctx, ws, 2)):
        with pytest.raises(ValueError):
            pa.decode_i4(*args)
    for args in ((q, c, bt.long(), ctx, ws, 2), (q, c, bt, ctx.float(), ws, 2),
                 (q, c, bt, ctx, ws.int(), 2), (q, c, bt.cpu(), ctx, ws, 2), (q, c, bt, ctx, None, 2)):
        with pytest.raises(TypeError):
            pa.decode_i4(*args)
    with pytest.raises(ValueError):
        pa.decode_i4(q, c, bt, ctx, ws, 2, out=f16(2, 4, 128))
    with pytest.raises(ValueError):
        pa.decode_i4(q, c, bt, ctx, ws, 2, status=i32(2))
    with pytest.raises(TypeError):  # a pool of another kind
        pa.decode_i4(q, pa.CacheI8(1, 4, 2, 64), bt, ctx, ws, 2)
    with pytest.raises(TypeError):
        pa.kv_read_i4(c, None, ctx, ctx, f16(4, 2, 64))
    with pytest.raises(ValueError):
        pa.kv_read_i4(c, bt, ctx, ctx, f16(4, 128))
    with pytest.raises(ValueError):
        pa.prefill_varlen_i4(q, c, i32(4), i32(3), bt, 1, 2, ws)
