"""The 4-bit KV cache without a GPU: the oracle's quantisation pinned by worked
examples, its error bound and the tile layout, and the host side of the
library's entry points (sizes, refusals)."""

import ctypes

import numpy as np
import pytest
import torch

from oracle import reference as orc
from paged_kv_gqa_rope_gb300 import pa


def test_worked_example():
    x = np.arange(32, dtype=np.float16)[None]  # 0 .. 31: step 31/15 rounded up, ties to even
    c, s, m = orc.kv_quantize_int4(x)
    assert m[0, 0] == 0 and float(s[0, 0]) >= 31 / 15 > float(np.nextafter(s[0, 0], np.float16(0)))
    assert c[0, 0] == 0 and c[0, 1] == 0 and c[0, 2] == 1 and c[0, 31] == 15
    x = (np.arange(32) % 16).astype(np.float16)[None] - 7  # step exactly 1
    c, s, m = orc.kv_quantize_int4(x)
    assert s[0, 0] == 1 and m[0, 0] == -7 and np.array_equal(c[0], np.arange(32) % 16)


@pytest.mark.parametrize("scale", [6e-8, 1e-6, 1e-3, 0.05, 1.0, 30.0, 6e4])
def test_reads_back_within_half_a_step(scale):
    rng = np.random.default_rng(3)
    x = np.clip(rng.standard_normal((200, 128)) * scale, -65504, 65504).astype(np.float16)
    c, s, m = orc.kv_quantize_int4(x)
    step, least = (np.repeat(y.astype(np.float64), 32, -1) for y in (s, m))
    # half a step, and the fp32 rounding of the quotient (below 15.5) where it decided
    err = np.abs(least + step * c - x.astype(np.float64))
    assert (err <= step * (0.5 + 16 * 2.0 ** -23)).all()
    assert c.max() == 15 or scale < 1e-7


def test_constant_and_non_finite_groups():
    x = np.full((3, 64), 5.0, np.float16)
    x[1, 40] = np.inf
    x[2, 3] = np.nan
    c, s, m = orc.kv_quantize_int4(x)
    assert (c == 0).all() and s[0].tolist() == [0, 0] and m[0].tolist() == [5, 5]
    assert s[1, 1] == 0 and np.isnan(m[1, 1]) and m[1, 0] == 5
    assert s[2, 0] == 0 and np.isnan(m[2, 0]) and m[2, 1] == 5
    x = np.zeros((1, 32), np.float16)
    x[0, :2] = [-65504, 65504]  # the widest range: the step is finite, the top saturates
    c, s, m = orc.kv_quantize_int4(x)
    assert np.isfinite(s).all() and c[0, 1] == 15
    assert orc.read_rows_i4(m.astype(np.float64) + s.astype(np.float64) * 15)[0, 0] == 65504


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("is_v", [False, True])
def test_tile_layout_is_a_bijection(d, is_v):
    byte, shift, step, least = orc.kv_i4_places(d, is_v)
    nib = 2 * byte + shift // 4
    assert sorted(nib.ravel()) == list(range(16 * d))
    assert sorted(np.concatenate([step.ravel(), least.ravel()])) == list(range(d))


@pytest.mark.parametrize("d", [64, 128])
def test_write_agrees_with_pack_and_reads_back(d):
    rng = np.random.default_rng(5)
    pool = rng.standard_normal((2, 2, 3, 16, 2, d)).astype(np.float16)
    tiles = orc.pack_cache_i4(pool)
    got = orc.new_cache_i4(2, 3, 2, d)
    for layer in range(2):
        orc.kv_write_i4(got, layer, pool[0, layer].reshape(48, 2, d),
                        pool[1, layer].reshape(48, 2, d), rng.permutation(48) * 0 + np.arange(48))
    assert np.array_equal(got, tiles)
    vals = orc.dequantize_cache_i4(tiles)
    c, s, m = orc.kv_quantize_int4(pool)
    want = np.repeat(m.astype(np.float64), 32, -1) + np.repeat(s.astype(np.float64), 32, -1) * c
    assert np.array_equal(vals, want)


def test_sizes(libpa):
    assert pa.cache_i4_bytes(2, 10, 16, 8, 128) == 2 * 10 * 8 * 2 * 1280
    assert pa.cache_i4_bytes(1, 1, 16, 1, 64) == 1280
    assert pa.cache_i4_bytes(1, 0, 16, 1, 64) == 0
    # 5/16 of the fp16 pool
    assert 16 * pa.cache_i4_bytes(3, 7, 16, 5, 128) == 5 * pa.cache_bytes(3, 7, 16, 5, 128)
    assert pa.cache_i4_bytes(80, 1 << 20, 16, 8, 128) == 80 * (1 << 20) * 8 * 2560  # past 32 bits
    assert pa.cache_i4_bytes(1 << 30, 1 << 27, 16, 1 << 20, 64) == 0  # past 64
    assert pa.cache_i4_bytes(1 << 30, 1 << 27, 16, 1, 4) == (1 << 61) * 5
    assert pa.cache_i4_bytes(1 << 30, 1 << 27, 16, 1, 7) == 0  # (the values fit)
    assert libpa.pa_decode_i4_workspace_bytes(0, 8, 8, 128) == 0
    assert libpa.pa_decode_i4_workspace_bytes(32, 64, 8, 128) > 0
    assert libpa.pa_prefill_i4_workspace_bytes(0, 1, 1, 8, 128) == 0
    assert libpa.pa_prefill_i4_workspace_bytes(100, 2, 30, 8, 128) >= 100 * 16 * 8 * 128 * 4 + 240


def test_prefill_workspace_past_64_bits(libpa):
    big = 2**31 - 1
    size = libpa.pa_prefill_i4_workspace_bytes
    assert size(big, 1, 1, big, 128) == 0
    assert size(1 << 30, 1, 1, 1 << 30, 128) == 0  # 2^73: all 64 low bits are 0
    assert size(1, big, big, big, big) == 0        # (each part fits)
    assert size(1 << 28, 1, 1, 1 << 20, 128) == (1 << 61) + 256
    with pytest.raises(ValueError):
        pa.prefill_i4_workspace(1 << 30, 1, 1, 1 << 30, 128)


def descriptor(libpa, heads=2, d=64, layers=1, blocks=10):
    c = pa.PaCacheI4()
    fake = ctypes.c_void_p(1 << 20)  # never dereferenced on the host
    assert libpa.pa_alloc_cache_i4(ctypes.byref(c), layers, blocks, 16, heads, d, fake) == pa.PA_OK
    return c


def test_descriptor(libpa):
    c = descriptor(libpa, layers=3)
    assert c.base == 1 << 20 and c.owns == 0 and c.layers == 3 and c.num_blocks == 10
    assert libpa.pa_free_cache_i4(ctypes.byref(c)) == pa.PA_OK and not c.base
    assert libpa.pa_free_cache_i4(None) == pa.PA_ERR_INVALID
    fake = ctypes.c_void_p(1 << 20)
    r = ctypes.byref(c)
    assert libpa.pa_alloc_cache_i4(None, 1, 1, 16, 1, 64, fake) == pa.PA_ERR_INVALID
    assert libpa.pa_alloc_cache_i4(r, 1, 10, 8, 8, 128, fake) == pa.PA_ERR_UNSUPPORTED
    assert libpa.pa_alloc_cache_i4(r, 1, 10, 16, 8, 96, fake) == pa.PA_ERR_UNSUPPORTED
    assert libpa.pa_alloc_cache_i4(r, 1, 0, 16, 8, 128, fake) == pa.PA_ERR_INVALID
    assert libpa.pa_alloc_cache_i4(r, 1, 1 << 28, 16, 8, 128, fake) == pa.PA_ERR_INVALID
    assert libpa.pa_alloc_cache_i4(r, 1, 1, 16, 1 << 20, 128, fake) == pa.PA_ERR_UNSUPPORTED
    assert libpa.pa_alloc_cache_i4(r, 1, 10, 16, 8, 128,
                                   ctypes.c_void_p(1 << 20 | 16)) == pa.PA_ERR_INVALID


def test_pool_in_host_memory_is_refused(libpa):
    with pytest.raises(ValueError):
        pa.CacheI4(1, 4, 2, 64, device="cpu")
    with pytest.raises(TypeError):
        pa.CacheI4(1, 4, 2, 64, buffer=torch.empty(1 << 16, dtype=torch.uint8))


BUF = ctypes.c_void_p(1 << 24)
APART = ctypes.c_void_p(1 << 26)
ODD = ctypes.c_void_p((1 << 26) + 8)


def test_write_refusals(libpa):
    c = descriptor(libpa)

    def call(q=BUF, q_out=BUF, k=APART, v=APART, pos=BUF, slots=BUF, T=4, H=4, Hk=2, d=64,
             table=BUF, maxpos=8, cache=c, layer=0):
        return libpa.pa_rope_kv_write_i4(q, q_out, k, v, pos, slots, T, H, Hk, d, table, maxpos,
                                         None if cache is None else ctypes.byref(cache), layer,
                                         None, None)

    assert call(T=0, q=None, k=None) == pa.PA_OK
    assert call(d=96) == pa.PA_ERR_UNSUPPORTED
    assert call(T=1, H=2**26) == pa.PA_ERR_UNSUPPORTED
    for bad in (dict(T=-1), dict(H=5), dict(Hk=4), dict(layer=1), dict(layer=-1), dict(maxpos=0),
                dict(cache=None), dict(q=None), dict(q_out=None), dict(k=None), dict(v=None),
                dict(pos=None), dict(slots=None), dict(table=None), dict(q=ODD), dict(q_out=ODD),
                dict(k=ODD), dict(v=ODD), dict(table=ODD), dict(T=2**31 - 1, H=2**30, Hk=2)):
        assert call(**bad) == pa.PA_ERR_INVALID, bad
    # q_out may be q, but not overlap it otherwise, nor k or v
    assert call(q_out=ctypes.c_void_p((1 << 24) + 16)) == pa.PA_ERR_INVALID
    assert call(q_out=APART) == pa.PA_ERR_INVALID
    assert call(q=APART, q_out=APART, k=BUF, v=APART) == pa.PA_ERR_INVALID


def test_read_refusals(libpa):
    c = descriptor(libpa)

    def call(cache=c, layer=0, bt=BUF, maxb=4, lens=BUF, first=None, rows=BUF, B=2, total=64,
             Hk=2, d=64, k=BUF, v=BUF):
        return libpa.pa_kv_read_i4(None if cache is None else ctypes.byref(cache), layer, bt, maxb,
                                   lens, first, rows, B, total, Hk, d, k, v, None, None)

    assert call(B=0, bt=None, lens=None) == pa.PA_OK
    assert call(k=None, v=None) == pa.PA_OK  # nothing to write
    assert call(d=96) == pa.PA_ERR_UNSUPPORTED
    assert call(B=4097) == pa.PA_ERR_UNSUPPORTED
    for bad in (dict(B=-1), dict(total=-1), dict(maxb=0), dict(maxb=(2**31 - 1) // 16 + 1),
                dict(Hk=4), dict(Hk=0), dict(layer=1), dict(cache=None), dict(bt=None),
                dict(lens=None), dict(rows=None), dict(k=ODD), dict(v=ODD)):
        assert call(**bad) == pa.PA_ERR_INVALID, bad


def test_decode_refusals(libpa):
    c = descriptor(libpa)

    def call(q=BUF, cache=c, layer=0, bt=BUF, maxb=4, ctx=BUF, B=2, H=4, Hk=2, d=64, scale=0.0,
             ws=BUF, wsb=1 << 30, out=BUF):
        return libpa.pa_decode_i4(q, None if cache is None else ctypes.byref(cache), layer, bt,
                                  maxb, ctx, B, H, Hk, d, scale, ws, wsb, out, None, None)

    assert call(B=0, q=None, ws=None) == pa.PA_OK
    assert call(d=96) == pa.PA_ERR_UNSUPPORTED
    assert call(H=32) == pa.PA_ERR_UNSUPPORTED  # a group of 16
    assert call(B=4097) == pa.PA_ERR_UNSUPPORTED
    assert call(wsb=16) == pa.PA_ERR_WORKSPACE
    for bad in (dict(B=-1), dict(H=5), dict(Hk=4), dict(layer=1), dict(maxb=0),
                dict(maxb=(2**31 - 1) // 16 + 1), dict(scale=-1.0), dict(scale=float("nan")),
                dict(cache=None), dict(q=None), dict(bt=None), dict(ctx=None), dict(ws=None),
                dict(out=None), dict(q=ODD), dict(out=ODD),
                dict(ws=ctypes.c_void_p((1 << 24) + 128))):
        assert call(**bad) == pa.PA_ERR_INVALID, bad


def test_prefill_refusals(libpa):
    c = descriptor(libpa)

    def call(q=BUF, T=8, cache=c, layer=0, cuq=BUF, cuk=BUF, bt=BUF, maxb=4, B=2, mq=4, H=4, Hk=2,
             d=64, scale=0.0, ws=BUF, wsb=1 << 30, out=BUF):
        return libpa.pa_prefill_varlen_i4(q, T, None if cache is None else ctypes.byref(cache),
                                          layer, cuq, cuk, bt, maxb, B, mq, H, Hk, d, scale, ws,
                                          wsb, out, None, None)

    assert call(B=0, q=None) == pa.PA_OK
    assert call(T=0, q=None) == pa.PA_OK
    assert call(d=96) == pa.PA_ERR_UNSUPPORTED
    assert call(B=2049) == pa.PA_ERR_UNSUPPORTED
    need = libpa.pa_prefill_i4_workspace_bytes(1, 2, 4, 2, 64)
    assert call(wsb=need - 1) == pa.PA_ERR_WORKSPACE
    for bad in (dict(B=-1), dict(T=-1), dict(mq=-1), dict(H=5), dict(Hk=4), dict(layer=1),
                dict(maxb=0), dict(scale=-1.0), dict(cache=None), dict(q=None), dict(cuq=None),
                dict(cuk=None), dict(bt=None), dict(ws=None), dict(out=None), dict(q=ODD),
                dict(out=ODD), dict(ws=ctypes.c_void_p((1 << 24) + 128))):
        assert call(**bad) == pa.PA_ERR_INVALID, bad
