"""Edges of the 4-bit cache's calls: values at the end of fp16's range, sequences
without new tokens in a prefill batch, outputs made on a stream of the caller's, a
length bound and a layer past 32 bits."""

import numpy as np
import pytest
import torch

from oracle import reference as orc
from paged_kv_gqa_rope_gb300 import pa
from tests.gpu_helpers import assert_attention_close

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib(libpa):
    assert torch.cuda.is_available()
    assert pa.check_device() == pa.PA_OK
    return libpa


def dev(x):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


def cache_of(tiles):
    L, NB, Hk, _, n = tiles.shape
    c = pa.CacheI4(L, NB, Hk, n // 10)
    c.tiles.copy_(torch.from_numpy(tiles))
    return c


@pytest.mark.parametrize("n,sequences", [(1, 1), (5, 3), (40, 2), (3000, 1)])
@pytest.mark.parametrize("d", [64, 128])
def test_decode_saturates(d, n, sequences):
    """Finite values give finite outputs: of V rows all alike, each with -65504 and
    65504 in every group, whose step is rounded up so that the top code stands for
    65536 = -65504 + 15 * 8736, the output is V's row; a NaN's group stays NaN."""
    H, Hk, NB = 4, 2, -(-n // 16)
    rng = np.random.default_rng(3)
    pool = rng.standard_normal((2, 1, NB, 16, Hk, d)).astype(np.float16)
    row = np.where(np.arange(d) % 2, 65504, -65504).astype(np.float16)
    pool[1] = row
    pool[1, 0, 0, 0, 1, 40] = np.nan
    tiles = orc.pack_cache_i4(pool)
    assert orc.dequantize_cache_i4(tiles)[1, 0, 0, 0, 0].max() == 65536
    q = rng.standard_normal((sequences, H, d)).astype(np.float16)
    bt = dev(np.tile(np.arange(NB, dtype=np.int32), (sequences, 1)))
    ctx = torch.full((sequences,), n, dtype=torch.int32, device="cuda")
    ws = pa.decode_i4_workspace(sequences, H, Hk, d)
    out = pa.decode_i4(dev(q), cache_of(tiles), bt, ctx, ws, Hk).cpu().numpy()
    nan = np.zeros((H, d), bool)
    nan[H // Hk:, 32:64] = True
    assert np.array_equal(np.isnan(out), np.broadcast_to(nan, out.shape))
    got = out.astype(np.float64)[:, ~nan]
    want = np.broadcast_to(row.astype(np.float64), (H, d))[~nan]
    # below the saturation, three roundings of 2^-11 of at most 8 s + |m + 8 s| = 74272
    assert np.isfinite(got).all() and (np.abs(got - want) <= 3 * 2.0 ** -11 * 74272).all()


@pytest.mark.parametrize("case", ["idle", "bad table", "bad length"])
def test_prefill_leaves_out_contexts_that_no_query_sees(case):
    """A workspace for the sequences with new tokens is enough beside long idle
    ones (or one refused for its length), and an idle sequence's block table is not
    looked at."""
    H, Hk, d = 8, 2, 64
    rng = np.random.default_rng(5)
    past, new = np.array([5000, 20, 0, 3000, 7]), np.array([0, 30, 17, 0, 1])
    lens = past + new
    need = -(-lens // 16)
    NB = int(need.sum())
    tiles = orc.pack_cache_i4(rng.standard_normal((2, 1, NB, 16, Hk, d)).astype(np.float16))
    order, at = rng.permutation(NB).astype(np.int32), 0
    bt = np.full((5, need.max()), -1, np.int32)
    for s, n in enumerate(need):
        bt[s, :n] = order[at:at + n]
        at += n
    cu_q, cu_k = (np.concatenate([[0], np.cumsum(x)]).astype(np.int32) for x in (new, lens))
    q = rng.standard_normal((int(new.sum()), H, d)).astype(np.float16)
    vals = orc.read_rows_i4(orc.dequantize_cache_i4(tiles)).astype(np.float64)
    want = orc.attention_prefill(q, vals, 0, cu_q, cu_k, bt, H, Hk)
    used, rows, status = need[new > 0].sum(), slice(None), 0
    if case == "bad table":
        bt[0] = NB
        bt[3, 1] = -1
    if case == "bad length":  # more keys than its table has room for; nothing of it is read
        cu_k = cu_k.copy()
        cu_k[2:] += 16 * bt.shape[1]
        used, rows, status = used - need[1], slice(30, None), pa.PA_DEV_BAD_LENGTH
    ws = pa.prefill_i4_workspace(int(used), 5, bt.shape[1], Hk, d)
    ws.fill_(0xFF)
    got = pa.new_status()
    out = pa.prefill_varlen_i4(dev(q), cache_of(tiles), dev(cu_q), dev(cu_k), dev(bt), 30, Hk, ws,
                               status=got)
    assert int(got.item()) == status
    assert_attention_close(out, want, rows=rows)


def test_outputs_belong_to_the_stream_that_writes_them():
    """An output made by the call is not memory that was freed on the current
    stream, where work may still be using it, when the call is given another."""
    B, H, Hk, d = 64, 16, 2, 128
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    q = torch.randn(B, H, d, device="cuda").half()
    bt = torch.arange(B, dtype=torch.int32, device="cuda")[:, None]
    ctx, cu = torch.full((B,), 1, dtype=torch.int32, device="cuda"), i32(*range(B + 1))
    c4, c16 = pa.CacheI4(1, B, Hk, d), pa.Cache(1, B, Hk, d)
    c4.buffer.zero_()
    c16.tensor.zero_()
    ws4, ws16 = pa.decode_i4_workspace(B, H, Hk, d), pa.decode_workspace(B, H, Hk, d)
    wsp = pa.prefill_i4_workspace(B, B, 1, Hk, d)
    side = torch.cuda.Stream()
    for call in (lambda: pa.decode_i4(q, c4, bt, ctx, ws4, Hk, stream=side),
                 lambda: pa.prefill_varlen_i4(q, c4, cu, cu, bt, 1, Hk, wsp, stream=side),
                 lambda: pa.decode(q, c16, bt, ctx, ws16, Hk, stream=side),
                 lambda: pa.prefill_varlen(q, c16, cu, cu, bt, 1, Hk, stream=side)):
        torch.cuda.synchronize()
        freed = torch.empty_like(q)
        torch.cuda.synchronize()
        at = freed.data_ptr()
        del freed
        again = torch.empty_like(q)  # the allocator gives the block out again
        assert again.data_ptr() == at
        del again
        out = call()
        torch.cuda.synchronize()
        assert out.data_ptr() != at
        assert out.shape == q.shape and not bool(out.any())


@pytest.mark.parametrize("bound", [2**31 - 1, 2**32, 2**32 + 1, 2**63])
def test_prefill_with_a_bound_past_32_bits(bound):
    """max_seqlen_q bounds the lengths; one past int32 is no other bound, nor none."""
    T, H, Hk, d = 20, 4, 2, 64
    rng = np.random.default_rng(6)
    tiles = orc.pack_cache_i4(rng.standard_normal((2, 1, 2, 16, Hk, d)).astype(np.float16))
    q = dev(rng.standard_normal((T, H, d)).astype(np.float16))
    cu, bt = dev(np.array([0, T], np.int32)), dev(np.array([[1, 0]], np.int32))
    ws = pa.prefill_i4_workspace(2, 1, 2, Hk, d)
    outs = []
    for n in (T, bound):
        status, out = pa.new_status(), torch.full_like(q, 7.0)
        pa.prefill_varlen_i4(q, cache_of(tiles), cu, cu, bt, n, Hk, ws, out=out, status=status)
        assert int(status.item()) == 0
        outs.append(out)
    assert torch.equal(*outs) and not bool((outs[0] == 7).all())


@pytest.mark.parametrize("layer", [2**32, -2**32, 2**32 + 1, 2, -1])
def test_a_layer_outside_the_pool_is_refused(layer):
    """A layer past int32 is refused too, and not taken for its low 32 bits."""
    B, H, Hk, d = 2, 4, 2, 64
    f16 = lambda *s: torch.ones(*s, dtype=torch.float16, device="cuda")  # noqa: E731
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    c = pa.CacheI4(2, 2, Hk, d)
    c.buffer.fill_(7)
    q, bt, rows = f16(B, H, d), i32(0, 1)[:, None], i32(0, 16)
    k_out = torch.full((32, Hk, d), 9.0, dtype=torch.float16, device="cuda")
    wsd, wsp = pa.decode_i4_workspace(B, H, Hk, d), pa.prefill_i4_workspace(2, B, 1, Hk, d)
    for call in (lambda: pa.rope_kv_write_i4(q, f16(B, Hk, d), f16(B, Hk, d), i32(0, 0), rows,
                                             pa.rope_table(1, d), c, layer=layer),
                 lambda: pa.kv_read_i4(c, bt, i32(1, 1), rows, k_out, layer=layer),
                 lambda: pa.decode_i4(q, c, bt, i32(1, 1), wsd, Hk, layer=layer),
                 lambda: pa.prefill_varlen_i4(q, c, i32(0, 1, 2), i32(0, 1, 2), bt, 1, Hk, wsp,
                                              layer=layer)):
        with pytest.raises((ValueError, pa.PAError)):
            call()
    torch.cuda.synchronize()
    assert bool((c.buffer == 7).all()) and bool((k_out == 9).all()) and bool((q == 1).all())
