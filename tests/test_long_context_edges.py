"""The long-context operators' sizes, refusals and host state that test_long_context_host.py
leaves out, without a GPU."""

import ctypes
import math
import sys

import numpy as np
import pytest

from paged_kv_gqa_rope_gb300 import pa

BUF = ctypes.c_void_p(1 << 24)
INT_MAX = 2**31 - 1


def desc_of(libpa, Hk, d=64):
    x = pa.PaCache()
    assert libpa.pa_alloc_cache(ctypes.byref(x), 1, 64, 16, Hk, d, ctypes.c_void_p(1 << 20)) == 0
    return ctypes.byref(x)


def test_limits_on_heads(libpa):
    """More (sequence, KV head) pairs than 2^18 are in order (here the workspace alone is
    too small); rows past int32 and KV heads past a grid's y are not."""
    def shared(B, H, Hk):
        return libpa.pa_decode_shared(BUF, desc_of(libpa, Hk), 0, BUF, 4, BUF, B, BUF, BUF, 1, H, Hk,
                                      64, 0.0, BUF, 0, BUF, None, None)

    def weights(B, H, Hk):
        return libpa.pa_decode_weights(BUF, desc_of(libpa, Hk), 0, BUF, 4, BUF, B, H, Hk, 64, 0.0,
                                       BUF, BUF, 64, BUF, 0, BUF, None, None)

    assert shared(4096, 128, 128) == weights(4096, 128, 128) == pa.PA_ERR_WORKSPACE
    assert shared(4096, 2**19 - 1, 2**19 - 1) == pa.PA_ERR_WORKSPACE
    assert shared(4096, 2**19, 2**19) == pa.PA_ERR_UNSUPPORTED
    assert weights(4096, 65535, 65535) == pa.PA_ERR_WORKSPACE
    assert weights(1, 65536, 65536) == pa.PA_ERR_UNSUPPORTED


def test_shared_workspace_size_does_not_wrap(libpa):
    """4 (num_seqs n_kv_heads) bytes of cut words pass 64 bits where the rows do not."""
    size = libpa.pa_decode_shared_workspace_bytes
    assert size(INT_MAX, 1, INT_MAX, 128) == size(INT_MAX, 8, INT_MAX, 64) == 0
    assert size(INT_MAX, 1, 2**30, 128) > 2**63
    assert size(4096, 64, 8, 128) > 2 * 4096 * 64 * 132 * 4


def test_workspace_sizes_of_the_largest_rows(libpa):
    """head_dim + 4 values a row, counted past int32."""
    row = 4 * (INT_MAX + 4)
    assert libpa.pa_decode_shared_workspace_bytes(1, 1, 1, INT_MAX) > 608 * 16 * row
    assert libpa.pa_decode_weights_workspace_bytes(1, 1, 1, INT_MAX, 1) > 608 * 16 * row
    assert libpa.pa_decode_workspace_bytes(1, 1, 1, INT_MAX) > 608 * 16 * row
    assert libpa.pa_decode_workspace_bytes(1, 1, 1, INT_MAX) < 609 * 16 * row


def test_no_append_while_evicting(libpa):
    """pa_bm_can_append says what pa_bm_append will do between begin and end; the count of
    tokens is right at each step of a loop that evicts."""
    bm = pa.BlockManager(8)
    bm.allocate(1, list(range(40)))
    bm.mark_computed(1, 40)
    n = 40
    for step in range(30):
        assert bm.can_append(1)
        bm.append(1, step)
        n += 1
        assert bm.num_tokens(1) == n
        if step in (3, 17):
            n = 40 if step == 3 else n  # (the second time nothing goes)
            bm.evict_begin(1, n)
            assert bm.num_tokens(1) == n and not bm.can_append(1)
            with pytest.raises(pa.PAError):
                bm.append(1, 0)
            bm.evict_end(1)
            assert bm.num_tokens(1) == n and bm.can_append(1)
    assert len(bm.block_table(1)) == -(-n // 16)


def test_binding_does_not_cut_to_32_bits(libpa):
    """Numbers past int32 reach the library as themselves, bounds, or not at all; cut to
    their low 32 bits they would be another call's."""
    far = 2**32
    bm = pa.BlockManager(8)
    bm.allocate(1, list(range(60)))
    bm.mark_computed(1, 60)
    for keep in (far + 16, 2**31 + 16, sys.maxsize):
        bm.evict_begin(1, keep)  # more than it has: nothing goes
        bm.evict_end(1)
        assert bm.num_tokens(1) == 60 and len(bm.block_table(1)) == 4
    for keep in (-far + 16, 0):
        with pytest.raises(pa.PAError):
            bm.evict_begin(1, keep)
    yarn = dict(scaling="yarn", factor=2.0, original_positions=64)
    for bad in (dict(original_positions=far + 64), dict(original_positions=-far + 64)):
        with pytest.raises(ValueError):
            pa.rope_table_scaled(8, 64, **{**yarn, **bad})
    for shape in ((far + 8, 64), (8, far + 64)):
        with pytest.raises(ValueError):
            pa.rope_table_scaled(*shape, **yarn)
    with pytest.raises(ValueError):
        pa.prepare_shared(np.zeros((1, 2), np.int32), np.zeros(1, np.int32), block_size=far + 16)
    for make, sizes in ((pa.decode_shared_workspace, (2, 8, 2, 64)),
                        (pa.decode_weights_workspace, (2, 8, 2, 64, 3)),
                        (pa.kv_evict_workspace, (2, 2, 8))):
        for i in range(len(sizes)):
            if i == 4:
                continue  # (blocks of scores: int64)
            with pytest.raises(ValueError):
                make(*(x + far * (i == j) for j, x in enumerate(sizes)), device="cpu")
        assert make(*sizes, device="cpu").numel() > 0


def test_scaled_tables_take_a_base_above_one(libpa):
    def call(theta, sc=None):
        return libpa.pa_rope_table_init_scaled(BUF, 8, 64, theta,
                                               None if sc is None else ctypes.byref(sc), None)

    kinds = [None] + [pa.PaRopeScaling(k, 64, 2.0, 1.0, 4.0, 0.0) for k in range(5)]
    for sc in kinds:
        for theta in (1.0, 0.5, 0.0, -2.0, math.inf, math.nan):
            assert call(theta, sc) == pa.PA_ERR_INVALID
    # the base that NTK makes of it
    assert call(1e300, pa.PaRopeScaling(2, 0, 1e30, 0.0, 0.0, 0.0)) == pa.PA_ERR_INVALID
