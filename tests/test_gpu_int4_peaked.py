"""Decode over the 4-bit cache where one key has most of the weight and V is
small, and its relative error over sizes of K and V: against the attention
formula, in 64 bits, on the values that the codes stand for.

The bound, on the L2 error of a sequence's outputs.  A rounding to fp16 is off by
an even distribution over one step, at most 2^-10 of the value, so by an rms of at
most u = 2^-10 / sqrt(12) of it.  The kernel rounds p s once (a term p s (c - 8)),
and p and the centre m + 8 s once each (a term p (m + 8 s)); for normal values of
variance 1 in groups of 32 the two terms' mean squares are 1.08 and 0.14 (half the
range's variance, and s^2 / 4), so that those three roundings come to
sqrt(1.08 + 2 * 0.14) u = 1.17 u of the output, which is less than 2 u; with a mean
the centre's part of the output only grows.  The fp16 output's own rounding has an
rms of its step / sqrt(12), which the bound adds.  fp32 scores of at most some tens,
off by some 2^-20, do not show beside it.

Where the output is a few subnormal steps of fp16, its own rounding is all that the
bound holds, and an rms taken over N outputs scatters: the square of an error even
over one step h has the mean h^2 / 12 and the variance h^4 / 180, so the mean of N
of them the relative deviation sqrt(144 / 180 / N), of which four are allowed (512
outputs: 7.6 % of the rms)."""

import math

import numpy as np
import pytest
import torch

from oracle import reference as orc
from paged_kv_gqa_rope_gb300 import pa

pytestmark = pytest.mark.gpu

U = 2.0 ** -10 / math.sqrt(12)


@pytest.fixture(scope="module", autouse=True)
def _lib(libpa):
    assert torch.cuda.is_available()
    assert pa.check_device() == pa.PA_OK
    return libpa


def step16(x):
    """The fp16 step at every value of x (fp64), below the normal range 2^-24."""
    _, e = torch.frexp(x.abs().clamp(min=2.0 ** -14, max=65504))
    return torch.ldexp(torch.ones_like(x), e - 11)


def bound(want):
    own = step16(want).norm() / math.sqrt(12) * math.sqrt(1 + 4 * math.sqrt(0.8 / want.numel()))
    return float(2 * U * want.norm() + own)


def values(cache, table, n):
    """K and V [Hk, n, d] in 64 bits of one sequence's first n tokens."""
    d = cache.desc.head_dim
    tiles = cache.tiles[0, table.long()]  # [blocks, Hk, 2, 10 d]
    out = []
    for kv in (0, 1):
        byte, shift, step, least = (torch.from_numpy(x).cuda() for x in orc.kv_i4_places(d, kv == 1))
        p = tiles[:, :, kv, 8 * d:].contiguous().view(torch.float16).double()
        c = (tiles[:, :, kv][..., byte].int() >> shift) & 15
        x = p[..., least].repeat_interleave(32, -1) + p[..., step].repeat_interleave(32, -1) * c
        out.append(x.transpose(0, 1).flatten(1, 2)[:, :n])
    return out


def attend(q, k, v, keep=None):
    """softmax(q K^T / sqrt(d)) V for q [H, d], over the keys `keep`, in 64 bits."""
    H, d = q.shape
    x = q.double().view(k.shape[0], -1, d) @ k.transpose(-1, -2) / math.sqrt(d)
    if keep is not None:
        x = x.masked_fill(~keep, -math.inf)
    w = torch.softmax(x, -1)
    return (w @ v).view(H, d), w


def codes_and_centres(cache, table, n):
    """|c - 8| s and |m + 8 s| [Hk, n, d] of V, and its largest step."""
    d = cache.desc.head_dim
    byte, shift, step, least = (torch.from_numpy(x).cuda() for x in orc.kv_i4_places(d, True))
    x = cache.tiles[0, table.long()][:, :, 1]
    p = x[..., 8 * d:].contiguous().view(torch.float16).double()
    c = (x[..., byte].int() >> shift) & 15
    s, m = (p[..., y].repeat_interleave(32, -1) for y in (step, least))
    rows = lambda y: y.transpose(0, 1).flatten(1, 2)[:, :n]  # noqa: E731
    return rows((c - 8).abs() * s), rows((m + 8 * s).abs()), float(rows(s).max())


def fill(lens, Hk, d, make, seed):
    """A pool with every sequence's K and V rows as `make(rng, s, n)` gives them,
    appended without rotation; returns (cache, block tables)."""
    need = [-(-n // 16) for n in lens]
    rng = torch.Generator(device="cuda").manual_seed(seed)
    order = torch.randperm(sum(need), device="cuda", generator=rng).int()
    bt = torch.full((len(lens), max(need)), -1, dtype=torch.int32, device="cuda")
    cache, table, at = pa.CacheI4(1, sum(need), Hk, d), pa.rope_table(1, d), 0
    for s, n in enumerate(lens):
        bt[s, :need[s]] = order[at:at + need[s]]
        at += need[s]
        k, v = make(rng, s, n)
        t = torch.arange(n, device="cuda")
        slots = bt[s, t // 16] * 16 + t.int() % 16
        q = torch.zeros(n, Hk, d, dtype=torch.float16, device="cuda")
        pa.rope_kv_write_i4(q, k.half(), v.half(), torch.zeros_like(slots), slots, table, cache)
    return cache, bt


def decode(q, cache, bt, lens):
    B, H, d = q.shape
    Hk, status = cache.desc.n_kv_heads, pa.new_status()
    ctx = torch.tensor(lens, dtype=torch.int32, device="cuda")
    out = pa.decode_i4(q, cache, bt, ctx, pa.decode_i4_workspace(B, H, Hk, d), Hk, status=status)
    assert int(status.item()) == 0
    return out.double()


# (sequences, Q heads, KV heads, d): a few pairs, cut between many warps, and as many
# pairs as the 152 x 12 warps of a launch, so that a warp holds whole pairs
FEW = [(2, 8, 2, 128), (3, 2, 1, 64)]
MANY = [(57, 32, 32, 128), (228, 16, 8, 64)]


@pytest.mark.parametrize("shape,n", [(s, n) for s in FEW + MANY for n in (2000, 4096)] +
                         [(s, 32768) for s in FEW + MANY[1:]])
@pytest.mark.parametrize("weight,std,mean", [(0.7, 0.3, 0.0), (0.9, 0.1, 0.0), (0.75, 0.05, 0.0),
                                             (0.98, 0.05, 0.0), (0.9, 0.02, 0.0), (0.9, 0.02, 0.01),
                                             (0.9, 1e-3, 1e-3), (0.9, 40.0, 0.0)])
def test_decode_beside_a_key_with_most_of_the_weight(shape, n, weight, std, mean):
    B, H, Hk, d = shape
    lens = [n - 3 * (s % 5) for s in range(B)]
    rng = torch.Generator(device="cuda").manual_seed(7)
    # every query has 8 along one direction, which the heavy key points along
    u = torch.nn.functional.normalize(torch.randn(d, device="cuda", generator=rng), dim=0)
    q = torch.randn(B, H, d, device="cuda", generator=rng)
    q = (q + (8 - q @ u)[..., None] * u).half()
    # the sum of exp over the others, whose scores have a variance of (|q| / sqrt(d))^2
    rest = math.log(n) + (d + 64) / d / 2
    heavy = (math.log(weight / (1 - weight)) + rest) * math.sqrt(d) / 8 * u

    def make(rng, s, n):
        k, v = (torch.randn(n, Hk, d, device="cuda", generator=rng) for _ in range(2))
        at = (0, n // 2, n - 1)[s % 3]
        k[at], v = heavy, v * std + mean
        v[at] = 0
        return k, v

    cache, bt = fill(lens, Hk, d, make, 11)
    got = decode(q, cache, bt, lens)
    for s in {0, 1, 2, B // 2, B - 1} & set(range(B)):
        k, v = values(cache, bt[s, :-(-lens[s] // 16)], lens[s])
        want, w = attend(q[s], k, v)
        most = w.amax(-1)
        assert weight - 0.2 < float(most.mean()) < weight + 0.15, float(most.mean())
        tol = bound(want)
        # what the bound has to see: no output at all, and a block left out (with a
        # mean, whose share of the output one block hardly moves, eight)
        keep = torch.ones(lens[s], dtype=torch.bool, device="cuda")
        keep[80:208 if mean else 96] = False
        assert float(want.norm()) > 100 * tol
        assert float((attend(q[s], k, v, keep)[0] - want).norm()) > tol
        err = float((got[s] - want).norm())
        assert err <= tol, (s, err / float(want.norm()), tol / float(want.norm()))


@pytest.mark.parametrize("H,Hk,d", [(16, 4, 128), (8, 8, 64)])
@pytest.mark.parametrize("std_k,std_v,mean", [(1.0, 1.0, 0.0), (1e-3, 1.0, 0.0), (4.0, 1.0, 0.0),
                                              (1.0, 0.05, 0.0), (1.0, 1e-3, 0.0), (1.0, 1e-5, 0.0),
                                              (1.0, 5e3, 0.0), (1.0, 1.0, 50.0)])
def test_decode_relative_error(H, Hk, d, std_k, std_v, mean):
    """A bound that is a share of the output, whatever the size of V and the length."""
    lens = [1, 16, 100, 999, 20000]
    rng = torch.Generator(device="cuda").manual_seed(8)
    q = torch.randn(len(lens), H, d, device="cuda", generator=rng).half()

    def make(rng, s, n):
        k, v = (torch.randn(n, Hk, d, device="cuda", generator=rng) for _ in range(2))
        return k * std_k, v * std_v + mean

    cache, bt = fill(lens, Hk, d, make, 12)
    got = decode(q, cache, bt, lens)
    for s, n in enumerate(lens):
        k, v = values(cache, bt[s, :-(-n // 16)], n)
        want = attend(q[s], k, v)[0]
        err = float((got[s] - want).norm())
        assert err <= bound(want), (n, err / float(want.norm()), bound(want) / float(want.norm()))


@pytest.mark.parametrize("std_v,mean", [(1.0, 0.0), (0.02, 0.0), (0.02, 1.0), (30.0, 0.0)])
@pytest.mark.parametrize("H,Hk,d", [(8, 8, 128), (32, 8, 128), (64, 8, 128), (16, 8, 64), (8, 1, 64),
                                    (8, 1, 128), (14, 2, 64), (6, 2, 128), (35, 7, 128),
                                    (1, 1, 128), (1, 1, 64)])
def test_decode_edge_lengths_value_by_value(H, Hk, d, std_v, mean):
    """Every output within what its roundings can come to, a share of the weighted
    values.  With w the weights relative to the largest:
      - p s, p and the centre, half a step of fp16 each: 2^-11 of |c - 8| s w and
        of |m + 8 s| w twice, and 2^-20 of both for the second order and fp32;
      - p s below the normal range: 2^-33 of the largest step s' for each key,
        times |c - 8| <= 8, and p there 2^-38 of the centre, which does not show;
      - the tensor core's truncated sums of p s c, c <= 15, of up to 16 keys a
        block: 2^-23 of at most 240 s' (w = 1) for each block of 16 keys;
      - scores of at most 16, off by 300 roundings of 2^-24 of that: the weights
        by 2^-12, relatively, of which half stays after the normalisation's
        average at the very most: 2^-12 of the weighted size of V about its mean;
      - half a step of the output."""
    lens = [1, 2, 7, 8, 9, 15, 16, 17, 31, 32, 33, 47, 48, 49, 255, 256, 257, 1000, 4100]
    rng = torch.Generator(device="cuda").manual_seed(H + Hk + d)
    q = torch.randn(len(lens), H, d, device="cuda", generator=rng).half()

    def make(rng, s, n):
        k, v = (torch.randn(n, Hk, d, device="cuda", generator=rng) for _ in range(2))
        return k, v * std_v + mean

    cache, bt = fill(lens, Hk, d, make, 15)
    got = decode(q, cache, bt, lens)
    for s, n in enumerate(lens):
        table = bt[s, :-(-n // 16)]
        k, v = values(cache, table, n)
        code, centre, top = codes_and_centres(cache, table, n)
        want, w = attend(q[s], k, v)

        def mean_of(x):
            return (w @ x).view(H, d)

        most = w.amax(-1, keepdim=True).expand(-1, -1, d).reshape(H, d)  # 1 / sum of w
        about = mean_of(v.square()) - want.square()
        tol = (2.0 ** -11 + 2.0 ** -20) * (mean_of(code) + 2 * mean_of(centre)) + \
            n * top * most * (2.0 ** -30 + 2.0 ** -23 * 15) + \
            2.0 ** -12 * about.clamp(min=0).sqrt() + step16(want) / 2
        off = (got[s] - want).abs()
        assert bool((off <= tol).all()), (n, float((off / tol).max()))
        # no output, and a block left out, are seen (not beside a mean of 50 times the
        # spread: 16 of 1000 keys move the output by 0.02 * 4 / 1000 = 8e-5, less than
        # half a step of an fp16 output of 1, 2.4e-4)
        assert float((want.abs() / tol).max()) > 20
        if n > 32 and mean == 0:
            keep = torch.arange(n, device="cuda") >= 16
            assert bool(((attend(q[s], k, v, keep)[0] - want).abs() > tol).any()), n


@pytest.mark.parametrize("shape", [(2, 8, 2, 128), (228, 16, 8, 64)])
@pytest.mark.parametrize("order", ["growing", "falling", "mixed"])
def test_decode_values_of_many_sizes(shape, order):
    """V from 2^-11 to 2^10 along one history: every size of step is met before and
    after larger ones."""
    B, H, Hk, d = shape
    lens = [3000 - 7 * (s % 5) for s in range(B)]
    rng = torch.Generator(device="cuda").manual_seed(9)
    q = torch.randn(B, H, d, device="cuda", generator=rng).half()

    def make(rng, s, n):
        size = torch.linspace(-11, 10, n, device="cuda")
        if order == "falling":
            size = size.flip(0)
        if order == "mixed":
            size = size[torch.randperm(n, device="cuda", generator=rng)]
        k, v = (torch.randn(n, Hk, d, device="cuda", generator=rng) for _ in range(2))
        return k, v * torch.exp2(size)[:, None, None]

    cache, bt = fill(lens, Hk, d, make, 13)
    got = decode(q, cache, bt, lens)
    for s in {0, 1, B // 2, B - 1}:
        k, v = values(cache, bt[s, :-(-lens[s] // 16)], lens[s])
        want = attend(q[s], k, v)[0]
        err = float((got[s] - want).norm())
        assert err <= bound(want), (s, err / float(want.norm()), bound(want) / float(want.norm()))


def test_decode_scores_past_every_fp32_integer():
    """Scores of 1e8 and more, whose fp32 steps are larger than the distance kept
    between them and the running maximum.  The two largest differ by far more than
    their rounding, so one key has all the weight."""
    lens = [300, 1000]
    rng = torch.Generator(device="cuda").manual_seed(10)
    H, Hk, d = 8, 2, 128
    q = (torch.randn(2, H, d, device="cuda", generator=rng) * 1e4).half()

    def make(rng, s, n):
        k, v = (torch.randn(n, Hk, d, device="cuda", generator=rng) for _ in range(2))
        return (k * 1e4).clamp(-6e4, 6e4), v

    cache, bt = fill(lens, Hk, d, make, 14)
    got = decode(q, cache, bt, lens)
    for s, n in enumerate(lens):
        k, v = values(cache, bt[s, :-(-n // 16)], n)
        want, w = attend(q[s], k, v)
        assert float(w.amax(-1).min()) == 1.0
        assert float((got[s] - want).norm()) <= bound(want)
