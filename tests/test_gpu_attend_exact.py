"""MLA attention (hkv_mla_attend) where the logits are exact, so that what is
left of the error is the probabilities' and the sums': a few non-zero entries
of the queries and keys, small whole numbers times powers of two."""
import math

import numpy as np
import pytest
import torch

from tests.pool_cases import half_step
from tests.test_gpu_attend import Case

pytestmark = pytest.mark.gpu

TYPES = [("bf16", "bf16"), ("fp16", "fp16"), ("bf16", "e4m3"), ("fp16", "e4m3")]
# (heads, table columns of 16 tokens): 16, 32 and 64 heads to a workgroup; the
# widest tables of 2-byte rows are read past the caches too
SIZES = [(16, None), (32, 5300), (128, 5300)]
U = 2.0 ** -24


def put(c, s, rows):
    """Stores rows [tokens][width] (what they stand for) as sequence s's cache."""
    n = c.pool.n
    x = (rows / c.cache_scale).to(c.cache)
    assert torch.equal(x.float() * c.cache_scale, rows)
    kind = torch.uint8 if c.cache.itemsize == 1 else c.cache
    stored = c.pool.rows(c.layer, kind)
    x = x.view(kind).cuda()
    for j in range(-(-rows.shape[0] // n)):
        if c.table[s, j] >= 0:
            k = min(n, rows.shape[0] - j * n)
            stored[int(c.table[s, j]), :k] = x[j * n:j * n + k]


def live_tokens(c, s):
    n = c.pool.n
    return [t for t in range(c.lens[s]) if c.table[s, t // n] >= 0]


@pytest.mark.parametrize("dtype,cache", TYPES)
@pytest.mark.parametrize("heads,columns", SIZES)
def test_every_token_counts_once(dtype, cache, heads, columns):
    """All logits of a head are the same, so that P = 1 and the sums are whole
    numbers, which fp32 holds exactly: out is count / live tokens, off by two
    fp32 roundings and the output's one; a token more or less changes a column
    by a twentieth and lse by 1 / tokens."""
    c = Case([9001, 0, 333, 2050, 1], heads=heads, dtype=dtype, cache=cache, seed=1, block_size=16,
             columns=columns, holes=[(0, 0), (0, 7), (0, 100), (0, 101), (0, 562), (2, 20), (3, 1)],
             weights=True)
    c.scale = 1.0
    c.weights.zero_()
    z = torch.arange(heads) % 9 - 4.0
    c.q.zero_()
    c.q[:, :, 575] = z.to(c.dt).cuda()
    for s, n in enumerate(c.lens):
        rows = torch.zeros(n, 576)
        rows[torch.arange(n), torch.arange(n) % 512] = 1.0
        rows[:, 575] = 1.0
        put(c, s, rows)
    c.run()
    h = half_step(c.dt)
    for s in range(len(c.lens)):
        live = live_tokens(c, s)
        want = torch.zeros(512, dtype=torch.float64)
        if live:
            want += torch.bincount(torch.tensor(live) % 512, minlength=512).double() / len(live)
        tol = want * (h + 3 * U) + torch.finfo(c.dt).tiny * h
        out = c.out[s].cpu().double()
        assert (out - want).abs().le(tol).all(), (s, ((out - want).abs() / tol.clamp(min=1e-30)).max())
        # log2 to an ulp or two, its product with ln 2, the sum with the maximum
        lse = torch.full((heads,), -math.inf, dtype=torch.float64)
        off = 0.0
        if live:
            lse = z.double() + math.log(len(live))
            off = 8 * U * (4 + math.log(len(live)))
        got = c.lse[s].cpu().double()
        assert torch.equal(got, lse) if not live else (got - lse).abs().le(off).all(), s
        weights = torch.zeros(c.weights.shape[1], dtype=torch.float64)
        weights[live] = heads / max(1, len(live))
        tol = weights * (off + (heads + 16) * U)  # exp of (z - lse), sums over the heads
        assert (c.weights[s].cpu().double() - weights).abs().le(tol).all(), s


@pytest.mark.parametrize("dtype,cache", TYPES)
@pytest.mark.parametrize("heads,columns", SIZES)
def test_probabilities_keep_sixteen_bits(dtype, cache, heads, columns):
    """Tokens in pairs of nearly the same weight and opposite values: what is
    left of a column is far below the weights, and P rounded once to 8 or 11
    bits would show.  P is off by two roundings to 16 bits (h^2), the logits'
    difference by its rounding and the conversion to powers of two (|z| < 1:
    4 u), exp and the sum by 16 u, the sums over n tokens by n u."""
    lens = [64, 0, 40]
    c = Case(lens, heads=heads, dtype=dtype, cache=cache, seed=2, block_size=16, columns=columns)
    rng = np.random.default_rng(3)
    c.scale = 1.0
    sign = torch.from_numpy(rng.choice([1.0, -1.0, 0.75, -0.75, 0.5, 1.25], heads)).float()
    q = torch.zeros(heads, 576)
    q[:, 572:] = sign.view(-1, 1) * torch.tensor([2.0 ** -4, 2.0 ** -7, 2.0 ** -10, 2.0 ** -13])
    c.q.copy_(q.expand_as(c.q).to(c.dt))
    assert torch.equal(c.q[0].cpu().float(), q)
    h, all_rows = half_step(c.dt), []
    for s, n in enumerate(lens):
        k = rng.integers(0, 8, (n // 2, 1, 4)).repeat(2, 1)
        k[:, 1, 3] = rng.integers(0, 8, n // 2)
        v = rng.choice([1.0, -1.0], (n // 2, 1, 512)).repeat(2, 1)
        v[:, 1] = -v[:, 0]
        rows = torch.zeros(n, 576)
        rows[:, 572:] = torch.from_numpy(k.reshape(n, 4)).float()
        rows[:, :512] = torch.from_numpy(v.reshape(n, 512)).float()
        put(c, s, rows)
        all_rows.append(rows.double())
    c.run()
    worst = 0.0
    for s, n in enumerate(lens):
        if n == 0:
            assert (c.out[s] == 0).all()
            continue
        p = torch.softmax(q.double() @ all_rows[s].t(), 1)
        want = p @ all_rows[s][:, :512]
        rel = 2 * 4 * U + 16 * U + h * h + (n + 4) * U
        tol = h * want.abs() * (1 + 2 * h) + rel + torch.finfo(c.dt).tiny * h
        worst = max(worst, ((c.out[s].cpu().double() - want).abs() / tol).max().item())
    assert worst <= 1.0, worst


@pytest.mark.parametrize("size", [2.0 ** 20, 2.0 ** 45, 2.0 ** 100])
@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_a_large_query_value_that_meets_zeros(size, cache):
    """The others of the head then make the logits, however small beside it."""
    c = Case([70, 300], heads=33, cache=cache, seed=4)
    stored = c.pool.rows(c.layer, torch.uint8 if cache == "e4m3" else torch.bfloat16)
    for s, n in enumerate(c.lens):
        for j in range(-(-n // c.pool.n)):
            stored[int(c.table[s, j]), :min(c.pool.n, n - j * c.pool.n), 570] = 0
    c.q[:, :, 570] = size
    c.run().check()
