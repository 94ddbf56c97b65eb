"""MLA attention (hkv_mla_attend) where the logits are exact, so that what is
left of the error is the probabilities' and the sums': a few non-zero entries
of the queries and keys, small whole numbers times powers of two."""
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
