"""hkv_kda_prefill in every variant within bounds that a dropped low term would break."""
import pytest
import torch

from tests.prefill_cases import Case
from tests.prefill_exact import check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("new,heads", [([130], 1), ([130], 6), ([130], 33), ([70, 130, 64, 25], 12), ([20], 2), ([5, 9], 3)],
                         ids=["one", "six", "tiles", "batch", "short", "shorts"])
def test_states_of_every_variant(new, heads, dtype):
    """16 and 32 columns a scanning workgroup, and token by token."""
    check(Case(new, heads=heads, dtype=dtype, seed=heads, lead=1, tail=2))


@pytest.mark.parametrize("d", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_states_token_by_token(d, dtype):
    check(Case([70, 11], heads=2, d=d, dtype=dtype, taps=4 if dtype == "fp32" else 3, seed=d))


@pytest.mark.parametrize("decay", [0.0, 0.05, 5.0])
def test_states_by_decay(decay):
    check(Case([200, 190], heads=2, seed=1, decay=decay))


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("heads", [1, 33])
def test_outputs_that_cancel(heads, dtype):
    """With beta 1, without decays, a query that is its token's key reads that token's
    value.  Where the value is zero the output is what all terms before it, up to 64 times
    larger, leave of each other: no rounding of it hides theirs."""
    c = Case([190], heads=heads, dtype=dtype, seed=2, beta=(1.0, 1.0), decay=0.0)
    hd = heads * 128
    c.weight.zero_()
    c.weight[:, -1] = 1.0
    c.x[:, :hd] = c.x[:, hd:2 * hd]
    c.x[::2, 2 * hd:] = 0
    c.x[1::2, 2 * hd:] *= 8
    c.eps = 0.0
    check(c)
    assert (c.out[::2].double().abs().max() < 1e-3 * c.out[1::2].double().abs().max())


def test_rows_of_small_channels():
    """Keys with channels far below the others: their rows of the state are as exact as the
    column's largest allows."""
    c = Case([130], heads=1, seed=3, src=[None])
    size = torch.ones(128, device="cuda")
    size[1::3], size[2::3] = 1e-3, 1e-6
    c.weight[128:256] = (c.weight[128:256].float() * size.unsqueeze(1)).to(c.dt)
    check(c)
    c = Case([130], heads=1, seed=4)
    c.rec()[:, :, 2::3] *= 1e-6   # and of the source's state
    check(c)


@pytest.mark.parametrize("block_size,width", [(16, 4160), (48, 1408), (64, 1088)])
@pytest.mark.parametrize("new", [[100], [70, 33, 130]])
def test_blocks_no_larger_than_a_chunk(block_size, width, new, monkeypatch):
    """Heads of 128, whose pages need wide MLA rows to fit blocks so short."""
    import tests.prefill_cases as cases

    pool = cases.Pool
    monkeypatch.setattr(cases, "Pool", lambda *a, **kw: pool(*a, mla_width=width, **kw))
    c = Case(new, at=[5 * i for i in range(len(new))], heads=1, block_size=block_size, seed=block_size)
    assert c.pool.n == block_size
    c.run()
