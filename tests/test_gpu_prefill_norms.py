"""hkv_kda_prefill's norms where the squares' sum is below fp32's normal numbers."""
import pytest

from tests.prefill_cases import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d,dtype", [(16, "bf16"), (64, "fp32"), (128, "bf16"), (256, "fp32")])
@pytest.mark.parametrize("power", [-60, -64, -66])
@pytest.mark.parametrize("tokens", [9, 100])
def test_tiny_queries_and_keys(d, dtype, power, tokens):
    """One channel of q and k of 2^power / 2 (silu of a tiny value is half of it), whose
    square is a power of two, below 2^-126 for some: every step is exact, and q and k are
    unit vectors."""
    c = Case([tokens], heads=1, d=d, dtype=dtype, seed=d - power)
    c.eps = 0.0
    c.weight.zero_()
    c.weight[:, -1] = 1.0
    c.x[:, :2 * d] = 0
    for part in (0, 1):
        c.x[:, part * d + 5] = 2.0 ** power
    c.run()
