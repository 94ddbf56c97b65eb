"""hkv_kda_prefill without an eps: q and k over their plain norms."""
import pytest

from tests.prefill_cases import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("tokens", [10, 64, 65, 100, 130])
def test_without_eps(tokens, dtype):
    """Chunks that are full and chunks that are not: a token that a chunk lacks has
    no norm to divide by."""
    c = Case([tokens], heads=2, dtype=dtype, seed=tokens)
    c.eps = 0.0
    c.run()


def test_without_eps_over_block_ends():
    c = Case([400, 33, 70, 1], at=[5, 0, 100, 7], src=["own", None, "other", "own"], heads=2, block_size=160, seed=1)
    c.eps = 0.0
    c.run()


@pytest.mark.parametrize("new", [[1300], [1250, 100, 2]])
def test_without_eps_in_parts(new):
    c = Case(new, heads=1, block_size=480, seed=2)
    c.eps = 0.0
    c.run()


def test_without_eps_in_two_column_tiles():
    c = Case([70, 5, 130, 64], heads=12, seed=3)
    c.eps = 0.0
    c.run()
