"""Long runs that hkv_kda_prefill cuts into parts: the state that each part starts from
is joined from what the parts before it make of any state."""
import numpy as np
import pytest
import torch

from tests.prefill_cases import Case
from tests.prefill_exact import check, follow, state_errors

pytestmark = pytest.mark.gpu

PART = 6 * 64   # the least tokens of a part


def evenly(c, lo, hi, rows=slice(None)):
    """Decays between lo and hi a token, in all channels."""
    c.log_decay[rows] = -(lo + (hi - lo) * torch.rand(c.log_decay[rows].shape, generator=c.gen).cuda())


WEAK = [(0.0, 0.0), (0.0, 0.001), (0.001, 0.001), (0.004, 0.005)]


@pytest.mark.parametrize("lo,hi", [*WEAK, (0.02, 0.06)])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_weak_decays(lo, hi, dtype):
    """A large source state that outlives the parts."""
    c = Case([1500], heads=2, dtype=dtype, seed=1, block_size=320, beta=(0.0, 0.05))
    c.rec().mul_(50.0)
    evenly(c, lo, hi)
    check(c)


def test_more_parts():
    c = Case([3000], heads=1, seed=2, block_size=960)
    c.rec().mul_(50.0)
    evenly(c, 0.0, 0.002)
    check(c)


@pytest.mark.parametrize("decay", [0.01, 0.03, 0.05])
def test_states_that_fade_where_nothing_comes_in(decay):
    """What is left of the source's state behind parts without new values: exactly
    the decays' product times it, a small fraction of it."""
    c = Case([1500], heads=1, seed=3, block_size=320)
    evenly(c, decay, decay)
    c.beta[100:] = 0.0
    c.x[97:, 256:] = 0
    check(c)


def test_one_channel_outlives_the_others():
    """A small row of the state that does not decay beside large ones that do.  A token
    multiplies it by 1, and nothing is added: 2^-23 a token is more than it may lose."""
    c = Case([1500], heads=1, seed=4, block_size=320, beta=(0.0, 0.0))
    c.rec().mul_(100.0)
    c.rec()[:, :, 77].mul_(2.0 ** -22)
    evenly(c, 0.005, 0.005)
    c.log_decay[:, 77] = 0.0
    want = c.rec()[int(c.src[0]), :, 77].double()
    c.enqueue()
    torch.cuda.synchronize()
    for b in c.table[0]:
        assert ((c.rec()[int(b), :, 77].double() - want).abs() <= 1500 * 2.0 ** -23 * want.abs()).all(), b


def test_values_that_jump_between_parts():
    """From 2^-60 to 2^70 where a part ends, and back."""
    c = Case([1500], heads=1, seed=5, block_size=320, decay=3.0)
    for lo, power in ((0, -60), (PART, 70), (2 * PART, -60), (3 * PART, 70)):
        c.x[lo:lo + PART, 256:] = (c.x[lo:lo + PART, 256:].float().abs() * 2.0 ** power).to(c.dt)
    c.run()


@pytest.mark.parametrize("decay", [0.25, 0.5])
def test_states_that_vanish_before_ordinary_tokens(decay):
    """A part behind which the state is near fp32's least numbers, then ordinary ones."""
    c = Case([1500], heads=1, seed=6, block_size=320)
    evenly(c, decay, decay, slice(0, PART))
    c.beta[:PART] = 0.0
    c.run()
    c = Case([1500], heads=1, seed=7, block_size=320)   # nothing but zeros come in
    evenly(c, decay, decay, slice(0, PART))
    c.x[:PART, 256:] = 0
    c.conv().zero_()
    c.run()


def test_parts_of_several_runs():
    c = Case([1300, 1500, 2], at=[0, 100, 3], src=["own", "other", None], heads=2, seed=8, block_size=480,
             beta=(0.0, 0.2))
    evenly(c, 0.0, 0.004)
    check(c)


def test_a_run_in_parts_goes_on_from_its_own_pages():
    """Two calls one after another against one."""
    c = Case([2560], heads=1, seed=9, block_size=320, spare=3)
    evenly(c, 0.0, 0.002)
    before, n = c.pool.bytes.clone(), 4 * 320
    c.enqueue()
    torch.cuda.synchronize()
    ends = [int(c.table[0, 3]), int(c.table[0, 7])]
    want = [c.rec()[b].double() for b in ends]
    c.pool.bytes.copy_(before)
    src = int(c.src[0])
    for at, source in ((0, src), (n, ends[0])):
        c.at, c.src, c.starts, c.new, c.most = [at], np.array([source]), np.array([at, at + n]), [n], n
        c.upload()
        c.enqueue()
    torch.cuda.synchronize()
    for b, w in zip(ends, want):
        # both are within 2^-19 a token of the same state, 2 sqrt(2560) of them
        assert float((c.rec()[b].double() - w).norm() / w.norm()) < 2 * 2560 ** 0.5 * 2.0 ** -19


@pytest.mark.parametrize("lo,hi", WEAK)
def test_the_checks_see_a_wrong_join(lo, hi):
    """A state that is a thousandth off where a part begins, in the definition."""
    c = Case([1500], heads=1, seed=10, block_size=320, beta=(0.0, 0.05))
    c.rec().mul_(50.0)
    evenly(c, lo, hi)
    want, _ = follow(c)
    wrong, _ = follow(c, join=(2 * PART - 1, 1.001))
    wrong_states = {b: w[0] for b, w in wrong.items()}
    for b in c.table[0, 2:]:   # behind it
        assert (state_errors(wrong_states, {int(b): want[int(b)]}) > 1).all(), b
