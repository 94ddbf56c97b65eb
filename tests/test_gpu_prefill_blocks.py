"""hkv_kda_prefill's look at the block ids of calls with many blocks, which are counted
instead of compared pair by pair: the same refusals, in time that grows with the blocks."""
import numpy as np
import pytest
import torch

import tests.prefill_cases as cases
from tests.prefill_cases import Case

pytestmark = pytest.mark.gpu

N = 16


@pytest.fixture(params=[16, 128])
def many(request, monkeypatch):
    """Cases with blocks of 16 tokens, of heads that go token by token and in chunks."""
    if request.param == 128:   # wide MLA rows, so that pages so short hold a state
        pool = cases.Pool
        monkeypatch.setattr(cases, "Pool", lambda *a, **kw: pool(*a, mla_width=4160, **kw))

    def make(new, **kw):
        c = Case(new, heads=1, d=request.param, block_size=N, **kw)
        assert c.x.shape[0] // N > 24
        return c

    return make


def test_runs_of_many_blocks(many):
    many([700, 400, 3, 0], at=[5, 0, 31, 7], src=["own", "other", None, "other"], seed=1).run()


def test_one_run_of_many_blocks(many):
    many([1100], null=[(0, 3), (0, 68)], seed=2).run()


def test_clashes(many):
    c = many([300] * 8, seed=3)
    c.table[1, 17] = c.table[0, 0]      # 0 and 1 write one block
    c.src[3] = c.table[2, 18]           # 2 would write what 3 reads; 3 may go on
    c.table[4, 2] = c.table[4, 9]       # twice in its own table
    c.src[6] = c.src[5]                 # one source for two
    c.src[7] = c.table[7, 11]           # its own block
    c.refused = {0, 1, 2, 4}
    c.upload()
    c.run()


def test_bad_ids(many):
    c = many([300] * 6, seed=4)
    c.table[0, 18], c.table[1, 0] = c.pool.blocks, -3
    c.src[2], c.src[3] = -2, c.pool.blocks
    c.src[4] = -1
    c.refused = {0, 1, 2, 3}
    c.upload()
    c.run()


def test_sequences_that_do_not_count(many):
    """Sources and blocks of a sequence without tokens clash with nobody's; those of one
    that is refused do."""
    c = many([500, 0, 300, 300], seed=5)
    c.src[1] = c.table[0, 3]
    c.src[3] = c.pool.blocks            # refused, but it names a block of 2
    c.table[3, 5] = c.table[2, 5]
    c.refused = {2, 3}
    c.upload()
    c.run()


def test_captured_and_replayed(many):
    """Counts start anew with every replay."""
    c = many([600, 600], seed=6)
    before, table = c.pool.bytes.clone(), c.table.copy()
    c.enqueue()
    torch.cuda.synchronize()
    g, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(g, stream=s):
        c.enqueue()
    for refused in (set(), {0, 1}, {1}, set()):
        c.table = table.copy()
        if refused == {0, 1}:
            c.table[0, 30] = c.table[1, 3]
        elif refused:
            c.table[1, 30] = c.table[1, 3]
        c.refused = refused
        c.d_table.copy_(torch.from_numpy(c.table))
        c.pool.bytes.copy_(before)
        c.out.fill_(7.0)
        torch.cuda.synchronize()
        want = c.expect()
        g.replay()
        c.compare(want)


@pytest.mark.parametrize("seqs", [1, 2, 64])
def test_the_longest_tables(seqs):
    """2^20 tokens in blocks of 16 that name the pool's few blocks again and again."""
    c = Case([40], heads=1, d=16, block_size=N, seed=7)
    tokens = 1 << 20
    each, columns = tokens // seqs, tokens // seqs // N
    before = c.pool.bytes.clone()
    c.x = torch.zeros(1, 48, dtype=c.dt, device="cuda").expand(tokens, 48)
    c.log_decay = torch.zeros(1, 16, device="cuda").expand(tokens, 16)
    c.beta = torch.zeros(1, 1, device="cuda").expand(tokens, 1)
    c.out = torch.zeros(tokens, 16, dtype=c.dt, device="cuda")
    c.new, c.at, c.most, c.columns = [each] * seqs, [0] * seqs, each, columns
    c.src = np.full(seqs, -1)
    c.starts = np.arange(seqs + 1) * each
    c.table = (np.arange(seqs * columns) % c.pool.blocks).reshape(seqs, columns)
    c.upload()
    c.enqueue()
    torch.cuda.synchronize()
    assert c.out.isnan().all()
    assert torch.equal(before, c.pool.bytes)
