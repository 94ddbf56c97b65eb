"""Paths of the decode-step operators that only large calls take: weights in
several pieces, and the eviction of rows that many workgroups share, captured,
repeated, in place and on two streams; and calls from several threads."""
import threading

import numpy as np
import pytest
import torch

import retrieve_store_chunk_amd as hkv
from tests import test_gpu_attend as attend
from tests import test_gpu_evict as evict
from tests import test_gpu_kda as kda

pytestmark = pytest.mark.gpu


def test_weights_of_more_tokens_than_one_pass_over_the_grid():
    """700 sequences have 23 workgroups of 64 tokens each: more than 1472 tokens
    take several passes."""
    rng = np.random.default_rng(1)
    lens = [int(x) for x in rng.integers(0, 20, 700)]
    lens[3], lens[77], lens[699], lens[400] = 1473, 3100, 2000, 1472
    attend.Case(lens, heads=8, width=64, values=64, seed=1, block_size=16, weights=True,
                holes=[(77, 100), (699, 92)]).run().check()


def long_case(seed, **kw):
    return evict.Case([20000, 500, 17001, 30000], 9000, sinks=3, recent=700, layers=2, width=16,
                      mla_bytes=1, block_size=1024, seed=seed, **kw)


@pytest.mark.parametrize("weights", ["spread", "ties", "odd"])
def test_long_rows_in_place(weights):
    long_case(2, in_place=True, weights=weights).run()


def test_long_rows_on_one_workspace_again_and_again():
    c = long_case(3, weights="ties")
    ws, pristine = c.workspace(), c.pool.bytes.clone()
    rng = np.random.default_rng(4)
    for lens, budget in (([20000, 500, 17001, 30000], 9000), ([20000, 500, 17001, 30000], 9000),
                         ([9001, 3, 0, 8999], 9000), ([16385, 499, 17000, 29999], 8192)):
        c.lens, c.budget = lens, budget
        c.w = rng.integers(0, 5, c.w.shape).astype(np.float32)
        c.d_w.copy_(torch.from_numpy(c.w))
        c.d_lens.copy_(torch.tensor(lens, dtype=torch.int32))
        c.pool.bytes.copy_(pristine)
        c.w_out.fill_(9.0)
        c.pos_out.fill_(9)
        want = c.expect()
        c.enqueue(ws)
        c.compare(want)


def test_long_rows_captured_and_replayed():
    c = long_case(5)
    pristine, ws = c.pool.bytes.clone(), c.workspace()
    g = torch.cuda.CUDAGraph()
    s = torch.cuda.Stream()
    with torch.cuda.graph(g, stream=s):
        c.enqueue(ws)
    rng = np.random.default_rng(6)
    for lens in ([20000, 500, 17001, 30000], [9001, 499, 0, 16385], [8999, 3, 17001, 29999]):
        c.lens = lens
        c.w = rng.exponential(size=c.w.shape).astype(np.float32)
        c.d_w.copy_(torch.from_numpy(c.w))
        c.d_lens.copy_(torch.tensor(lens, dtype=torch.int32))
        c.pool.bytes.copy_(pristine)
        c.w_out.fill_(9.0)
        c.pos_out.fill_(9)
        torch.cuda.synchronize()
        want = c.expect()
        g.replay()
        c.compare(want)


def test_long_rows_on_two_streams_at_once():
    cs = [long_case(7), long_case(8, in_place=True, weights="ties")]
    ss = [torch.cuda.Stream() for _ in cs]
    want, ws = [c.expect() for c in cs], [c.workspace() for c in cs]
    torch.cuda.synchronize()
    for c, w, s in zip(cs, ws, ss):
        c.enqueue(w, s.cuda_stream)
    for c, x in zip(cs, want):
        c.compare(x)


def test_a_row_of_more_chunks_than_threads():
    """9 million slots are more than 1024 chunks; the ties with the least kept
    weight end in the last hundred of them."""
    n, budget, recent = 9_000_000, 5_900_000, 1000
    c = evict.Case([n], budget, sinks=2, recent=recent, layers=1, width=3, mla_bytes=1, seed=9,
                   block_size=65536, weights="ties")
    assert c.cap > 1024 * 8192
    w, pos = c.w[0, 0, :n], c.pos[0, 0, :n]
    held = (pos < c.sinks) | (pos >= int(c.next[0]) - recent)
    kept = np.zeros(n, bool)
    kept[np.lexsort((np.arange(n), np.where(held, 0.0, -w), ~held))[:budget]] = True
    last_tie = np.flatnonzero(kept & ~held & (w == w[kept & ~held].min())).max()
    assert 8192 * 1024 < last_tie < n
    holes, movers = np.flatnonzero(~kept[:budget]), budget + np.flatnonzero(kept[budget:])
    w_out, pos_out = np.full_like(c.w, 9.0), np.full_like(c.pos, 9)
    w_out[0, 0, :budget], pos_out[0, 0, :budget] = w[:budget], pos[:budget]
    w_out[0, 0, holes], pos_out[0, 0, holes] = w[movers], pos[movers]
    w_out[0, 0, budget:n], pos_out[0, 0, budget:n] = 0.0, -1
    L, pool = c.pool.layers[c.layers[0]], c.pool.bytes.cpu().numpy()

    def at(slots):
        first = (L["pool_offset"] + c.table[0, slots // c.pool.n].astype(np.int64) * L["stride"]
                 + slots % c.pool.n * 3)
        return first[:, None] + np.arange(3)

    after = pool.copy()
    after[at(holes)] = pool[at(movers)]
    ws = c.workspace()
    c.enqueue(ws)
    c.compare((after, w_out, pos_out, np.array([budget], np.int32)))


def test_calls_from_several_threads_on_one_layout():
    """Each thread has its own stream, buffers and workspace; the layout and the
    pool are shared (the KDA steps write blocks of their own)."""
    shared = attend.Case([900, 33, 0, 2100], heads=32, seed=10, block_size=32, weights=True)
    cases = []
    for i in range(4):
        c = attend.Case([900, 33, 0, 2100], heads=32, seed=10, block_size=32, weights=True)
        c.pool = shared.pool
        c.q = (c.q.float() * (1 + i)).to(c.dt)
        cases.append(c)
    steps = [kda.Case([2 * i, -1], [2 * i, 2 * i + 1], heads=4, d=64, seed=11, blocks=8) for i in range(4)]
    for k in steps[1:]:
        k.pool = steps[0].pool
    want = [k.expect() for k in steps]
    evicts = [evict.Case([700, 90], 200, seed=20 + i) for i in range(4)]
    want_evict = [e.expect() for e in evicts]
    ws = [(c.workspace(), e.workspace(), torch.cuda.Stream()) for c, e in zip(cases, evicts)]
    torch.cuda.synchronize()
    failed = []

    def work(i):
        try:
            wa, we, s = ws[i]
            for _ in range(20):
                cases[i].pool.layout.mla_attend(cases[i].pool.ptr, cases[i].args(), wa.data_ptr(),
                                                wa.numel(), s.cuda_stream)
            steps[i].enqueue(s.cuda_stream)
            evicts[i].enqueue(we, s.cuda_stream)
        except Exception as e:  # noqa: BLE001 (reported by the test's thread)
            failed.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failed, failed
    for c in cases:
        grown = c.weights - c.weights_in
        c.weights = None
        c.check()
        for s, n in enumerate(c.lens):  # 20 times a sum of 1 a head
            assert grown[s].double().sum().item() == pytest.approx(20 * 32 * (n > 0), rel=1e-4)
    before = want[0][1]
    for k, (res, _) in zip(steps, want):
        for s in range(2):
            assert (k.out[s].cpu().double() - res["out"][s]).abs().le(res["out_tol"][s]).all()
        for b, new in res["rec"].items():
            assert (k.rec()[b].cpu().double() - new).abs().le(res["tol"][b]).all()
            assert torch.equal(k.conv()[b].cpu(), res["conv"][b])
    assert not torch.equal(before, steps[0].pool.bytes)
    for e, x in zip(evicts, want_evict):
        e.compare(x)


def test_the_kda_step_of_a_layout_with_the_codec():
    """The codec is the objects' form: the pool's pages are the same."""
    a, b = (kda.Case([0, -1, 2], [3, 1, 2], heads=2, d=64, seed=12) for _ in range(2))
    b.pool.layout = hkv.Layout(dict(b.pool.desc, kda_codec=1))
    assert b.pool.layout.info["kda_codec"] == 1 and b.pool.layout.layers[b.layer]["stride"] == \
        a.pool.layers[a.layer]["stride"]
    a.run()
    b.run()
    assert torch.equal(a.out, b.out) and torch.equal(a.pool.bytes, b.pool.bytes)


@pytest.mark.parametrize("dtype,cache", [("bf16", "bf16"), ("bf16", "e4m3")])
@pytest.mark.parametrize("block_size", [16, 48, 768])
def test_sequences_whose_older_blocks_are_all_null(dtype, cache, block_size):
    """Most workers' runs then hold nothing, and a few hold everything."""
    lens = [9001, 4000, 31, 6000]
    holes = [(s, j) for s, n in enumerate(lens) for j in range(2 * -(-n // block_size) // 3)]
    attend.Case(lens, heads=32, dtype=dtype, cache=cache, seed=13, block_size=block_size,
                holes=holes, weights=True).run().check()
