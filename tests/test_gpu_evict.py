"""Eviction by accumulated weight (hkv_mla_evict): every byte of the pool and
every weight, position and length against the definition."""
import math

import numpy as np
import pytest
import torch

import retrieve_store_chunk_amd as hkv
from tests.pool_cases import Pool, stream, tables

pytestmark = pytest.mark.gpu


class Case:
    def __init__(self, lens, budget, sinks=0, recent=0, layers=2, path=0, seed=0, block_size=16,
                 width=576, mla_bytes=2, in_place=False, weights="spread", columns=None):
        rng = np.random.default_rng(seed)
        need = sum(-(-x // 16) for x in lens) if block_size == 16 else sum(-(-x // block_size) for x in lens)
        self.pool = pool = Pool(path, need + 2, block_size, width, mla_bytes,
                                is_mla=(0, 1, 1, 0, 1), head_dim=4, conv_dim=4)
        pool.bytes.copy_(torch.from_numpy(rng.integers(0, 256, pool.bytes.numel(), dtype=np.uint8)))
        self.layers = pool.mla[:layers]
        self.lens, self.budget, self.sinks, self.recent = list(lens), budget, sinks, recent
        self.table = tables(lens, pool.n, pool.blocks, rng, columns)
        n, self.cap = len(lens), self.table.shape[1] * pool.n
        shape = (layers, n, self.cap)
        w = rng.exponential(size=shape).astype(np.float32)
        if weights == "ties":
            w = rng.integers(0, 3, shape).astype(np.float32)
        elif weights == "equal":
            w[:] = 1.5
        elif weights == "odd":  # every kind of value a comparison can go wrong on
            w = rng.choice(np.array([0.0, -0.0, 1e-45, -1e-45, math.inf, -math.inf, math.nan, -1.0, 2.0,
                                     3.4e38], np.float32), shape)
        pos = np.sort(rng.permutation(4 * self.cap)[:self.cap]).astype(np.int32)
        pos = np.stack([[rng.permutation(pos) for _ in range(n)] for _ in range(layers)]).astype(np.int32)
        self.w, self.pos = w, pos
        self.next = np.array([max([int(pos[i, s, :x].max(initial=-1)) for i in range(layers)]) + 1
                              for s, x in enumerate(lens)], np.int32)
        self.d_w, self.d_pos = torch.from_numpy(w).cuda(), torch.from_numpy(pos).cuda()
        self.w_out = self.d_w if in_place else torch.full(shape, 9.0, device="cuda")
        self.pos_out = self.d_pos if in_place else torch.full(shape, 9, dtype=torch.int32, device="cuda")
        self.in_place = in_place
        self.d_table = torch.from_numpy(self.table).cuda()
        self.d_lens = torch.tensor(lens, dtype=torch.int32, device="cuda")
        self.d_next = torch.from_numpy(self.next).cuda()
        self.new_lens = torch.full((n,), 77, dtype=torch.int32, device="cuda")
        self.left = set()  # sequences expected to be left as they are

    def args(self):
        a = hkv.hkv_mla_evict_args(
            n_seqs=len(self.lens), max_blocks=self.table.shape[1], budget=self.budget,
            sinks=self.sinks, recent=self.recent, block_table=self.d_table.data_ptr(),
            table_stride=self.d_table.stride(0), seq_lens=self.d_lens.data_ptr(),
            next_positions=self.d_next.data_ptr(), weights=self.d_w.data_ptr(),
            positions=self.d_pos.data_ptr(), weights_out=self.w_out.data_ptr(),
            positions_out=self.pos_out.data_ptr(), layer_stride=self.d_w.stride(0),
            seq_stride=self.d_w.stride(1), new_lens=self.new_lens.data_ptr())
        a.set_layers(self.layers)
        return a

    def workspace(self):
        return torch.full((self.pool.layout.mla_evict_workspace(self.args()),), 0xFF,
                          dtype=torch.uint8, device="cuda")

    def expect(self):
        """(pool, weights, positions, new lengths) by the definition."""
        pool = self.pool.bytes.cpu().numpy().copy()
        old = pool.copy()
        w = self.w.copy() if self.in_place else np.full_like(self.w, 9.0)
        pos = self.pos.copy() if self.in_place else np.full_like(self.pos, 9)
        new = []
        row_bytes = self.pool.desc["mla_width"] * self.pool.desc["mla_bytes"]
        for s, n in enumerate(self.lens):
            if s in self.left or n <= self.budget:
                if 0 <= n <= self.cap:
                    w[:, s, :n], pos[:, s, :n] = self.w[:, s, :n], self.pos[:, s, :n]
                new.append(-1 if s in self.left else n)
                continue
            new.append(self.budget)
            for i, layer in enumerate(self.layers):
                L = self.pool.layers[layer]

                def at(slot):
                    b = int(self.table[s, slot // self.pool.n])
                    return L["pool_offset"] + b * L["stride"] + (slot % self.pool.n) * row_bytes

                def rank(t):
                    if self.pos[i, s, t] < self.sinks or self.pos[i, s, t] >= self.next[s] - self.recent:
                        return (0, 0.0, t)
                    x = float(self.w[i, s, t])
                    return (2, 0.0, t) if math.isnan(x) else (1, -x, t)

                kept = set(sorted(range(n), key=rank)[:self.budget])
                holes = [t for t in range(self.budget) if t not in kept]
                movers = [t for t in range(self.budget, n) if t in kept]
                for t in range(n):
                    if t < self.budget and t in kept:
                        w[i, s, t], pos[i, s, t] = self.w[i, s, t], self.pos[i, s, t]
                    elif t >= self.budget:
                        w[i, s, t], pos[i, s, t] = 0.0, -1
                for to, frm in zip(holes, movers):
                    w[i, s, to], pos[i, s, to] = self.w[i, s, frm], self.pos[i, s, frm]
                    pool[at(to):at(to) + row_bytes] = old[at(frm):at(frm) + row_bytes]
        return pool, w, pos, np.array(new, np.int32)

    def enqueue(self, ws, st=None):
        self.pool.layout.mla_evict(self.pool.ptr, self.args(), ws.data_ptr(), ws.numel(),
                                   stream() if st is None else st)

    def compare(self, want):
        torch.cuda.synchronize()
        pool, w, pos, new = want
        assert np.array_equal(self.new_lens.cpu().numpy(), new)
        assert np.array_equal(self.pos_out.cpu().numpy(), pos)
        assert np.array_equal(self.w_out.cpu().numpy().view(np.uint32), w.view(np.uint32))
        assert np.array_equal(self.pool.bytes.cpu().numpy(), pool)

    def run(self):
        want, ws = self.expect(), self.workspace()
        self.enqueue(ws)
        self.compare(want)
        return self


@pytest.mark.parametrize("n,budget", [(1, 1), (2, 1), (17, 16), (40, 39), (40, 1), (64, 32), (100, 100),
                                      (100, 200), (1000, 300), (5000, 4100), (9000, 4096)])
@pytest.mark.parametrize("in_place", [False, True])
def test_sizes(n, budget, in_place):
    Case([n], budget, seed=n, in_place=in_place, path=n % 2, block_size=48).run()


@pytest.mark.parametrize("weights", ["spread", "ties", "equal", "odd"])
@pytest.mark.parametrize("in_place", [False, True])
def test_values(weights, in_place):
    Case([300, 33, 700, 0, 64], 60, sinks=5, recent=20, layers=3, weights=weights, seed=4,
         in_place=in_place).run()


@pytest.mark.parametrize("sinks,recent", [(0, 0), (50, 0), (0, 50), (25, 25), (1, 3)])
def test_protected_slots(sinks, recent):
    Case([200, 51, 50, 49], 50, sinks=sinks, recent=recent, seed=5).run()


@pytest.mark.parametrize("width,mla_bytes", [(576, 2), (576, 1), (9, 1), (8, 2), (320, 4), (1024, 2), (3, 1)])
@pytest.mark.parametrize("path", [0, 1])
def test_rows_of_any_width(width, mla_bytes, path):
    Case([150, 90], 40, width=width, mla_bytes=mla_bytes, path=path, seed=6, layers=3, recent=4,
         block_size=32).run()


def test_many_short_sequences():
    rng = np.random.default_rng(7)
    Case([int(x) for x in rng.integers(0, 60, 300)], 24, sinks=1, recent=8, seed=7, layers=1).run()


@pytest.mark.parametrize("n,budget,weights", [(40000, 12345, "spread"), (70001, 40000, "ties"),
                                              (66000, 65000, "odd")])
def test_long_sequences(n, budget, weights):
    Case([n, 10, 20000], budget, sinks=4, recent=1000, layers=1, width=16, mla_bytes=1, seed=8,
         block_size=1024, weights=weights).run()


def test_a_repeated_call_finds_its_inputs_unchanged():
    c = Case([300, 200], 64, recent=8, seed=9)
    want, ws = c.expect(), c.workspace()
    for _ in range(3):
        c.w_out.fill_(9.0)
        c.pos_out.fill_(9)
        c.enqueue(ws)
        c.compare(want)


def test_bad_tables_are_left_alone():
    c = Case([100, 100, 100, 100, 100, 100, 100, 100], 40, seed=10, block_size=32)
    c.table[0, 3] = -1                       # a null block
    c.table[1, 0] = c.pool.blocks            # outside the pool
    c.table[2, 1] = -7
    c.table[3, 2] = c.table[4, 0]            # two sequences share a block
    c.table[5, 1] = c.table[5, 0]            # one names a block twice
    c.lens[6] = c.cap + 1
    c.d_table = torch.from_numpy(c.table).cuda()
    c.d_lens = torch.tensor(c.lens, dtype=torch.int32, device="cuda")
    c.left = {0, 1, 2, 3, 4, 5, 6}
    c.run()


def test_ids_past_the_end_do_not_count():
    c = Case([40, 70], 30, seed=11, block_size=32, columns=6)
    c.table[0, 2:] = c.table[1, 0]
    c.table[1, 3:] = -1
    c.d_table = torch.from_numpy(c.table).cuda()
    c.run()


def test_captured_and_replayed():
    c = Case([300, 500, 64], 100, recent=10, seed=12)
    pristine, ws = c.pool.bytes.clone(), c.workspace()
    g = torch.cuda.CUDAGraph()
    s = torch.cuda.Stream()
    with torch.cuda.graph(g, stream=s):
        c.enqueue(ws)
    rng = np.random.default_rng(13)
    for lens in ([300, 500, 64], [101, 0, 64], [300, 99, 7]):
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


def test_two_streams_at_once():
    cs = [Case([3000, 100], 700, seed=14), Case([40, 2500, 9], 31, seed=15, in_place=True)]
    ss = [torch.cuda.Stream() for _ in cs]
    want, ws = [c.expect() for c in cs], [c.workspace() for c in cs]
    torch.cuda.synchronize()
    for c, w, s in zip(cs, ws, ss):
        c.enqueue(w, s.cuda_stream)
    for c, x in zip(cs, want):
        c.compare(x)


def test_strided_metadata():
    c = Case([120, 90], 30, seed=16, layers=2)
    big_w = torch.full((2, 2, c.cap + 13), 5.0, device="cuda").transpose(0, 1)
    big_p = torch.full((2, 2, c.cap + 13), 5, dtype=torch.int32, device="cuda").transpose(0, 1)
    out_w, out_p = torch.full_like(big_w, 9.0), torch.full_like(big_p, 9)
    big_w[:, :, :c.cap], big_p[:, :, :c.cap] = c.d_w, c.d_pos
    c.d_w, c.d_pos = big_w[:, :, :c.cap], big_p[:, :, :c.cap]
    c.w_out, c.pos_out = out_w[:, :, :c.cap], out_p[:, :, :c.cap]
    assert c.w_out.stride() == c.d_w.stride()
    c.run()
    assert (out_w[:, :, c.cap:] == 9.0).all() and (out_p[:, :, c.cap:] == 9).all()


@pytest.mark.parametrize("long_rows", [False, True])
def test_many_blocks_are_counted(long_rows):
    """Tables too large to compare id by id."""
    if long_rows:
        c = Case([16 * 1100 - 3, 5000, 17000], 9000, recent=100, layers=2, width=16, mla_bytes=1, seed=17)
        assert c.table.shape[1] > 1024
    else:
        c = Case([8000] + [1000 + 7 * i for i in range(8)], 900, recent=50, layers=2, width=16, mla_bytes=1,
                 seed=18, columns=512)
        assert c.table.shape[0] * c.table.shape[1] ** 2 > 1 << 20
    c.table[1, 7] = c.table[2, 9]
    c.d_table = torch.from_numpy(c.table).cuda()
    c.left = {1, 2}
    c.run()
    c = Case([16 * 1100 - 3, 5000, 17000], 9000, layers=1, width=16, mla_bytes=1, seed=19)
    c.table[0, 700] = c.pool.blocks
    c.table[1, 3] = -1
    c.d_table = torch.from_numpy(c.table).cuda()
    c.left = {0, 1}
    c.run()


def test_budgets_around_the_chunks_of_long_rows():
    for n, budget in ((20000, 8192), (20000, 8191), (16385, 16384), (30000, 1), (24576, 16384)):
        Case([n], budget, recent=min(budget, 7), layers=1, width=16, mla_bytes=1, seed=n + budget,
             block_size=512, weights="ties").run()
