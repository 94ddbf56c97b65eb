"""A whole decode step (KDA layers, attention, eviction) captured into one HIP
graph and replayed, with lengths, positions, block tables and state blocks
updated on the device between the replays; and the pages that such steps leave,
stored into chunk objects and retrieved into another pool."""
import numpy as np
import pytest
import torch

from tests.pool_cases import half_step, stream
from tests.test_gpu_decode_loop import BUDGET, HEADS, KDA_HEADS, VALUES, D, Engine

pytestmark = pytest.mark.gpu


class Steps(Engine):
    """An engine whose step is one call sequence over fixed buffers."""

    def __init__(self, **kw):
        super().__init__(**kw)
        p, n = self.pool, self.n
        k = len(p.mla)
        self.outs = torch.zeros(k, n, HEADS, VALUES, dtype=torch.bfloat16, device="cuda")
        self.kda_outs = torch.zeros(len(p.kda), n, KDA_HEADS * D, dtype=torch.bfloat16, device="cuda")
        used = set(self.table.flatten().tolist()) | set(self.state.tolist())
        self.free = [b for b in range(p.blocks) if b not in used]
        self.next_state = self.state.clone()

    def start(self, lens, rows):
        """Sequences that hold rows [layer][seq][token][width] already."""
        for s, n in enumerate(lens):
            for t in range(n):
                block = int(self.table[s, t // self.pool.n])
                for i in range(len(self.pool.mla)):
                    self.rows(i)[block, t % self.pool.n] = rows[i, s, t].cuda()
        self.lens.copy_(torch.tensor(lens, dtype=torch.int32))
        self.next.copy_(self.lens)
        self.positions[:] = torch.arange(self.cap, dtype=torch.int32, device="cuda")

    def step(self):
        """What a step enqueues; nothing but the library's calls."""
        lay, ptr, st = self.pool.layout, self.pool.ptr, stream()
        for i in range(len(self.pool.kda)):
            a = self.step_args(i)
            a.dst_blocks, a.out = self.next_state.data_ptr(), self.kda_outs[i].data_ptr()
            lay.kda_step(ptr, a, st)
        for i in range(len(self.pool.mla)):
            a = self.attend_args(i)
            a.out = self.outs[i].data_ptr()
            lay.mla_attend(ptr, a, self.ws_a.data_ptr(), self.ws_a.numel(), st)
        lay.mla_evict(ptr, self.evict_args(), self.ws_e.data_ptr(), self.ws_e.numel(), st)

    def feed(self, x):
        """The next token's inputs, its rows appended."""
        self.x.copy_(x["x"])
        self.decay.copy_(x["decay"])
        self.beta.copy_(x["beta"])
        self.q.copy_(x["q"])
        self.append(x["new"].cuda())

    def finish(self):
        self.lens.copy_(self.new_lens)
        self.state.copy_(self.next_state)

    def move_block(self, s, j):
        """Gives entry j of sequence s another block."""
        old, new = int(self.table[s, j]), self.free.pop(0)
        for i in range(len(self.pool.mla)):
            self.rows(i)[new] = self.rows(i)[old]
            self.rows(i)[old] = 9.0
        self.table[s, j] = new
        self.free.append(old)

    def new_state_block(self, s):
        """The next step leaves the old state as a snapshot."""
        self.next_state[s] = self.free.pop(0)

    def all(self):
        return dict(pool=self.pool.bytes, outs=self.outs, kda=self.kda_outs, weights=self.weights,
                    positions=self.positions, new_lens=self.new_lens)


def inputs(e, seed):
    gen = torch.Generator().manual_seed(seed)
    n, k = e.n, len(e.pool.mla)
    return dict(x=torch.randn(e.x.shape, generator=gen), decay=-torch.rand(e.decay.shape, generator=gen),
                beta=torch.rand(e.beta.shape, generator=gen),
                q=torch.randn(e.q.shape, generator=gen) * 2,
                new=torch.randn(k, n, e.q.shape[2], generator=gen).bfloat16())


def attention_by_definition(e):
    """[layer][seq] outputs in 64 bits, and how far bf16's rounding and fp32 sums
    may be off, from the rows that the pool holds now."""
    for i in range(len(e.pool.mla)):
        rows = e.rows(i).cpu().double()
        for s, n in enumerate(e.lens.tolist()):
            at = torch.arange(n)
            held = rows[e.table[s].cpu().long()[at // e.pool.n], at % e.pool.n]
            p = torch.softmax(e.q[s].cpu().double() @ held.t() * 0.25, 1)
            ref = p @ held[:, :VALUES]
            # logits of 64 products are off by 68 u of their terms' sizes, below 1e-5 here
            yield i, s, ref, half_step(torch.bfloat16) * ref.abs() * 1.01 + (p @ held[:, :VALUES].abs()) * 1e-4


def test_a_captured_step_follows_the_device_between_replays():
    lens = [3, 30, BUDGET - 1]
    graph_side, eager = Steps(seed=5), Steps(seed=5)
    gen = torch.Generator().manual_seed(6)
    rows = torch.randn(2, 3, BUDGET, eager.q.shape[2], generator=gen).bfloat16()
    for e in (graph_side, eager):
        e.start(lens, rows)
    g = torch.cuda.CUDAGraph()
    s = torch.cuda.Stream()
    with torch.cuda.graph(g, stream=s):
        graph_side.step()
    evicted = moved = 0
    for step in range(30):
        x = inputs(eager, 100 + step)
        for e in (graph_side, eager):
            e.feed(x)
            if step % 7 == 3:
                e.move_block(step % 3, 0)
                e.new_state_block((step + 1) % 3)
                moved += 1
        want = list(attention_by_definition(eager))
        torch.cuda.synchronize()
        eager.step()
        g.replay()
        torch.cuda.synchronize()
        for (name, a), b in zip(graph_side.all().items(), eager.all().values()):
            assert torch.equal(a, b), (step, name)
        for i, q, ref, tol in want:
            assert (graph_side.outs[i, q].cpu().double() - ref).abs().le(tol).all(), (step, i, q)
        evicted += int((graph_side.lens > BUDGET).sum())
        assert graph_side.new_lens.tolist() == [min(n, BUDGET) for n in graph_side.lens.tolist()]
        for e in (graph_side, eager):
            e.finish()
    assert evicted >= 30 and moved >= 6


def test_pages_that_steps_left_survive_store_and_retrieve():
    a, b = Steps(seed=7), Steps(seed=8)
    gen = torch.Generator().manual_seed(9)
    a.start([10, 35, BUDGET], torch.randn(2, 3, BUDGET, a.q.shape[2], generator=gen).bfloat16())
    for step in range(12):
        a.feed(inputs(a, 200 + step))
        a.step()
        a.finish()
    lay = a.pool.layout
    info, n = lay.info, a.pool.n
    lens = a.lens.tolist()
    assert lens == [22, BUDGET, BUDGET] and lay.k == 1
    group = {bool(L["is_mla"]): L["kv_group"] for L in a.pool.layers}
    # one chunk a block; the sequence's state goes with its last
    chunks = [(s, j) for s in range(3) for j in range(-(-lens[s] // n))]
    tokens = np.array([min(n, lens[s] - j * n) for s, j in chunks], np.int32)
    objs = [[torch.full((max(16, info["obj_bytes"][o]),), 0xA5, dtype=torch.uint8, device="cuda")
             for o in range(lay.O)] for _ in chunks]
    ptrs = [o.data_ptr() for x in objs for o in x]

    def ids(e):
        t = np.full((len(chunks), lay.G, 1), -1, np.int32)
        for c, (s, j) in enumerate(chunks):
            t[c, group[True], 0] = int(e.table[s, j])
            if (j + 1) * n >= lens[s]:
                t[c, group[False], 0] = int(e.state[s])
        return t

    ws = torch.empty(lay.workspace_size(len(chunks)), dtype=torch.uint8, device="cuda")
    lay.store(a.pool.ptr, ids(a), ptrs, ws.data_ptr(), ws.numel(), stream(), chunk_tokens=tokens)
    b.pool.bytes.fill_(0x55)
    assert not np.array_equal(ids(a), ids(b))
    b.pool.layout.retrieve(b.pool.ptr, ids(b), ptrs, ws.data_ptr(), ws.numel(), stream(),
                           chunk_tokens=tokens)
    for name in ("lens", "next", "weights", "positions", "conv_w"):
        getattr(b, name).copy_(getattr(a, name))
    for step in range(3):
        x = inputs(a, 300 + step)
        for e in (a, b):
            e.feed(x)
            e.step()
            e.finish()
        torch.cuda.synchronize()
        assert a.outs.isfinite().all() and a.kda_outs.isfinite().all()
        for name in ("outs", "kda_outs", "weights", "positions", "new_lens"):
            assert torch.equal(getattr(a, name), getattr(b, name)), (step, name)
        for i in range(2):
            for s, m in enumerate(a.lens.tolist()):
                at = torch.arange(m, device="cuda")
                x, y = (e.rows(i)[e.table[s].long()[at // n], at % n] for e in (a, b))
                assert torch.equal(x, y), (step, i, s)
