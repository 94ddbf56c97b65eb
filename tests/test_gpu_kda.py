"""The KDA layers' step on the pool's state pages (hkv_kda_step) against the
definition in 64 bits."""
import math

import numpy as np
import pytest
import torch

import retrieve_store_chunk_amd as hkv
from tests.pool_cases import TYPES, Pool, half_step, stream

pytestmark = pytest.mark.gpu


class Case:
    def __init__(self, src, dst, heads=2, d=128, dtype="bf16", taps=4, path=0, seed=0, blocks=None,
                 decay=1.0):
        gen = torch.Generator().manual_seed(seed)
        self.dt, self.dt_id = TYPES[dtype]
        blocks = blocks or max([*src, *dst, 0]) + 3
        self.pool = pool = Pool(path, blocks, 0, 576, 2, heads, d, self.dt.itemsize, taps)
        pool.bytes.fill_(0x3C)
        self.heads, self.d, self.taps, self.layer = heads, d, taps, pool.kda[1]
        self.conv().copy_(torch.randn(self.conv().shape, generator=gen).to(self.dt))
        self.rec().copy_(torch.randn(self.rec().shape, generator=gen) * 0.2)
        n, hd = len(src), heads * d
        self.src, self.dst = list(src), list(dst)
        self.x = torch.randn(n, 3 * hd, generator=gen).to(self.dt).cuda()
        self.weight = (torch.randn(3 * hd, taps, generator=gen) * 0.5).to(self.dt).cuda()
        self.log_decay = -decay * torch.rand(n, hd, generator=gen).cuda()
        self.beta = torch.rand(n, heads, generator=gen).cuda()
        self.out = torch.full((n, hd), 7.0, dtype=self.dt, device="cuda")
        self.d_src = torch.tensor(src, dtype=torch.int32, device="cuda")
        self.d_dst = torch.tensor(dst, dtype=torch.int32, device="cuda")
        self.scale, self.eps = d ** -0.5, 1e-6
        self.refused = set()

    def page(self, dtype, shape, offset):
        L, es = self.pool.layers[self.layer], dtype.itemsize
        stride, at = [], 1
        for x in reversed(shape):
            stride.insert(0, at)
            at *= x
        return self.pool.bytes.view(dtype).as_strided(
            (self.pool.blocks, *shape), (L["stride"] // es, *stride), (L["pool_offset"] + offset) // es)

    def conv(self):
        return self.page(self.dt, (3 * self.heads * self.d, self.taps - 1), 0)

    def rec(self):
        conv_bytes = 3 * self.heads * self.d * (self.taps - 1) * self.dt.itemsize
        return self.page(torch.float32, (self.heads, self.d, self.d), conv_bytes)

    def args(self):
        return hkv.hkv_kda_step_args(
            layer=self.layer, n_seqs=len(self.src), dtype=self.dt_id, scale=self.scale, eps=self.eps,
            x=self.x.data_ptr(), x_stride=self.x.stride(0), conv_weight=self.weight.data_ptr(),
            log_decay=self.log_decay.data_ptr(), decay_stride=self.log_decay.stride(0),
            beta=self.beta.data_ptr(), beta_stride=self.beta.stride(0),
            src_blocks=self.d_src.data_ptr(), dst_blocks=self.d_dst.data_ptr(),
            out=self.out.data_ptr(), out_stride=self.out.stride(0))

    def expect(self):
        """By the definition, with how far fp32 may be off.  u = 2^-24, m = taps
        + d + 16 roundings bound every sum below relative to the sum of its
        terms' sizes; the conv's error reaches q, k relative to their norm."""
        u, m = 2.0 ** -24, self.taps + self.d + 16
        conv, rec = self.conv().cpu(), self.rec().cpu()
        pool = self.pool.bytes.clone()
        n, h, d = len(self.src), self.heads, self.d
        res = dict(out=[], out_tol=[], rec={}, tol={}, conv={})
        wt = self.weight.cpu().double()
        for s in range(n):
            taps = conv[self.src[s]] if self.src[s] >= 0 else torch.zeros_like(conv[0])
            taps = torch.cat([taps, self.x[s].cpu().unsqueeze(1)], 1)
            terms = taps.double() * wt
            y = terms.sum(1)
            y = (y / (1 + torch.exp(-y))).view(3, h, d)
            ey = (terms.abs().sum(1).view(3, h, d) * 1.2 + y.abs()) * m * u
            norm = torch.sqrt((y ** 2).sum(2, keepdim=True) + self.eps)
            q, k, v = y[0] / norm[0] * self.scale, y[1] / norm[1], y[2]
            # off by the channel's own error and by the norm's
            rel = torch.sqrt((ey ** 2).sum(2, keepdim=True)) / norm + m * u
            eq = (ey[0] / norm[0] + (y[0] / norm[0]).abs() * rel[0]) * abs(self.scale)
            ek = ey[1] / norm[1] + k.abs() * rel[1]
            state = rec[self.src[s]].double() if self.src[s] >= 0 else torch.zeros(h, d, d, dtype=torch.float64)
            g = self.log_decay[s].cpu().double().view(h, d, 1)
            sp = torch.exp(g) * state
            esp = sp.abs() * 6 * u
            seen = (k.unsqueeze(2) * sp).sum(1)
            eseen = (k.abs().unsqueeze(2) * (esp + m * u * sp.abs()) + ek.unsqueeze(2) * sp.abs()).sum(1)
            beta = self.beta[s].cpu().double().unsqueeze(1)
            uu = beta * (v - seen)
            eu = beta.abs() * (ey[2] + eseen) + uu.abs() * 4 * u
            new = sp + k.unsqueeze(2) * uu.unsqueeze(1)
            enew = (esp + ek.unsqueeze(2) * uu.abs().unsqueeze(1) + k.abs().unsqueeze(2) * eu.unsqueeze(1)
                    + (new.abs() + (k.unsqueeze(2) * uu.unsqueeze(1)).abs()) * 4 * u)
            o = (q.unsqueeze(2) * new).sum(1)
            # out is taken as S'^T q + u (k . q): both parts' sizes count
            size = (q.abs().unsqueeze(2) * sp.abs()).sum(1) + uu.abs() * (k * q).abs().sum(1, keepdim=True)
            eo = ((eq.unsqueeze(2) * new.abs()).sum(1) + (q.abs().unsqueeze(2) * enew).sum(1)
                  + uu.abs() * (ek * q.abs() + eq * k.abs()).sum(1, keepdim=True) + 3 * m * u * size)
            o, eo = o.reshape(-1), eo.reshape(-1)
            if s in self.refused:
                o = torch.full_like(o, math.nan)
            res["out"].append(o)
            res["out_tol"].append(eo + half_step(self.dt) * o.abs() * 1.01 + torch.finfo(self.dt).tiny)
            if s not in self.refused and self.dst[s] >= 0:
                res["rec"][self.dst[s]], res["tol"][self.dst[s]] = new, enew + new.abs() * u
                res["conv"][self.dst[s]] = taps[:, 1:]
        return res, pool

    def compare(self, want):
        torch.cuda.synchronize()
        res, before = want
        for s, (o, tol) in enumerate(zip(res["out"], res["out_tol"])):
            got = self.out[s].cpu().double()
            if s in self.refused:
                assert got.isnan().all(), s
            else:
                assert (got - o).abs().le(tol).all(), (s, ((got - o).abs() / tol).max())
        for b, new in res["rec"].items():
            got = self.rec()[b].cpu().double()
            assert (got - new).abs().le(res["tol"][b]).all(), b
            assert torch.equal(self.conv()[b].cpu(), res["conv"][b])
        # nothing else in the pool changed
        after = self.pool.bytes.clone()
        mine, self.pool.bytes = self.pool.bytes, after
        old_rec, old_conv = {}, {}
        self.pool.bytes = before
        for b in res["rec"]:
            old_rec[b], old_conv[b] = self.rec()[b].clone(), self.conv()[b].clone()
        self.pool.bytes = after
        for b in res["rec"]:
            self.rec()[b].copy_(old_rec[b])
            self.conv()[b].copy_(old_conv[b])
        assert torch.equal(after, before)
        self.pool.bytes = mine

    def enqueue(self, st=None):
        self.pool.layout.kda_step(self.pool.ptr, self.args(), stream() if st is None else st)

    def run(self):
        want = self.expect()
        self.enqueue()
        self.compare(want)
        return self


@pytest.mark.parametrize("d", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_head_dims_and_types(d, dtype):
    Case([3, -1, 0], [1, 2, 0], heads=3, d=d, dtype=dtype, seed=d, path=d // 16 % 2).run()


@pytest.mark.parametrize("taps", [1, 2, 3, 4, 5, 8])
def test_conv_kernels(taps):
    Case([0, 1], [2, 1], heads=2, d=64, taps=taps, seed=taps).run()


@pytest.mark.parametrize("heads", [1, 6, 32])
def test_heads(heads):
    Case([0], [0], heads=heads, d=128, seed=heads, path=1).run()


def test_no_destination_writes_no_page():
    Case([0, -1, 2], [-1, -1, 2], seed=3).run()


def test_one_source_for_several_destinations():
    """A shared prefix's snapshot is continued into blocks of their own."""
    Case([4, 4, 4, -1], [0, 1, 2, 3], seed=4).run()


def test_in_place_steps_follow_each_other():
    c = Case([0, 2, 1], [0, 2, 1], heads=2, d=64, seed=5)
    for i in range(4):
        c.x.copy_(torch.randn(c.x.shape, generator=torch.Generator().manual_seed(i)).to(c.dt))
        c.run()


def test_clashing_destinations_are_refused():
    c = Case([0, 1, 2, 3, -1], [0, 5, 5, 4, 0], seed=6, blocks=8)
    # 0: its block is 4's destination; 1 and 2 share one; 3 is alone; 4 clashes with 0
    c.refused = {0, 1, 2, 4}
    c.run()
    c = Case([0, 0], [0, 1], seed=7)  # 0 would write what 1 reads; 1 may go on
    c.refused = {0}
    c.run()


def test_ids_outside_the_pool_are_refused():
    c = Case([0, 1, 2, 3], [4, 5, 6, 7], seed=8, blocks=9)
    ref = Case([0, 1, 2, 3], [4, 5, 6, 7], seed=8, blocks=9)
    assert torch.equal(c.pool.bytes, ref.pool.bytes)
    c.d_src[0], c.d_dst[1], c.d_src[2], c.d_dst[3] = 9, 9, -2, -3
    c.refused = {0, 1, 2, 3}
    c.run()


def test_extremes():
    Case([0, 1], [0, 1], seed=9, decay=300.0).run()       # states that vanish
    c = Case([0], [1], seed=10)
    c.x.zero_()
    c.conv()[0].zero_()                                    # q = k = v = 0: eps alone
    c.run()
    c = Case([0], [1], heads=2, d=32, seed=11)
    c.rec()[0, 0, 3, 5] = math.inf                         # only column 5 of head 0 sees it
    c.enqueue()
    torch.cuda.synchronize()
    bad = ~c.rec()[1].isfinite()
    assert bad[0, :, 5].all() and bad.sum() == 32
    assert c.out.isfinite().sum() == 63


def test_strides():
    c = Case([0, 1, 2], [0, 1, 2], heads=2, d=32, seed=12)
    hd = 64
    x = torch.full((3, 3 * hd + 5), 9.0, dtype=c.dt, device="cuda")
    x[:, :3 * hd] = c.x
    c.x = x[:, :3 * hd]
    c.log_decay = c.log_decay[:1].expand(3, hd)
    c.beta = torch.cat([c.beta, c.beta], 1)[:, :2]
    out = torch.full((3, hd + 12), 7.0, dtype=c.dt, device="cuda")
    c.out = out[:, :hd]
    c.run()
    assert (out[:, hd:] == 7.0).all()


def test_captured_steps():
    c = Case([0, 1, -1], [3, 4, 5], heads=2, d=128, seed=13)
    g = torch.cuda.CUDAGraph()
    s = torch.cuda.Stream()
    with torch.cuda.graph(g, stream=s):
        c.enqueue()
    for src, dst in (([0, 1, -1], [3, 4, 5]), ([3, 4, 5], [0, 1, 2]), ([-1, -1, 0], [3, -1, 5])):
        c.src, c.dst = src, dst
        c.d_src.copy_(torch.tensor(src, dtype=torch.int32))
        c.d_dst.copy_(torch.tensor(dst, dtype=torch.int32))
        torch.cuda.synchronize()
        want = c.expect()
        g.replay()
        c.compare(want)


def test_two_streams_at_once():
    cs = [Case(list(range(40)), list(range(40)), heads=4, seed=14), Case([0], [1], d=256, seed=15)]
    want = [c.expect() for c in cs]
    ss = [torch.cuda.Stream() for _ in cs]
    torch.cuda.synchronize()
    for c, s in zip(cs, ss):
        c.enqueue(s.cuda_stream)
    for c, w in zip(cs, want):
        c.compare(w)
