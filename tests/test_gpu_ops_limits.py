"""The decode step's operators at the limits of their calls: the most sequences,
metadata of which one array is updated in place, outputs that may be left out,
and graphs that share a workspace."""
import math

import numpy as np
import pytest
import torch

import retrieve_store_chunk_amd as hkv
from tests import test_gpu_attend as attend
from tests import test_gpu_evict as evict
from tests import test_gpu_kda as kda
from tests.pool_cases import Pool, stream

pytestmark = pytest.mark.gpu


def test_attention_of_the_most_sequences():
    """65535 short sequences over 9 shared blocks.  The roundings are those of
    the attention's other tests: logits of 64 products, sums of 16 tokens."""
    n, width, values = 65535, 64, 16
    gen = torch.Generator().manual_seed(1)
    pool = Pool(0, 10, 16, width, 2)
    assert pool.n == 16
    layer = pool.mla[0]
    rows = pool.rows(layer, torch.bfloat16)
    rows.copy_(torch.randn(rows.shape, generator=gen).bfloat16())
    q = torch.randn(n, 1, width, generator=gen).bfloat16().cuda()
    table = torch.randint(0, 9, (n, 1), generator=gen, dtype=torch.int32).cuda()
    lens = torch.randint(0, 17, (n,), generator=gen, dtype=torch.int32).cuda()
    out = torch.full((n, 1, values), 7.0, dtype=torch.bfloat16, device="cuda")
    weights = torch.rand(n, 16, generator=gen).cuda()
    was = weights.clone()
    a = hkv.hkv_mla_attend_args(
        layer=layer, n_seqs=n, n_heads=1, value_width=values, dtype=hkv.HKV_BF16,
        cache_dtype=hkv.HKV_BF16, max_blocks=1, scale=0.25, cache_scale=1.0, q=q.data_ptr(),
        q_seq_stride=width, q_head_stride=width, block_table=table.data_ptr(), table_stride=1,
        seq_lens=lens.data_ptr(), out=out.data_ptr(), out_seq_stride=values,
        out_head_stride=values, weights=weights.data_ptr(), weights_stride=16)
    ws = torch.full((pool.layout.mla_attend_workspace(a),), 0xFF, dtype=torch.uint8, device="cuda")
    pool.layout.mla_attend(pool.ptr, a, ws.data_ptr(), ws.numel(), stream())
    torch.cuda.synchronize()
    k = rows.cpu().double()[table.cpu().long()[:, 0]]
    live = torch.arange(16) < lens.cpu().view(-1, 1)
    terms = q.cpu().double() * k * 0.25
    z = terms.sum(2)
    d = terms.abs().sum(2).amax(1, keepdim=True) * (width + 4) * 2.0 ** -24
    p = torch.where(live, torch.exp(z - torch.where(live, z, -math.inf).amax(1, keepdim=True)), 0.0)
    p = torch.where(live, p / p.sum(1, keepdim=True).clamp(min=1e-300), 0.0)
    want = (p.unsqueeze(2) * k[:, :, :values]).sum(1)
    size = (p.unsqueeze(2) * k[:, :, :values].abs()).sum(1)
    h, u = 2.0 ** -8, 2.0 ** -24
    rel = 2 * d + 36 * u + h * h
    tol = h * want.abs() * (1 + 2 * h) + size * rel + 2.0 ** -126
    assert (out[:, 0].cpu().double() - want).abs().le(tol).all()
    grown = weights.cpu().double() - was.cpu().double()
    assert torch.equal(weights.cpu()[~live], was.cpu()[~live])
    tol = p * (2 * d + 36 * u) + 2 * u * weights.cpu().double()
    assert (grown - p).abs().le(tol).all()


def test_kda_step_of_the_most_sequences():
    """The same bits as four calls of a quarter each."""
    n = 4096
    ids = np.random.default_rng(2).permutation(2 * n)
    src, dst = ids[:n].tolist(), ids[n:].tolist()
    src[5::7] = [-1] * len(src[5::7])
    c = kda.Case(src, dst, heads=1, d=16, seed=2, blocks=2 * n)
    before = c.pool.bytes.clone()
    c.pool.layout.kda_step(c.pool.ptr, c.args(), stream())
    torch.cuda.synchronize()
    out, after = c.out.clone(), c.pool.bytes.clone()
    assert out.isfinite().all() and not torch.equal(before, after)
    c.pool.bytes.copy_(before)
    c.out.fill_(7.0)
    for at in range(0, n, n // 4):
        a = c.args()
        a.n_seqs = n // 4
        for name, t in (("x", c.x), ("log_decay", c.log_decay), ("beta", c.beta),
                        ("src_blocks", c.d_src), ("dst_blocks", c.d_dst), ("out", c.out)):
            setattr(a, name, t[at:].data_ptr())
        c.pool.layout.kda_step(c.pool.ptr, a, stream())
    torch.cuda.synchronize()
    assert torch.equal(out, c.out) and torch.equal(after, c.pool.bytes)


@pytest.mark.parametrize("n", [200, 20000])
def test_eviction_with_one_array_in_place(n):
    c = evict.Case([n, 50], n // 3, seed=3, weights="ties")
    want, ws = c.expect(), c.workspace()
    c.w_out = c.d_w  # the slots past a sequence's end then keep the input's weights
    w = want[1]
    for s, x in enumerate(c.lens):
        w[:, s, x:] = c.w[:, s, x:]
    c.enqueue(ws)
    c.compare(want)


@pytest.mark.parametrize("n", [200, 20000])
def test_eviction_without_new_lens(n):
    c = evict.Case([n, 50], n // 3, seed=4)
    want, ws, a = c.expect(), c.workspace(), c.args()
    a.new_lens = None
    c.pool.layout.mla_evict(c.pool.ptr, a, ws.data_ptr(), ws.numel(), stream())
    torch.cuda.synchronize()
    assert (c.new_lens == 77).all()
    c.new_lens.copy_(torch.from_numpy(want[3]))
    c.compare(want)


def test_eviction_of_more_layers_and_sequences_than_compute_units():
    evict.Case([90, 130, 0, 47] * 30, 40, layers=3, seed=5, recent=5, sinks=2).run()


def test_graphs_that_share_a_workspace():
    """Attention of two batches and an eviction, captured apart, replayed in turn."""
    a = attend.Case([900, 30], heads=32, seed=6, weights=True)
    b = attend.Case([33, 2100, 0], heads=64, cache="e4m3", seed=7)
    e = evict.Case([700, 64], 300, seed=8)
    size = max(x.workspace().numel() for x in (a, b, e))
    ws = torch.full((size,), 0xFF, dtype=torch.uint8, device="cuda")
    graphs = []
    for call in (lambda: a.pool.layout.mla_attend(a.pool.ptr, a.args(), ws.data_ptr(), size, stream()),
                 lambda: b.pool.layout.mla_attend(b.pool.ptr, b.args(), ws.data_ptr(), size, stream()),
                 lambda: e.enqueue(ws)):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call()
        graphs.append(g)
    want, pristine = e.expect(), e.pool.bytes.clone()
    for _ in range(3):
        a.weights.copy_(a.weights_in)
        a.out.fill_(7.0)
        b.out.fill_(7.0)
        e.w_out.fill_(9.0)
        e.pos_out.fill_(9)
        e.pool.bytes.copy_(pristine)
        torch.cuda.synchronize()
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        a.check()
        b.check()
        e.compare(want)
