"""MLA attention over the pool (hkv_mla_attend) against the definition in 64
bits, at the lengths, widths, types and masks where it can go wrong."""
import math

import numpy as np
import pytest
import torch

import retrieve_store_chunk_amd as hkv
from tests.pool_cases import TYPES, Pool, half_step, stream, tables

pytestmark = pytest.mark.gpu


class Case:
    def __init__(self, lens, heads=16, width=576, values=512, dtype="bf16", cache=None, path=0,
                 seed=0, block_size=0, columns=None, weights=False, holes=(), spread=3.0,
                 blocks=None, share=False):
        self.rng = np.random.default_rng(seed)
        gen = torch.Generator().manual_seed(seed)
        cache = cache or dtype
        self.dt, self.dt_id = TYPES[dtype]
        self.cache, self.cache_id = TYPES[cache]
        probe = Pool(path, 1, block_size, width, self.cache.itemsize)
        need = sum(-(-max(0, x) // probe.n) for x in lens)
        self.pool = pool = Pool(path, blocks or need + 3, block_size, width, self.cache.itemsize)
        self.layer = pool.mla[1]
        # what no sequence owns reads as NaN
        pool.bytes.fill_(0xFF)
        self.lens = list(lens)
        self.table = tables(lens, pool.n, pool.blocks, self.rng, columns)
        if share:  # every sequence starts with the first one's first block
            self.table[:, 0] = self.table[0, 0]
        rows = pool.rows(self.layer, torch.uint8 if self.cache.itemsize == 1 else self.cache)
        self.cache_scale = 1 / 16 if cache == "e4m3" else 1.0
        for s, n in enumerate(lens):
            for j in range(-(-max(0, n) // pool.n)):
                k = min(pool.n, n - j * pool.n) if not share else pool.n
                v = torch.randn(k, width, generator=gen)
                v = (v * 16).to(self.cache).view(torch.uint8) if cache == "e4m3" else v.to(self.cache)
                rows[self.table[s, j], :k] = v.cuda()
        for s, j in holes:
            self.table[s, j] = -1
        n = len(lens)
        self.heads, self.width, self.values = heads, width, values
        self.q = (torch.randn(n, heads, width, generator=gen) * spread).to(self.dt).cuda()
        self.scale = width ** -0.5
        self.out = torch.full((n, heads, values), 7.0, dtype=self.dt, device="cuda")
        self.lse = torch.full((n, heads), 7.0, device="cuda")
        self.cap = self.table.shape[1] * pool.n
        self.weights = (torch.rand(n, self.cap + 5, generator=gen).cuda() if weights else None)
        self.weights_in = None if self.weights is None else self.weights.clone()
        self.d_table = torch.from_numpy(self.table).cuda()
        self.d_lens = torch.tensor(lens, dtype=torch.int32, device="cuda")

    def args(self):
        a = hkv.hkv_mla_attend_args(
            layer=self.layer, n_seqs=len(self.lens), n_heads=self.heads, value_width=self.values,
            dtype=self.dt_id, cache_dtype=self.cache_id, max_blocks=self.table.shape[1],
            scale=self.scale, cache_scale=self.cache_scale, q=self.q.data_ptr(),
            q_seq_stride=self.q.stride(0), q_head_stride=self.q.stride(1),
            block_table=self.d_table.data_ptr(), table_stride=self.d_table.stride(0),
            seq_lens=self.d_lens.data_ptr(), out=self.out.data_ptr(),
            out_seq_stride=self.out.stride(0), out_head_stride=self.out.stride(1),
            lse=self.lse.data_ptr())
        if self.weights is not None:
            a.weights, a.weights_stride = self.weights.data_ptr(), self.weights.stride(0)
        return a

    def workspace(self):
        size = self.pool.layout.mla_attend_workspace(self.args())
        return torch.full((size,), 0xFF, dtype=torch.uint8, device="cuda")

    def run(self):
        ws = self.workspace()
        before = self.pool.bytes.clone()
        self.pool.layout.mla_attend(self.pool.ptr, self.args(), ws.data_ptr(), ws.numel(), stream())
        torch.cuda.synchronize()
        assert torch.equal(before, self.pool.bytes)
        return self

    def check(self):
        """Against the definition in 64 bits.  With u = 2^-24 and A_t the sum of
        |scale q k| of a logit, a logit is off by at most (width + 4) u A_t (a
        product is exact, an fp32 sum of `width` of them and two roundings are
        not): d.  p is then off by 2 d + 16 u relative (its own logit, the sum
        and exp's roundings), is kept as two 16-bit terms (h^2 with h the type's
        half step) and summed in fp32 over n tokens (n u); the output is rounded
        once (h)."""
        u, h = 2.0 ** -24, half_step(self.dt)
        rows = self.pool.rows(self.layer, torch.uint8 if self.cache.itemsize == 1 else self.cache)
        for s, n in enumerate(self.lens):
            keep, parts = [], []
            for j in range(-(-n // self.pool.n)):
                if self.table[s, j] < 0:
                    continue
                hi = min(self.pool.n, n - j * self.pool.n)
                parts.append(rows[int(self.table[s, j]), :hi].cpu().contiguous().view(self.cache).double())
                keep += range(j * self.pool.n, j * self.pool.n + hi)
            out, lse = self.out[s].cpu().double(), self.lse[s].cpu().double()
            if not keep:
                assert (out == 0).all() and (lse == -math.inf).all()
                if self.weights is not None:
                    assert torch.equal(self.weights[s], self.weights_in[s])
                continue
            k = torch.cat(parts) * self.cache_scale
            q = self.q[s].cpu().double()
            z = q @ k.t() * self.scale
            d = ((q.abs() @ k.abs().t()) * self.scale * (self.width + 4) * u).amax(1, keepdim=True)
            ref_lse = torch.logsumexp(z, 1)
            p = torch.exp(z - ref_lse.unsqueeze(1))
            v = k[:, :self.values]
            ref = p @ v
            rel = 2 * d + 16 * u + h * h + (len(keep) + 4) * u
            tol = h * ref.abs() * (1 + 2 * h) + (p @ v.abs()) * rel + torch.finfo(self.dt).tiny
            assert (out - ref).abs().le(tol).all(), (s, ((out - ref).abs() / tol).max())
            tol = d[:, 0] + (len(keep) + 8) * u + ref_lse.abs() * 4 * u
            assert (lse - ref_lse).abs().le(tol).all(), s
            if self.weights is not None:
                got, was = self.weights[s].cpu().double(), self.weights_in[s].cpu().double()
                want = was.clone()
                want[keep] += p.sum(0)
                tol = torch.zeros_like(want)
                tol[keep] = (p * (2 * d + (16 + len(keep)) * u)).sum(0) + self.heads * u * p.sum(0)
                tol += want.abs() * 2 * u
                live = torch.zeros_like(want, dtype=torch.bool)
                live[keep] = True
                assert torch.equal(got[~live], was[~live])
                assert (got - want).abs().le(tol).all(), s
        return self


@pytest.mark.parametrize("heads", [1, 5, 16, 17, 32, 33, 64, 65, 128])
def test_head_counts(heads):
    Case([77, 200], heads=heads, seed=heads, weights=True).run().check()


@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 129, 1000])
def test_lengths(n):
    Case([n], seed=n, path=n % 2).run().check()


@pytest.mark.parametrize("dtype,cache", [("bf16", "bf16"), ("fp16", "fp16"), ("bf16", "e4m3"),
                                         ("fp16", "e4m3")])
@pytest.mark.parametrize("heads", [16, 32, 64])
def test_types(dtype, cache, heads):
    Case([1, 400, 0, 97, 33], heads=heads, dtype=dtype, cache=cache, seed=3, path=1,
         weights=True).run().check()


@pytest.mark.parametrize("dtype,cache", [("bf16", "bf16"), ("fp16", "fp16"), ("bf16", "e4m3"),
                                         ("fp16", "e4m3")])
@pytest.mark.parametrize("heads", [20, 32, 64, 100, 128])
@pytest.mark.parametrize("columns", [2000, 5300])
def test_wide_tables_take_more_heads_to_a_workgroup(dtype, cache, heads, columns):
    Case([1, 400, 0, 97, 33], heads=heads, dtype=dtype, cache=cache, seed=heads, block_size=16,
         columns=columns, weights=True).run().check()


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("heads", [7, 32, 48])
def test_e4m3_tables_of_more_than_the_last_level_cache(dtype, heads):
    Case([1, 400, 0, 97, 1200], heads=heads, dtype=dtype, cache="e4m3", seed=heads, block_size=16,
         columns=6100, holes=[(1, 3), (4, 0)], weights=True).run().check()


@pytest.mark.parametrize("heads", [40, 64, 128])
def test_a_wide_table_of_split_sequences(heads):
    Case([9001, 40, 3000], heads=heads, seed=heads, block_size=944, columns=180,
         holes=[(0, 1), (2, 0)]).run().check()


@pytest.mark.parametrize("dtype,cache", [("bf16", "bf16"), ("fp16", "fp16"), ("bf16", "e4m3"),
                                         ("fp16", "e4m3")])
def test_the_many_beside_one_large_weight(dtype, cache):
    """One token takes nearly all the weight and has the value 0, so the output
    is what the 31 others, e^-L below it, add up to.  Their P is rounded to
    11 bits where it is kept as one term (e4m3 with bf16) and to 16 or more
    otherwise; a logit of L and its difference to the largest are off by 4 L
    2^-24, the sums by 64 2^-24, and the output is rounded once."""
    c = Case([32], heads=16, dtype=dtype, cache=cache, seed=1, block_size=32)
    top = torch.tensor([1.0, 4.0, 8.0, 10.0, 11.0, 12.0, 12.5, 13.0, 13.5, 14.0, 14.5, 15.0, 15.5,
                        16.0, 17.0, 18.0])
    stored = 448.0 if cache == "e4m3" else 28.0
    row = torch.zeros(32, 576)
    row[1:, :512] = stored
    row[0, 575] = 1 / c.cache_scale
    rows = c.pool.rows(c.layer, torch.uint8 if c.cache.itemsize == 1 else c.cache)
    rows[c.table[0, 0], :32] = (row.to(c.cache).view(torch.uint8) if cache == "e4m3"
                                else row.to(c.cache)).cuda()
    c.q.zero_()
    c.q[0, :, 575] = top.to(c.dt).cuda()
    c.scale = 1.0
    c.run()
    p = 31 * torch.exp(-top.double())
    want = (28.0 * p / (1 + p)).view(-1, 1)
    u, h = 2.0 ** -24, half_step(c.dt)
    term = 2.0 ** -11 if (dtype, cache) == ("bf16", "e4m3") else 2.0 ** -16
    tol = want * (h + term + (4 * 18 + 64) * u) * (1 + h) + torch.finfo(c.dt).tiny * h
    assert (c.out[0].cpu().double() - want).abs().le(tol).all()


@pytest.mark.parametrize("width,values", [(32, 16), (32, 32), (64, 48), (96, 96), (160, 128),
                                          (320, 256), (544, 512), (576, 576 - 64), (576, 208)])
@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_widths(width, values, cache):
    Case([50, 130], heads=20, width=width, values=values, cache=cache, seed=width).run().check()


@pytest.mark.parametrize("block_size", [16, 32, 48, 80, 112])
def test_pages_that_end_inside_a_tile(block_size):
    Case([500, 47, 16, 81], block_size=block_size, width=576, seed=block_size, weights=True).run().check()


def test_ragged_batch_with_empty_sequences():
    rng = np.random.default_rng(9)
    lens = [0, 0] + [int(x) for x in rng.integers(0, 300, 40)] + [0, 1, 2000, 0]
    Case(lens, heads=32, seed=5, path=1, weights=True).run().check()


def test_more_sequences_than_threads():
    rng = np.random.default_rng(10)
    Case([int(x) for x in rng.integers(0, 40, 700)], heads=8, width=64, values=64, seed=6).run().check()


def test_one_long_sequence_is_split_and_joined():
    Case([9001], heads=32, seed=7, weights=True, block_size=944).run().check()


def test_null_blocks_are_left_out():
    c = Case([200, 64, 100], block_size=32, heads=16, seed=8, weights=True,
             holes=[(0, 0), (0, 3), (1, 0), (1, 1), (2, 3)])
    c.run().check()  # sequence 1 has nothing left


def test_shared_blocks():
    Case([40, 32, 64], block_size=32, seed=11, share=True).run().check()


def test_strides_and_a_head_major_output():
    c = Case([70, 33, 5], heads=6, seed=12)
    n, h, w = c.q.shape
    q = torch.full((h, n, w + 40), 3.0, dtype=c.dt, device="cuda")
    q[:, :, :w] = c.q.transpose(0, 1)
    c.q = q.transpose(0, 1)[:, :, :w]
    big = torch.full((h, n, 512 + 24), 7.0, dtype=c.dt, device="cuda")
    c.out = big.transpose(0, 1)[:, :, :512]
    c.d_table = torch.cat([c.d_table, c.d_table.new_full((n, 3), 1 << 30)], 1)[:, :c.table.shape[1]]
    c.run().check()
    assert (big[:, :, 512:] == 7.0).all()


def test_a_broadcast_query():
    c = Case([70, 33], heads=6, seed=13)
    c.q = c.q[:1, :1].expand(2, 6, 576)
    c.run().check()


def test_bad_values_on_the_device_are_contained():
    c = Case([100, 90, 64, 50, 40], block_size=32, heads=16, seed=14, weights=True)
    c.table[1, 1] = c.pool.blocks      # first id past the pool
    c.table[2, 0] = -2
    c.d_table = torch.from_numpy(c.table).cuda()
    c.d_lens[3], c.d_lens[4] = -1, c.cap + 1
    c.run()
    for s in (1, 2, 3, 4):
        assert c.out[s].isnan().all() and c.lse[s].isnan().all(), s
    for s in (1, 2):
        assert c.weights[s, :c.lens[s]].isnan().all()
        assert torch.equal(c.weights[s, c.lens[s]:], c.weights_in[s, c.lens[s]:])
    for s in (3, 4):
        assert torch.equal(c.weights[s], c.weights_in[s])
    good = Case([100], block_size=32, heads=16, seed=14, weights=True)
    c.lens, c.heads = c.lens[:1], good.heads
    c.check()


def test_extreme_logits_and_infinite_values():
    c = Case([300], heads=4, seed=15, spread=400.0)  # logits in the thousands
    c.run().check()
    c = Case([64], heads=4, seed=16)
    rows = c.pool.rows(c.layer, torch.bfloat16)
    rows[int(c.table[0, 0]), 3] = math.nan           # a live NaN row reaches every head
    c.run()
    assert c.out.isnan().all() and c.lse.isnan().all()


def test_captured_calls_follow_the_device_arrays():
    c = Case([500, 40, 70], block_size=32, heads=32, seed=17)
    ws = c.workspace()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        c.pool.layout.mla_attend(c.pool.ptr, c.args(), ws.data_ptr(), ws.numel(), stream())
    full = list(c.lens)
    for cut in ([500, 40, 70], [1, 0, 33], [499, 40, 64], [32, 32, 32]):
        c.lens = cut
        c.d_lens.copy_(torch.tensor(cut, dtype=torch.int32))
        c.out.fill_(7.0)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        c.check()
    assert full == [500, 40, 70]


def test_two_streams_at_once():
    a, b = Case([3000, 20], seed=18, heads=32), Case([10, 2500, 7], seed=19, heads=64, cache="e4m3")
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    wa, wb = a.workspace(), b.workspace()
    torch.cuda.synchronize()
    for _ in range(5):
        a.pool.layout.mla_attend(a.pool.ptr, a.args(), wa.data_ptr(), wa.numel(), sa.cuda_stream)
        b.pool.layout.mla_attend(b.pool.ptr, b.args(), wb.data_ptr(), wb.numel(), sb.cuda_stream)
    torch.cuda.synchronize()
    a.check()
    b.check()


def test_the_same_call_gives_the_same_bits():
    c = Case([4000, 100, 0, 900], heads=48, seed=20, weights=True)
    c.run()
    first = (c.out.clone(), c.lse.clone(), c.weights.clone())
    c.weights.copy_(c.weights_in)
    c.run()
    assert all(torch.equal(x, y) for x, y in zip(first, (c.out, c.lse, c.weights)))


def test_rows_behind_four_gigabytes():
    """A page whose byte offset passes 32 bits."""
    c = Case([600], heads=16, seed=21, block_size=30000, path=1, blocks=60)
    assert c.pool.info["pool_bytes_used"] > (1 << 32)
    L = c.pool.layers[c.layer]
    rows = c.pool.rows(c.layer, torch.bfloat16)
    rows[59, :600] = rows[int(c.table[0, 0]), :600]
    rows[int(c.table[0, 0])] = math.nan
    c.table[0, 0] = 59
    c.d_table.fill_(59)
    assert L["pool_offset"] + 59 * L["stride"] > (1 << 32)
    c.run().check()


@pytest.mark.parametrize("size", [1e-30, 1e-4, 1.0, 1e4, 1e20])
def test_query_sizes_with_an_e4m3_cache(size):
    """A bf16 query of any size next to e4m3 rows (the logits' scale undoes it)."""
    c = Case([70, 300], heads=33, cache="e4m3", seed=22)
    c.q = (c.q.float() * size * torch.logspace(-3, 3, 33, base=2.0, device="cuda").view(1, 33, 1)).to(c.dt)
    c.scale = c.scale / size if size < 1e18 else float(np.float32(c.scale / size))
    c.run().check()


def test_an_infinite_query_value_keeps_the_others():
    c = Case([40], heads=3, cache="e4m3", seed=23)
    c.q[0, 1, 5] = math.inf
    c.q[0, 1, 6] = 1e30
    c.run()
    assert c.out[0, 1].isnan().all()                # inf logits of both signs
    assert c.out[0, 0].isfinite().all() and c.out[0, 2].isfinite().all()
