"""Appending tokens to the paged MLA cache and rotating their queries
(hkv_mla_append) against the definition in 64 bits."""
import math

import numpy as np
import pytest
import torch

import retrieve_store_chunk_amd as hkv
from tests.pool_cases import TYPES, Pool, half_step, stream

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


class Case:
    """old[s] tokens are cached, new[s] come in.  starts: rows before the first
    sequence (lead) and behind the last (tail) belong to nobody."""

    def __init__(self, old, new, heads=2, dtype="bf16", cache=None, width=576, latent=512, rotary=64,
                 halves=False, norm=True, path=0, seed=0, lead=0, tail=0, block_size=0, spare=2,
                 starts=True, scale=None, magnitude=1.0):
        self.gen = gen = torch.Generator().manual_seed(seed)
        rng = np.random.default_rng(seed)
        self.dt, self.dt_id = TYPES[dtype]
        self.cache, self.cache_id = TYPES[cache or dtype]
        es = self.cache.itemsize
        self.old, self.new, self.halves = list(old), list(new), halves
        self.width, self.latent, self.rotary, self.heads = width, latent, rotary, heads
        self.pool = pool = Pool(path, 1, block_size, width, es)
        n = pool.n
        spans = [(o // n, -(-(o + t) // n) if t else o // n) for o, t in zip(old, new)]
        need = sum(b - a for a, b in spans)
        self.pool = pool = Pool(path, need + spare, block_size, width, es)
        pool.bytes.copy_(torch.randint(0, 256, pool.bytes.shape, dtype=torch.uint8, generator=gen))
        self.layer = pool.mla[1]
        self.columns = max(1, max(b for _, b in spans))
        ids = rng.permutation(need + spare).astype(np.int32)
        self.table = np.full((len(old), self.columns), 0x7FFFFFFF, np.int32)
        at = 0
        for s, (a, b) in enumerate(spans):
            self.table[s, a:b] = ids[at:at + b - a]
            at += b - a
        tokens = lead + sum(new) + tail
        self.starts = np.concatenate([[0], np.cumsum(new)]).astype(np.int32) + lead if starts else None
        self.lens = np.add(old, new).astype(np.int32)
        self.positions = np.full(tokens, 1 << 30, np.int32)
        for s in range(len(old)):
            lo = lead + sum(new[:s])
            self.positions[lo:lo + new[s]] = old[s] + 7 * (s % 2) + np.arange(new[s])
        self.n_positions = int(max(np.add(old, new))) + 8
        angle = (torch.rand(self.n_positions, max(1, rotary // 2), generator=gen) * 6.3).double()
        self.cos_sin = torch.cat([angle.cos(), angle.sin()], 1).float().cuda()
        self.kv = (torch.randn(tokens, width, generator=gen) * magnitude).to(self.dt).cuda()
        self.kv[:lead], self.kv[lead + sum(new):] = math.nan, math.nan
        self.norm = (1 + torch.randn(max(8, latent), generator=gen) * 0.2).to(self.dt).cuda() if norm else None
        self.q = torch.randn(tokens, max(1, heads), rotary or 16, generator=gen).to(self.dt).cuda()
        self.q_out = torch.full((tokens, max(1, heads), width), 5.0, dtype=self.dt, device="cuda")
        self.eps, self.scale = 1e-6, scale or (1 / 16 if es == 1 else 1.0)
        self.unstored = set()      # rows that are not written to the pool
        self.unrotated = set()     # rows whose queries are left as they were
        self.nan_rotation = set()  # rows whose position is outside the table
        self.upload()

    def upload(self):
        self.d_table = torch.from_numpy(self.table.copy()).cuda()
        self.d_lens = torch.from_numpy(self.lens.copy()).cuda()
        self.d_starts = None if self.starts is None else torch.from_numpy(self.starts.copy()).cuda()
        self.d_positions = torch.from_numpy(self.positions.copy()).cuda()

    def args(self, **kw):
        q_out = self.q_out[:, :, self.width - self.rotary:]
        a = dict(
            layer=self.layer, n_seqs=len(self.old), n_tokens=self.kv.shape[0], n_heads=self.heads,
            dtype=self.dt_id, cache_dtype=self.cache_id, latent_width=self.latent,
            rotary_dim=self.rotary, rotary_halves=int(self.halves), n_positions=self.n_positions,
            max_blocks=self.columns, eps=self.eps, cache_scale=self.scale, kv=self.kv.data_ptr(),
            kv_stride=self.kv.stride(0), norm_weight=0 if self.norm is None else self.norm.data_ptr(),
            cos_sin=self.cos_sin.data_ptr(), positions=self.d_positions.data_ptr(),
            seq_starts=0 if self.d_starts is None else self.d_starts.data_ptr(),
            seq_lens=self.d_lens.data_ptr(), block_table=self.d_table.data_ptr(),
            table_stride=self.d_table.stride(0), q_in=self.q.data_ptr(),
            q_in_token_stride=self.q.stride(0), q_in_head_stride=self.q.stride(1),
            q_out=q_out.data_ptr(), q_out_token_stride=q_out.stride(0),
            q_out_head_stride=q_out.stride(1))
        a.update(kw)
        return hkv.hkv_mla_append_args(**a)

    def turned(self, x, row):
        """(value, how far fp32 may be off): two products and a sum, each rounded."""
        p = int(self.positions[row])
        if row in self.nan_rotation:
            return torch.full_like(x, math.nan), torch.zeros_like(x)
        cs = self.cos_sin[p].cpu().double()
        c, s = cs[:self.rotary // 2], cs[self.rotary // 2:]
        y, e = torch.empty_like(x), torch.empty_like(x)
        lo, hi = ((slice(0, self.rotary // 2), slice(self.rotary // 2, None)) if self.halves
                  else (slice(0, None, 2), slice(1, None, 2)))
        a, b = x[..., lo], x[..., hi]
        y[..., lo], y[..., hi] = a * c - b * s, a * s + b * c
        e[..., lo], e[..., hi] = [2.1 * U * ((a * m).abs() + (b * w).abs()) for m, w in ((c, s), (s, c))]
        return y, e

    def expect(self):
        """Stored rows with their tolerance by (block, slot), queries by row.  fp32: a
        sum of squares over w columns is off by at most (w + 1) u of itself, its root
        by half that; then six more roundings."""
        rows, queries = {}, {}
        kv, q = self.kv.cpu().double(), self.q.cpu().double()
        w = None if self.norm is None else self.norm.cpu().double()[:self.latent]
        n, lead = self.pool.n, 0 if self.starts is None else int(self.starts[0])
        row = lead
        for s, (old, new) in enumerate(zip(self.old, self.new)):
            for i in range(new):
                c, tol = kv[row].clone(), torch.zeros(self.width, dtype=torch.float64)
                if w is not None and self.latent:
                    part = c[:self.latent]
                    part = part / torch.sqrt((part ** 2).mean() + self.eps) * w
                    c[:self.latent] = part
                    tol[:self.latent] = part.abs() * (self.latent / 2 + 8) * U
                if self.rotary:
                    c[-self.rotary:], tol[-self.rotary:] = self.turned(c[-self.rotary:], row)
                    if self.heads and row not in self.unrotated:
                        y, e = self.turned(q[row], row)
                        queries[row] = y, e + half_step(self.dt) * (y.abs() + e) + torch.finfo(self.dt).tiny
                slot = int(self.lens[s]) - new + i
                if row not in self.unstored and 0 <= slot // n < self.columns:
                    b = int(self.table[s, slot // n])
                    if 0 <= b < self.pool.blocks:
                        rows[b, slot % n] = c / self.scale, tol / self.scale + 2 * U * (c / self.scale).abs()
                row += 1
        return rows, queries, self.pool.bytes.clone(), self.q_out.clone()

    def compare(self, want):
        torch.cuda.synchronize()
        rows, queries, pool, q_out = want
        got = self.pool.rows(self.layer, torch.uint8 if self.cache.itemsize == 1 else self.cache)
        for (b, t), (c, tol) in rows.items():
            g = got[b, t].view(self.cache).float().cpu().double()
            c, tol = c.clone(), tol.clone()
            if self.cache.itemsize == 1:
                c = torch.where(c.isnan(), c, c.clamp(-448, 448))
                # half a step: 2^-4 of the value, of the least normal number below it
                tol = tol * 1.1 + half_step(self.cache) * torch.maximum(c.abs() + tol, torch.tensor(2.0 ** -6))
            else:
                tol = tol * 1.1 + half_step(self.cache) * (c.abs() + tol) + torch.finfo(self.cache).tiny
            assert torch.equal(g.isnan(), c.isnan()), (b, t)
            off = torch.where(c.isnan() | (g == c), 0.0, (g - c).abs())
            assert off.le(tol).all() or off[c.isfinite()].le(tol[c.isfinite()]).all(), (b, t, (off / tol).max())
        for row, (y, tol) in queries.items():
            g = self.q_out[row, :, self.width - self.rotary:].cpu().double()
            assert torch.equal(g.isnan(), y.isnan()), row
            assert (g - y)[~y.isnan()].abs().le(tol[~y.isnan()]).all(), row
        # nothing else changed
        after, self.pool.bytes = self.pool.bytes, pool.clone()
        old = self.pool.rows(self.layer, torch.uint8 if self.cache.itemsize == 1 else self.cache)
        for b, t in rows:
            old[b, t] = got[b, t]
        assert torch.equal(self.pool.bytes, after)
        self.pool.bytes = after
        for row in queries:
            q_out[row, :, self.width - self.rotary:] = self.q_out[row, :, self.width - self.rotary:]
        assert torch.equal(self.q_out.view(torch.int16), q_out.view(torch.int16))

    def enqueue(self, st=None, **kw):
        self.pool.layout.mla_append(self.pool.ptr, self.args(**kw), stream() if st is None else st)

    def run(self, **kw):
        want = self.expect()
        self.enqueue(**kw)
        self.compare(want)
        return self


@pytest.mark.parametrize("halves", [False, True])
@pytest.mark.parametrize("dtype,cache", [("bf16", "bf16"), ("fp16", "fp16"), ("bf16", "e4m3"), ("fp16", "e4m3")])
def test_types(dtype, cache, halves):
    Case([0, 9, 30, 5], [3, 0, 21, 1], dtype=dtype, cache=cache, halves=halves, lead=2, tail=3, seed=1).run()


@pytest.mark.parametrize("width,latent,rotary", [
    (576, 512, 64), (576, 512, 0), (576, 0, 64), (64, 48, 16), (64, 0, 64), (16, 0, 16), (32, 32, 0),
    (1024, 512, 512), (1024, 1008, 16), (528, 264, 32), (592, 8, 80)])
@pytest.mark.parametrize("halves", [False, True])
def test_widths(width, latent, rotary, halves):
    Case([3, 14], [5, 4], width=width, latent=latent, rotary=rotary, halves=halves, heads=3, seed=width + rotary,
         path=width // 16 % 2).run()


@pytest.mark.parametrize("heads", [0, 1, 5, 16, 128])
@pytest.mark.parametrize("halves", [False, True])
def test_heads(heads, halves):
    Case([1, 2, 3], [1, 2, 9], heads=heads, halves=halves, seed=heads).run()


def test_without_a_norm_rows_are_copied():
    Case([5], [20], norm=False, seed=2).run()
    Case([5], [20], norm=False, cache="e4m3", seed=3, magnitude=30).run()


@pytest.mark.parametrize("n", [1, 7, 300])
def test_one_token_each(n):
    """The decode form: no starts."""
    Case([(i * 37) % 90 for i in range(n)], [1] * n, starts=False, seed=n, path=1).run()


@pytest.mark.parametrize("n", [63, 64, 65, 130, 4097])
def test_many_sequences(n):
    """Every row finds its sequence, empty ones between."""
    new = [(i * 7) % 3 for i in range(n)]
    Case([(i * 5) % 40 for i in range(n)], new, width=32, latent=16, rotary=16, heads=1, seed=n, lead=1, tail=70,
         block_size=32).run()


def test_runs_over_blocks():
    """Runs that begin and end inside blocks, at their ends, and cross several."""
    for old in (0, 1, 15, 16, 17):
        Case([old, 31], [50, 1], width=64, latent=32, rotary=32, block_size=16, seed=old).run()


def test_null_and_bad_blocks_are_not_stored():
    c = Case([0, 0, 0], [40, 40, 40], width=64, latent=32, rotary=32, block_size=16, seed=4)
    c.table[0, 1], c.table[1, 0], c.table[2, 2] = -1, c.pool.blocks, -7
    c.upload()
    c.run()


def test_bad_lengths_are_not_stored():
    c = Case([2, 2, 2, 2], [5, 5, 5, 5], width=64, latent=32, rotary=32, block_size=16, seed=5)
    c.lens[0], c.lens[1], c.lens[2] = 4, 17, -3  # shorter than its new tokens, past the table, negative
    c.unstored = set(range(15))
    c.upload()
    c.run()


def test_bad_starts_store_nothing_out_of_place():
    c = Case([2, 2, 2], [5, 6, 7], width=64, latent=32, rotary=32, block_size=16, seed=6, tail=4)
    c.starts[:] = [0, 5, 3, 18]  # the second decreases: rows from 3 on are found in the third
    c.upload()
    before = c.pool.bytes.clone()
    c.enqueue()
    torch.cuda.synchronize()
    rows = c.pool.rows(c.layer, c.dt)
    kept = {(int(c.table[s, 0]), t) for s in range(3) for t in range(16)}
    after, c.pool.bytes = c.pool.bytes, before
    old = c.pool.rows(c.layer, c.dt)
    for b, t in kept:
        old[b, t] = rows[b, t]
    assert torch.equal(after, before)
    c.starts[:] = [-4, 1 << 30, 5, -9]
    c.upload()
    c.enqueue()
    torch.cuda.synchronize()


def test_positions_outside_the_table_give_nan():
    c = Case([2], [5], width=64, latent=32, rotary=32, block_size=16, seed=7)
    c.positions[1], c.positions[3] = c.n_positions, -1
    c.nan_rotation = {1, 3}
    c.upload()
    c.run()


def test_extremes():
    c = Case([0], [6], seed=8)
    c.kv[0] = 0                      # eps alone
    c.kv[1, :512] = 3e38             # squares that overflow: the norm gives zeros
    c.kv[2, 3] = math.nan            # the whole latent part
    c.kv[3, 520] = math.inf          # its pair alone
    c.kv[4] *= 2.0 ** -60
    c.enqueue()
    torch.cuda.synchronize()
    got = c.pool.rows(c.layer, c.dt)[int(c.table[0, 0]), :6].float().cpu()
    assert (got[0, :512] == 0).all() and (got[1, :512] == 0).all()
    assert got[2, :512].isnan().all() and got[2, 512:].isfinite().all()
    assert got[3, :512].isfinite().all() and not got[3, 520:522].isfinite().any()
    assert got[3, 522:].isfinite().all() and got[3, 512:520].isfinite().all()
    assert got[4, :512].abs().max() < 2.0 ** -40
    c = Case([0], [3], cache="e4m3", norm=False, rotary=0, latent=0, seed=9, scale=0.5)
    c.kv[0, 0], c.kv[0, 1], c.kv[0, 2], c.kv[0, 3], c.kv[0, 4] = 1e4, -1e4, math.nan, math.inf, -math.inf
    c.enqueue()
    torch.cuda.synchronize()
    got = c.pool.rows(c.layer, torch.uint8)[int(c.table[0, 0]), 0].view(torch.float8_e4m3fn).float().cpu()
    assert got[0] == 448 and got[1] == -448 and got[2].isnan() and got[3] == 448 and got[4] == -448


def test_e4m3_rounds_to_nearest_even():
    """Every e4m3 value and every midpoint between two of them."""
    vals = torch.arange(0, 0x7F, dtype=torch.uint8).view(torch.float8_e4m3fn).float()
    mids = (vals[1:] + vals[:-1]) / 2
    x = torch.cat([vals, mids, -vals, -mids])
    pad = 576 - x.numel() % 576
    x = torch.cat([x, torch.zeros(pad)]).view(-1, 576)
    c = Case([0], [x.shape[0]], dtype="fp16", cache="e4m3", norm=False, rotary=0, latent=0, seed=10, scale=1.0)
    c.kv.copy_(x.half())
    assert torch.equal(c.kv.float().cpu(), x)
    c.enqueue()
    torch.cuda.synchronize()
    got = c.pool.rows(c.layer, torch.uint8)[int(c.table[0, 0]), :x.shape[0]].cpu()
    assert torch.equal(got, x.to(torch.float8_e4m3fn).view(torch.uint8))


def test_queries_in_place():
    for halves in (False, True):
        c = Case([4, 4], [9, 2], heads=3, halves=halves, seed=11)
        src = c.q.clone()
        c.q_out[:, :, 512:] = src
        c.q = c.q_out[:, :, 512:]
        want = c.expect()
        c.enqueue()
        c.compare(want)


def test_strides():
    c = Case([4, 4], [9, 2], heads=3, seed=12)
    kv = torch.full((11, 600), 3.0, dtype=c.dt, device="cuda")
    kv[:, 8:584] = c.kv
    c.kv = kv[:, 8:584]
    q = torch.zeros(3, 11, 200, dtype=c.dt, device="cuda")  # heads outermost
    q[:, :, 128:192] = c.q.transpose(0, 1)
    c.q = q[:, :, 128:192].transpose(0, 1)
    table = torch.full((2, 7), 0x7FFFFFFF, dtype=torch.int32, device="cuda")
    table[:, :c.columns] = c.d_table
    c.d_table = table
    c.run()
    # one kv row for all tokens
    c = Case([4, 4], [9, 2], heads=1, seed=13)
    c.kv = c.kv[:1].expand(11, 576)
    c.run()


def test_the_largest_row():
    """Blocks past 2^32 bytes of the pool."""
    free, _ = torch.cuda.mem_get_info()
    if free < 12 << 30:
        pytest.skip("needs 12 GiB")
    pool = Pool(1, 1, 1888, is_mla=(0, 1, 0, 1, 1))
    blocks = (5 << 30) // pool.info["block_stride"]
    c = Case([5], [4], seed=14, block_size=1888, path=1)
    big = Pool(1, blocks, 1888, is_mla=(0, 1, 0, 1, 1))
    c.pool = big
    c.table[0, 0] = blocks - 1
    c.upload()
    assert (blocks - 1) * big.info["block_stride"] > 1 << 32
    want = c.expect()
    c.enqueue()
    c.compare(want)


def test_captured_and_replayed():
    c = Case([0, 3, 9], [4, 1, 6], heads=4, seed=15, tail=5, block_size=32)
    g, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(g, stream=s):
        c.enqueue()
    for k, new in enumerate(([4, 1, 6], [1, 8, 2], [0, 0, 16], [1, 1, 1])):
        c.old, c.new = [5, 2, 8], new
        c.starts = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        c.lens = np.add(c.old, new).astype(np.int32)
        for t, v in ((c.d_starts, c.starts), (c.d_lens, c.lens)):
            t.copy_(torch.from_numpy(v))
        c.positions[:] = (np.arange(c.kv.shape[0]) * 5 + k) % c.n_positions
        c.d_positions.copy_(torch.from_numpy(c.positions))
        c.kv.copy_(torch.randn(c.kv.shape, generator=c.gen).to(c.dt))
        torch.cuda.synchronize()
        want = c.expect()
        g.replay()
        c.compare(want)


def test_two_streams_at_once():
    cs = [Case([0] * 20, [40] * 20, heads=8, seed=16), Case([3], [90], cache="e4m3", halves=True, seed=17)]
    want = [c.expect() for c in cs]
    ss = [torch.cuda.Stream() for _ in cs]
    torch.cuda.synchronize()
    for c, s in zip(cs, ss):
        c.enqueue(s.cuda_stream)
    for c, w in zip(cs, want):
        c.compare(w)
