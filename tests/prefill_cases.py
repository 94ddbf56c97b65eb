"""Cases of the KDA prefill and what it should leave, token by token in 64 bits."""
import math

import numpy as np
import torch

import retrieve_store_chunk_amd as hkv
from tests.pool_cases import TYPES, Pool, half_step, stream

U = 2.0 ** -24


class Case:
    """Sequences of new[s] tokens from position at[s] on; src[s] is a block, or None
    for a state of zeros, or "own" for the sequence's own first block.  Rows before
    the first sequence (lead) and behind the last (tail) belong to nobody."""

    def __init__(self, new, at=None, src=None, heads=2, d=128, dtype="bf16", taps=4, path=0, seed=0,
                 decay=1.0, lead=0, tail=0, block_size=0, spare=2, null=(), beta=(0.0, 1.0)):
        self.gen = gen = torch.Generator().manual_seed(seed)
        rng = np.random.default_rng(seed)
        self.dt, self.dt_id = TYPES[dtype]
        n_seqs = len(new)
        self.new, self.at = list(new), list(at or [0] * n_seqs)
        src = list(src or ["other"] * n_seqs)
        shape = dict(heads=heads, head_dim=d, conv_bytes=self.dt.itemsize, conv_kernel=taps,
                     block_size=block_size)
        n = Pool(path, 1, **shape).n
        spans = [(p // n, -(-(p + t) // n) if t else p // n) for p, t in zip(self.at, new)]
        blocks = sum(b - a for a, b in spans) + n_seqs + spare
        self.pool = pool = Pool(path, blocks, **shape)
        pool.bytes.copy_(torch.randint(0, 256, pool.bytes.shape, dtype=torch.uint8, generator=gen))
        self.heads, self.d, self.taps, self.layer = heads, d, taps, pool.kda[1]
        self.conv().copy_(torch.randn(self.conv().shape, generator=gen).to(self.dt))
        self.rec().copy_(torch.randn(self.rec().shape, generator=gen) * 0.2)
        ids = list(rng.permutation(blocks).astype(np.int32))
        self.columns = max(1, max(b for _, b in spans))
        self.table = np.full((n_seqs, self.columns), 0x7FFFFFFF, np.int32)
        for s, (a, b) in enumerate(spans):
            for j in range(a, b):
                self.table[s, j] = ids.pop()
        self.src = np.array([-1 if x is None else ids.pop() if x == "other" else
                             self.table[s, spans[s][0]] if x == "own" else x
                             for s, x in enumerate(src)], np.int32)
        for s, j in null:
            self.table[s, j] = -1
        hd, tokens = heads * d, lead + sum(new) + tail
        self.starts = (np.concatenate([[0], np.cumsum(new)]) + lead).astype(np.int32)
        self.most = max([*new, 0])
        self.x = torch.randn(tokens, 3 * hd, generator=gen).to(self.dt).cuda()
        self.weight = (torch.randn(3 * hd, taps, generator=gen) * 0.5).to(self.dt).cuda()
        self.log_decay = (-decay * torch.rand(tokens, hd, generator=gen) ** 3).cuda()
        self.beta = (beta[0] + (beta[1] - beta[0]) * torch.rand(tokens, heads, generator=gen)).cuda()
        for a in (self.x, self.log_decay, self.beta):
            a[:lead], a[lead + sum(new):] = math.nan, math.nan
        self.out = torch.full((tokens, hd), 7.0, dtype=self.dt, device="cuda")
        self.scale, self.eps = d ** -0.5, 1e-6
        self.refused = set()   # NaN in their rows, no page
        self.ignored = set()   # left as they were
        self.workspace = None
        self.upload()

    def upload(self):
        self.d_starts, self.d_at, self.d_src, self.d_table = (
            torch.from_numpy(np.array(v, np.int32)).cuda() for v in (self.starts, self.at, self.src, self.table))

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

    def args(self, **kw):
        a = dict(
            layer=self.layer, n_seqs=len(self.new), n_tokens=self.x.shape[0], max_seq_tokens=self.most,
            max_blocks=self.columns, dtype=self.dt_id, scale=self.scale, eps=self.eps,
            x=self.x.data_ptr(), x_stride=self.x.stride(0), conv_weight=self.weight.data_ptr(),
            log_decay=self.log_decay.data_ptr(), decay_stride=self.log_decay.stride(0),
            beta=self.beta.data_ptr(), beta_stride=self.beta.stride(0),
            seq_starts=self.d_starts.data_ptr(), positions=self.d_at.data_ptr(),
            src_blocks=self.d_src.data_ptr(), block_table=self.d_table.data_ptr(),
            table_stride=self.d_table.stride(0), out=self.out.data_ptr(), out_stride=self.out.stride(0))
        a.update(kw)
        return hkv.hkv_kda_prefill_args(**a)

    def expect(self):
        """By the definition, with a bound on what fp32 may be off.

        Column j of the state follows s_t = M_t s_{t-1} + beta_t v_tj k_t with |M_t| <= 1
        (decays <= 1, |k| <= 1, beta in [0, 2]), so errors that a token brings in do not
        grow: they add up.  A token brings in at most
          4 m u (|s_j| + 2 |v_j|)  for its sums and products: m = taps + d + 16
              roundings (u = 2^-24) bound any sum here relative to its terms' sizes, and
              a product of two-term fp16 operands (off by 2^-21 each, the two low
              terms' product of 2^-22 dropped) stays below 2^-19 <= 4 m u, relative to the norms,
          3 e_k (|s_j| + 2 |v_j|)  for k, off by e_k relative to its norm from the conv,
          2 e_v,j                  for v.
        out = s_j . q is off by |q| times the state's error, and by q's and the sum's own."""
        u, m = U, self.taps + self.d + 16
        conv, rec, x = self.conv().cpu(), self.rec().cpu(), self.x.cpu()
        h, d, n = self.heads, self.d, self.pool.n
        res = dict(out={}, rec={}, conv={})
        wt = self.weight.cpu().double()
        pool = self.pool.bytes.clone()
        out0 = self.out.clone()
        for s, tokens in enumerate(self.new):
            row0 = int(self.starts[s])
            if s in self.ignored or tokens == 0:
                continue
            if s in self.refused:
                for t in range(tokens):
                    res["out"][row0 + t] = None
                continue
            src = int(self.src[s])
            old = conv[src].double() if src >= 0 else torch.zeros(3 * h * d, self.taps - 1, dtype=torch.float64)
            state = rec[src].double() if src >= 0 else torch.zeros(h, d, d, dtype=torch.float64)
            rows = torch.cat([old.t(), x[row0:row0 + tokens].double()])  # [keep + tokens][channels]
            win = rows.unfold(0, self.taps, 1)                              # [tokens][channels][taps]
            terms = win * wt
            y = terms.sum(2)
            ey = ((terms.abs().sum(2) + y.abs() * 0) * 1.2) * m * u
            y = y / (1 + torch.exp(-y))
            ey = (ey + y.abs() * m * u).view(tokens, 3, h, d)
            y = y.view(tokens, 3, h, d)
            norm = torch.sqrt((y ** 2).sum(3) + self.eps)
            rel = torch.sqrt((ey ** 2).sum(3)) / norm + m * u              # [tokens][3][h]
            q, k, v = y[:, 0] / norm[:, 0, :, None] * self.scale, y[:, 1] / norm[:, 1, :, None], y[:, 2]
            g = self.log_decay[row0:row0 + tokens].cpu().double().clamp(max=0).view(tokens, h, d, 1)
            a = torch.exp(g)
            beta = self.beta[row0:row0 + tokens].cpu().double().unsqueeze(2)
            qn = torch.sqrt((q ** 2).sum(2, keepdim=True))
            err = torch.zeros(h, d, dtype=torch.float64)
            for t in range(tokens):
                size = state.norm(dim=1) + 2 * v[t].abs()
                state = a[t] * state
                uu = beta[t] * (v[t] - (k[t].unsqueeze(2) * state).sum(1))
                state = state + k[t].unsqueeze(2) * uu.unsqueeze(1)
                err = err + (4 * m * u + 3 * rel[t, 1].unsqueeze(1)) * size + 2 * ey[t, 2]
                o = (q[t].unsqueeze(2) * state).sum(1)
                eo = qn[t] * (err + (4 * m * u + 3 * rel[t, 0].unsqueeze(1)) * (size + state.norm(dim=1)))
                o, eo = o.reshape(-1), eo.reshape(-1)
                res["out"][row0 + t] = (o, eo + half_step(self.dt) * (o.abs() + eo) + torch.finfo(self.dt).tiny)
                p = self.at[s] + t
                if (p + 1) % n == 0 or t == tokens - 1:
                    b = int(self.table[s, p // n])
                    if b >= 0:
                        res["rec"][b] = state.clone(), err.unsqueeze(1).expand(h, d, d).clone() + state.abs() * u
                        res["conv"][b] = rows[t + 1:t + self.taps].t().to(self.dt)
        return res, pool, out0

    def compare(self, want):
        torch.cuda.synchronize()
        res, before, out0 = want
        for row, w in res["out"].items():
            got = self.out[row].cpu().double()
            if w is None:
                assert got.isnan().all(), row
            else:
                assert (got - w[0]).abs().le(w[1]).all(), (row, ((got - w[0]).abs() / w[1]).max())
        rest = torch.ones(self.out.shape[0], dtype=torch.bool)
        rest[list(res["out"])] = False
        assert torch.equal(self.out.cpu()[rest], out0.cpu()[rest])
        after = self.pool.bytes
        rec, conv = self.rec().clone(), self.conv().clone()
        for b, (state, tol) in res["rec"].items():
            got = rec[b].cpu().double()
            assert (got - state).abs().le(tol).all(), (b, ((got - state).abs() / tol).max())
            assert torch.equal(conv[b].cpu(), res["conv"][b]), b
        self.pool.bytes = before.clone()  # nothing else in the pool changed
        for b in res["rec"]:
            self.rec()[b].copy_(rec[b])
            self.conv()[b].copy_(conv[b])
        assert torch.equal(after, self.pool.bytes)
        self.pool.bytes = after

    def enqueue(self, st=None, **kw):
        a = self.args(**kw)
        size = self.pool.layout.kda_prefill_workspace(a)
        if self.workspace is None or self.workspace.numel() < size:
            self.workspace = torch.full((size,), 0xFF, dtype=torch.uint8, device="cuda")
        self.pool.layout.kda_prefill(self.pool.ptr, a, self.workspace.data_ptr(), self.workspace.numel(),
                                     stream() if st is None else st)

    def run(self, **kw):
        want = self.expect()
        self.enqueue(**kw)
        self.compare(want)
        return self

    def errors(self, want):
        """Norms of the difference over norms, of out and of the states."""
        torch.cuda.synchronize()
        res = want[0]
        o = torch.stack([w[0] for w in res["out"].values()])
        go = self.out.cpu().double()[list(res["out"])]
        s = torch.stack([w[0] for w in res["rec"].values()])
        gs = self.rec().cpu().double()[list(res["rec"])]
        return float((go - o).norm() / o.norm()), float((gs - s).norm() / s.norm())
