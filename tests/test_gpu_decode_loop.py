"""The decode-step operators used together, as an engine on the pool would: a
prefix is retrieved from chunk objects, then every token steps the KDA layers
and attends over the MLA layers (accumulating weights), sequences that outgrow
the budget are evicted, and later tokens append behind what was kept.  Compared
with a plain loop over float64 lists of what each sequence holds."""
import math

import numpy as np
import pytest
import torch

import retrieve_store_chunk_amd as hkv
from tests.pool_cases import Pool, half_step, stream

pytestmark = pytest.mark.gpu

HEADS, WIDTH, VALUES, BUDGET, RECENT = 4, 64, 48, 40, 12
KDA_HEADS, D = 2, 16


class Engine:
    def __init__(self, n=3, steps=30, seed=1):
        self.gen = torch.Generator().manual_seed(seed)
        self.pool = Pool(1, 64, 0, WIDTH, 2, KDA_HEADS, D, is_mla=(0, 1, 0, 1))
        p = self.pool
        assert p.layout.k == 1
        self.n, self.cap_blocks = n, -(-(100 + steps) // p.n)
        ids = torch.randperm(p.blocks, generator=self.gen).int()
        self.table = ids[:n * self.cap_blocks].view(n, self.cap_blocks).contiguous().cuda()
        self.state = ids[n * self.cap_blocks:n * self.cap_blocks + n].contiguous().cuda()
        self.cap = self.cap_blocks * p.n
        k = len(p.mla)
        self.lens = torch.zeros(n, dtype=torch.int32, device="cuda")
        self.next = torch.zeros(n, dtype=torch.int32, device="cuda")
        self.weights = torch.zeros(k, n, self.cap, device="cuda")
        self.positions = torch.full((k, n, self.cap), -1, dtype=torch.int32, device="cuda")
        self.q = torch.zeros(n, HEADS, WIDTH, dtype=torch.bfloat16, device="cuda")
        self.out = torch.zeros(n, HEADS, VALUES, dtype=torch.bfloat16, device="cuda")
        self.new_lens = torch.zeros_like(self.lens)
        self.x = torch.zeros(n, 3 * KDA_HEADS * D, dtype=torch.bfloat16, device="cuda")
        self.kda_out = torch.zeros(n, KDA_HEADS * D, dtype=torch.bfloat16, device="cuda")
        self.conv_w = (torch.randn(3 * KDA_HEADS * D, 4, generator=self.gen) * 0.5).bfloat16().cuda()
        self.decay = torch.zeros(n, KDA_HEADS * D, device="cuda")
        self.beta = torch.zeros(n, KDA_HEADS, device="cuda")
        a = self.attend_args(0)
        e = self.evict_args()
        self.ws_a = torch.empty(p.layout.mla_attend_workspace(a), dtype=torch.uint8, device="cuda")
        self.ws_e = torch.empty(p.layout.mla_evict_workspace(e), dtype=torch.uint8, device="cuda")

    def attend_args(self, i):
        w = self.weights[i]
        return hkv.hkv_mla_attend_args(
            layer=self.pool.mla[i], n_seqs=self.n, n_heads=HEADS, value_width=VALUES,
            dtype=hkv.HKV_BF16, cache_dtype=hkv.HKV_BF16, max_blocks=self.cap_blocks, scale=0.25,
            cache_scale=1.0, q=self.q.data_ptr(), q_seq_stride=HEADS * WIDTH, q_head_stride=WIDTH,
            block_table=self.table.data_ptr(), table_stride=self.cap_blocks,
            seq_lens=self.lens.data_ptr(), out=self.out.data_ptr(),
            out_seq_stride=HEADS * VALUES, out_head_stride=VALUES, weights=w.data_ptr(),
            weights_stride=w.stride(0))

    def evict_args(self):
        e = hkv.hkv_mla_evict_args(
            n_seqs=self.n, max_blocks=self.cap_blocks, budget=BUDGET, sinks=2, recent=RECENT,
            block_table=self.table.data_ptr(), table_stride=self.cap_blocks,
            seq_lens=self.lens.data_ptr(), next_positions=self.next.data_ptr(),
            weights=self.weights.data_ptr(), positions=self.positions.data_ptr(),
            weights_out=self.weights.data_ptr(), positions_out=self.positions.data_ptr(),
            layer_stride=self.weights.stride(0), seq_stride=self.weights.stride(1),
            new_lens=self.new_lens.data_ptr())
        e.set_layers(self.pool.mla)
        return e

    def step_args(self, i):
        return hkv.hkv_kda_step_args(
            layer=self.pool.kda[i], n_seqs=self.n, dtype=hkv.HKV_BF16, scale=0.25, eps=1e-6,
            x=self.x.data_ptr(), x_stride=self.x.stride(0), conv_weight=self.conv_w.data_ptr(),
            log_decay=self.decay.data_ptr(), decay_stride=self.decay.stride(0),
            beta=self.beta.data_ptr(), beta_stride=self.beta.stride(0),
            src_blocks=self.state.data_ptr(), dst_blocks=self.state.data_ptr(),
            out=self.kda_out.data_ptr(), out_stride=self.kda_out.stride(0))

    def rows(self, i):
        return self.pool.rows(self.pool.mla[i], torch.bfloat16)

    def append(self, new):
        """Writes each sequence's new rows [layer][seq][width] at its end."""
        s = torch.arange(self.n, device="cuda")
        at = self.lens.long()
        block = self.table[s, at // self.pool.n].long()
        for i in range(len(self.pool.mla)):
            self.rows(i)[block, at % self.pool.n] = new[i]
            self.weights[i, s, at] = 0.0
            self.positions[i, s, at] = self.next
        self.lens += 1
        self.next += 1

    def rand(self, *shape):
        return torch.randn(*shape, generator=self.gen)


def test_a_run_of_tokens_with_evictions():
    e = Engine()
    p, n, k = e.pool, e.n, len(e.pool.mla)
    # the prefix comes from chunk objects: one block of rows per sequence
    lay = p.layout
    info = lay.info
    objs = [[torch.zeros(max(16, info["obj_bytes"][o]), dtype=torch.uint8, device="cuda")
             for o in range(lay.O)] for _ in range(n)]
    prefix = e.rand(n, k, p.n, WIDTH).bfloat16()
    mla_group = {p.layers[i]["kv_group"] for i in p.mla}.pop()
    mla_obj = p.layers[p.mla[0]]["obj_group"]
    ids = np.full((n, lay.G, lay.k), -1, np.int32)
    for s in range(n):
        objs[s][mla_obj].view(torch.bfloat16)[:] = prefix[s].reshape(-1).cuda()
        ids[s, mla_group, 0] = int(e.table[s, 0])
    ws = torch.empty(lay.workspace_size(n), dtype=torch.uint8, device="cuda")
    lay.retrieve(p.ptr, ids, [o.data_ptr() for x in objs for o in x], ws.data_ptr(), ws.numel(), stream())
    for i in p.kda:  # no cached state: zero pages
        L = p.layers[i]
        for b in e.state.tolist():
            at = L["pool_offset"] + b * L["stride"]
            p.bytes[at:at + L["page_bytes"]] = 0
    e.lens.fill_(p.n)
    e.next.fill_(p.n)
    e.positions[:, :, :p.n] = torch.arange(p.n, dtype=torch.int32, device="cuda")
    # what each (layer, sequence) holds, in slot order: [row, weight, position]
    held = [[[[prefix[s, i, t].double(), 0.0, t] for t in range(p.n)] for s in range(n)] for i in range(k)]
    conv = torch.zeros(2, n, 3 * KDA_HEADS * D, 3, dtype=torch.float64)
    rec = torch.zeros(2, n, KDA_HEADS, D, D, dtype=torch.float64)
    evictions = 0
    for step in range(90):
        # KDA layers
        for i in range(2):
            e.x.copy_(e.rand(*e.x.shape))
            e.decay.copy_(-torch.rand(*e.decay.shape, generator=e.gen))
            e.beta.copy_(torch.rand(*e.beta.shape, generator=e.gen))
            p.layout.kda_step(p.ptr, e.step_args(i), stream())
            taps = torch.cat([conv[i], e.x.cpu().double().unsqueeze(2)], 2)
            conv[i] = taps[:, :, 1:]
            y = (taps * e.conv_w.cpu().double()).sum(2)
            y = (y / (1 + torch.exp(-y))).view(n, 3, KDA_HEADS, D)
            q = y[:, 0] / torch.sqrt((y[:, 0] ** 2).sum(2, keepdim=True) + 1e-6) * 0.25
            kk = y[:, 1] / torch.sqrt((y[:, 1] ** 2).sum(2, keepdim=True) + 1e-6)
            rec[i] *= torch.exp(e.decay.cpu().double()).view(n, KDA_HEADS, D, 1)
            u = e.beta.cpu().double().unsqueeze(2) * (y[:, 2] - (kk.unsqueeze(3) * rec[i]).sum(2))
            rec[i] += kk.unsqueeze(3) * u.unsqueeze(2)
            o = (q.unsqueeze(3) * rec[i]).sum(2).reshape(n, -1)
            # 90 steps of roundings relative to the state's size, then one to bf16
            tol = half_step(torch.bfloat16) * o.abs() * 1.01 + 1e-4
            assert (e.kda_out.cpu().double() - o).abs().le(tol).all(), step
        # MLA layers
        new = e.rand(k, n, WIDTH).bfloat16()
        e.append(new.cuda())
        for i in range(k):
            for s in range(n):
                held[i][s].append([new[i, s].double(), 0.0, p.n + step])
            e.q.copy_(e.rand(*e.q.shape) * 2)
            p.layout.mla_attend(p.ptr, e.attend_args(i), e.ws_a.data_ptr(), e.ws_a.numel(), stream())
            for s in range(n):
                rows = torch.stack([r for r, _, _ in held[i][s]])
                z = e.q[s].cpu().double() @ rows.t() * 0.25
                pr = torch.softmax(z, 1)
                ref = pr @ rows[:, :VALUES]
                tol = half_step(torch.bfloat16) * ref.abs() * 1.01 + (pr @ rows[:, :VALUES].abs()) * 1e-4
                assert (e.out[s].cpu().double() - ref).abs().le(tol).all(), (step, i, s)
                for t, x in enumerate(pr.sum(0).tolist()):
                    held[i][s][t][1] += x
        # evictions: by the device's own sums, so that the choice is the same
        if int(e.lens[0]) > BUDGET + 9:
            before = e.weights.cpu()
            p.layout.mla_evict(p.ptr, e.evict_args(), e.ws_e.data_ptr(), e.ws_e.numel(), stream())
            assert e.new_lens.tolist() == [BUDGET] * n
            nxt = p.n + step + 1
            for i in range(k):
                for s in range(n):
                    cur = held[i][s]
                    got = before[i, s, :len(cur)].double()
                    want = torch.tensor([w for _, w, _ in cur], dtype=torch.float64)
                    assert (got - want).abs().le(want.abs() * 1e-4 + 1e-6).all()
                    safe = [x[2] < 2 or x[2] >= nxt - RECENT for x in cur]
                    order = sorted(range(len(cur)), key=lambda t: (not safe[t], 0.0 if safe[t] else -float(got[t]), t))
                    kept = set(order[:BUDGET])
                    holes = [t for t in range(BUDGET) if t not in kept]
                    fill = [t for t in range(BUDGET, len(cur)) if t in kept]
                    for a, b in zip(holes, fill):
                        cur[a] = cur[b]
                    held[i][s] = cur[:BUDGET]
                    assert e.positions[i, s, :BUDGET].tolist() == [x[2] for x in held[i][s]]
            e.lens.copy_(e.new_lens)
            evictions += 1
    assert evictions >= 5
