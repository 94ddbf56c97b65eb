"""A prompt over a retrieved prefix, then decode steps, as a serving loop runs them:
chunks are retrieved, the rest of the prompt goes through hkv_mla_append and
hkv_kda_prefill, its tokens attend, decode steps go on from the pages, and the blocks
are stored.  Against a loop in 64 bits."""
import numpy as np
import pytest
import torch

import retrieve_store_chunk_amd as hkv
from tests.pool_cases import Pool, stream

pytestmark = pytest.mark.gpu

HEADS, D, Q_HEADS, WIDTH, LATENT, ROTARY = 2, 128, 5, 576, 512, 64


class Model:
    """One KDA and one MLA layer's worth of inputs for every token of a request."""

    def __init__(self, tokens, seed):
        gen = torch.Generator().manual_seed(seed)
        hd = HEADS * D
        bf = torch.bfloat16
        self.x = torch.randn(tokens, 3 * hd, generator=gen).to(bf)
        self.log_decay = -torch.rand(tokens, hd, generator=gen) ** 3
        self.beta = torch.rand(tokens, HEADS, generator=gen)
        self.kv = torch.randn(tokens, WIDTH, generator=gen).to(bf)
        self.q = torch.randn(tokens, Q_HEADS, WIDTH, generator=gen).to(bf)


def reference(m, weight, norm, cos_sin, states):
    """Token by token in 64 bits: KDA outputs, states behind each token that `states`
    names, cached rows, attention outputs."""
    n, hd = m.x.shape[0], HEADS * D
    x = torch.cat([torch.zeros(3, 3 * hd), m.x.float()]).double()
    y = (x.unfold(0, 4, 1) * weight.double()).sum(2)
    y = (y / (1 + torch.exp(-y))).view(n, 3, HEADS, D)
    q, k = (y[:, j] / torch.sqrt((y[:, j] ** 2).sum(2, keepdim=True) + 1e-6) for j in (0, 1))
    s, out, kept = torch.zeros(HEADS, D, D, dtype=torch.float64), [], {}
    for t in range(n):
        s = torch.exp(m.log_decay[t].double()).view(HEADS, D, 1) * s
        u = m.beta[t].double().unsqueeze(1) * (y[t, 2] - (k[t].unsqueeze(2) * s).sum(1))
        s = s + k[t].unsqueeze(2) * u.unsqueeze(1)
        out.append((q[t].unsqueeze(2) * s).sum(1).reshape(-1) * D ** -0.5)
        if t + 1 in states:
            kept[t + 1] = s.clone(), x[t + 1:t + 4].t()
    c = m.kv.double()
    c[:, :LATENT] *= norm.double() / torch.sqrt((c[:, :LATENT] ** 2).mean(1, keepdim=True) + 1e-6)
    turn = torch.complex(cos_sin[:n, :ROTARY // 2].double(), cos_sin[:n, ROTARY // 2:].double())

    def rotated(v, by):
        z = torch.view_as_complex(v.double().reshape(*v.shape[:-1], -1, 2).contiguous()) * by
        return torch.view_as_real(z).flatten(-2)

    c[:, LATENT:] = rotated(m.kv[:, LATENT:], turn)
    rows = c.to(torch.bfloat16).double()
    qr = torch.cat([m.q[:, :, :LATENT].double(), rotated(m.q[:, :, LATENT:], turn.unsqueeze(1)).to(torch.bfloat16).double()], 2)
    attn = []
    for t in range(n):
        z = qr[t] @ rows[:t + 1].t() * WIDTH ** -0.5
        attn.append(torch.softmax(z, 1) @ rows[:t + 1, :LATENT])
    return torch.stack(out), kept, rows, torch.stack(attn)


@pytest.mark.parametrize("path", [0, 1])
def test_prompt_after_a_retrieve_then_decode(path):
    pool = Pool(path, 24, 0, WIDTH, 2, HEADS, D)
    lay, n = pool.layout, pool.n
    mla, kda = pool.mla[0], pool.kda[0]
    gen = torch.Generator().manual_seed(7)
    weight = (torch.randn(3 * HEADS * D, 4, generator=gen) * 0.5).to(torch.bfloat16)
    norm = (1 + 0.2 * torch.randn(LATENT, generator=gen)).to(torch.bfloat16)
    prefix, prompt, steps = n, [n + 37, 20], 3     # the first prompt ends a block
    angle = torch.arange(prefix + max(prompt) + steps).double().unsqueeze(1) * \
        10000.0 ** (-torch.arange(0, ROTARY, 2).double() / ROTARY)
    cos_sin = torch.cat([angle.cos(), angle.sin()], 1).float().cuda()
    models = [Model(prefix + p + steps, 100 + i) for i, p in enumerate(prompt)]
    for m in models[1:]:                           # both share the prefix
        for name in ("x", "log_decay", "beta", "kv", "q"):
            getattr(m, name)[:prefix] = getattr(models[0], name)[:prefix]
    ends = [[prefix, *range(2 * n, prefix + p + 1, n), prefix + p, prefix + p + steps] for p in prompt]
    want = [reference(m, weight, norm, cos_sin.cpu(), e) for m, e in zip(models, ends)]
    dev = dict(weight=weight.cuda(), norm=norm.cuda())
    seqs, hd = len(prompt), HEADS * D
    ids = np.random.default_rng(path).permutation(24).astype(np.int32)
    columns = max(-(-(prefix + p + steps) // n) for p in prompt)
    mla_table = ids[:seqs * columns].reshape(seqs, columns)
    kda_table = ids[seqs * columns:2 * seqs * columns].reshape(seqs, columns)
    spare = ids[2 * seqs * columns:]

    def cuda(v):
        return torch.from_numpy(np.ascontiguousarray(v, np.int32)).cuda()

    def run(old, new, rows, kda_src):
        """New tokens of every sequence: appended, through the KDA layer, attended."""
        take = lambda name: torch.cat([getattr(m, name)[o:o + t] for m, o, t in zip(models, old, new)]).cuda()  # noqa: E731
        x, g, b, kv, q = (take(v) for v in ("x", "log_decay", "beta", "kv", "q"))
        tokens = x.shape[0]
        starts = cuda(np.concatenate([[0], np.cumsum(new)]))
        pos = cuda(np.concatenate([o + np.arange(t) for o, t in zip(old, new)]))
        lens = cuda(np.add(old, new))
        mt, kt = cuda(mla_table), cuda(kda_table)
        lay.mla_append(pool.ptr, hkv.hkv_mla_append_args(
            layer=mla, n_seqs=seqs, n_tokens=tokens, n_heads=Q_HEADS, dtype=hkv.HKV_BF16,
            cache_dtype=hkv.HKV_BF16, latent_width=LATENT, rotary_dim=ROTARY, rotary_halves=0,
            n_positions=cos_sin.shape[0], max_blocks=columns, eps=1e-6, cache_scale=1.0,
            kv=kv.data_ptr(), kv_stride=WIDTH, norm_weight=dev["norm"].data_ptr(),
            cos_sin=cos_sin.data_ptr(), positions=pos.data_ptr(), seq_starts=starts.data_ptr(),
            seq_lens=lens.data_ptr(), block_table=mt.data_ptr(), table_stride=columns,
            q_in=q.data_ptr() + LATENT * 2, q_in_token_stride=Q_HEADS * WIDTH, q_in_head_stride=WIDTH,
            q_out=q.data_ptr() + LATENT * 2, q_out_token_stride=Q_HEADS * WIDTH,
            q_out_head_stride=WIDTH), stream())
        out = torch.empty(tokens, hd, dtype=torch.bfloat16, device="cuda")
        src = cuda(kda_src)
        if max(new) > 1:
            at = cuda(old)
            a = hkv.hkv_kda_prefill_args(
                layer=kda, n_seqs=seqs, n_tokens=tokens, max_seq_tokens=max(new), max_blocks=columns,
                dtype=hkv.HKV_BF16, scale=D ** -0.5, eps=1e-6, x=x.data_ptr(), x_stride=3 * hd,
                conv_weight=dev["weight"].data_ptr(), log_decay=g.data_ptr(), decay_stride=hd,
                beta=b.data_ptr(), beta_stride=HEADS, seq_starts=starts.data_ptr(),
                positions=at.data_ptr(), src_blocks=src.data_ptr(), block_table=kt.data_ptr(),
                table_stride=columns, out=out.data_ptr(), out_stride=hd)
            ws = torch.full((lay.kda_prefill_workspace(a),), 0xFF, dtype=torch.uint8, device="cuda")
            lay.kda_prefill(pool.ptr, a, ws.data_ptr(), ws.numel(), stream())
        else:
            dst = cuda([kda_table[s, old[s] // n] for s in range(seqs)])
            lay.kda_step(pool.ptr, hkv.hkv_kda_step_args(
                layer=kda, n_seqs=seqs, dtype=hkv.HKV_BF16, scale=D ** -0.5, eps=1e-6, x=x.data_ptr(),
                x_stride=3 * hd, conv_weight=dev["weight"].data_ptr(), log_decay=g.data_ptr(),
                decay_stride=hd, beta=b.data_ptr(), beta_stride=HEADS, src_blocks=src.data_ptr(),
                dst_blocks=dst.data_ptr(), out=out.data_ptr(), out_stride=hd), stream())
        # every new token attends to the rows up to its own: a sequence each, tables shared
        attn = torch.empty(tokens, Q_HEADS, LATENT, dtype=torch.bfloat16, device="cuda")
        tables = mt[torch.repeat_interleave(torch.arange(seqs), torch.tensor(new)).cuda()].contiguous()
        upto = pos + 1
        a = hkv.hkv_mla_attend_args(
            layer=mla, n_seqs=tokens, n_heads=Q_HEADS, value_width=LATENT, dtype=hkv.HKV_BF16,
            cache_dtype=hkv.HKV_BF16, max_blocks=columns, scale=WIDTH ** -0.5, cache_scale=1.0,
            q=q.data_ptr(), q_seq_stride=Q_HEADS * WIDTH, q_head_stride=WIDTH,
            block_table=tables.data_ptr(), table_stride=columns, seq_lens=upto.data_ptr(),
            out=attn.data_ptr(), out_seq_stride=Q_HEADS * LATENT, out_head_stride=LATENT)
        ws2 = torch.empty(lay.mla_attend_workspace(a), dtype=torch.uint8, device="cuda")
        lay.mla_attend(pool.ptr, a, ws2.data_ptr(), ws2.numel(), stream())
        torch.cuda.synchronize()
        at = 0
        for s in range(seqs):
            lo, hi = old[s], old[s] + new[s]
            o, _, r, w = want[s]
            got = out[at:at + new[s]].cpu().double()
            # bf16's half step and, beside it, a hundredth of it for what fp32 sums are off
            assert (got - o[lo:hi]).norm() <= 2.0 ** -8 * 1.01 * o[lo:hi].norm(), (s, rows)
            got = attn[at:at + new[s]].cpu().double()
            assert (got - w[lo:hi]).norm() <= 2.0 ** -8 * 1.5 * w[lo:hi].norm(), (s, rows)
            cached = pool.rows(mla, torch.bfloat16)[torch.from_numpy(mla_table[s]).long().cuda()]
            cached = cached.reshape(-1, WIDTH)[lo:hi].cpu().double()
            assert (cached - r[lo:hi]).norm() <= 2.0 ** -8 * r[lo:hi].norm()
            at += new[s]

    # the prefix is computed once, stored, and retrieved into the second sequence's blocks
    run([0] * seqs, [prefix, 1], "prefix", [-1, -1])
    ws = torch.empty(lay.workspace_size(4), dtype=torch.uint8, device="cuda")
    objs = [torch.zeros(pool.info["obj_bytes"][o], dtype=torch.uint8, device="cuda") for o in range(lay.O)]

    def blocks(s):
        """The first chunk's block in every KV group (the KDA layers' groups share ids)."""
        t = np.empty((1, lay.G, lay.k), np.int32)
        for g in range(lay.G):
            t[0, g, 0] = mla_table[s, 0] if g == pool.layers[mla]["kv_group"] else spare[g]
        t[0, pool.layers[kda]["kv_group"], 0] = kda_table[s, 0]
        return t

    assert lay.k == 1 and pool.info["chunk_tokens"] == n
    lay.store(pool.ptr, blocks(0), [o.data_ptr() for o in objs], ws.data_ptr(), ws.numel(), stream())
    lay.retrieve(pool.ptr, blocks(1), [o.data_ptr() for o in objs], ws.data_ptr(), ws.numel(), stream())
    torch.cuda.synchronize()
    # both prompts behind the prefix, from its snapshot, in one call
    run([prefix] * seqs, prompt, "prompt", [kda_table[0, 0], kda_table[1, 0]])
    for t in range(steps):
        old = [prefix + p + t for p in prompt]
        run(old, [1] * seqs, "step", [kda_table[s, (old[s] - 1) // n] for s in range(seqs)])
    # the pages at the ends of blocks and behind the last token
    L = pool.layers[kda]
    conv_bytes = 3 * hd * 3 * 2
    for s in range(seqs):
        for done, (state, taps) in want[s][1].items():
            if done == prefix + prompt[s] and done % n:
                continue                           # overwritten by the steps
            base = L["pool_offset"] + int(kda_table[s, (done - 1) // n]) * L["stride"]
            page = pool.bytes[base:base + L["page_bytes"]]
            got = page[conv_bytes:].view(torch.float32).cpu().double().view(HEADS, D, D)
            assert (got - state).norm() <= 2e-6 * state.norm(), (s, done)
            conv = page[:conv_bytes].view(torch.bfloat16).cpu().double().view(3 * hd, 3)
            assert torch.equal(conv, taps), (s, done)
