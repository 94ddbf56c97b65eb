"""The operators that bring new tokens into the hybrid KDA+MLA pool, in plain
torch and through the library: appending MLA rows with the latent norm and the
position rotation (hkv_mla_append) and the KDA layers' prompt form
(hkv_kda_prefill).

A case names one rank's shapes ("kl_tp1", "kl_tp2", "k3_tp8": the workloads of
the same names) and a batch.  The pool is laid out as the library's planner
does for those shapes; only the pages of the layer a case uses hold values.
"""
import math

import numpy as np
import torch

own = False

# One rank's shapes: layer pattern, KDA heads x head_dim, conv rows, MLA bytes
# per value, block size N, pool path (0: shared padded pages, 1: packed).
_KL = [0, 0, 0, 1] * 6 + [0, 0, 1]
_K3 = [0, 0, 0, 1] * 23 + [1]
_SHAPES = {
    "kl_tp1": dict(is_mla=_KL, heads=32, head_dim=128, conv_dim=12288, mla_bytes=2, n=1888, path=1),
    "kl_tp2": dict(is_mla=_KL, heads=16, head_dim=128, conv_dim=6144, mla_bytes=2, n=944, path=0),
    "k3_tp8": dict(is_mla=_K3, heads=6, head_dim=128, conv_dim=2304, mla_bytes=1, n=768, path=0),
}
_WIDTH, _LATENT, _ROTARY, _KERNEL, _EPS = 576, 512, 64, 4, 1e-6
_TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "e4m3": torch.float8_e4m3fn}
_CACHE_SCALE = 1 / 16  # what a cached 1.0 of an e4m3 cache stands for


# ---------------------------------------------------------------- geometry
def _geometry(case):
    """Block size, page sizes and where the layer's pages sit."""
    sh = _SHAPES[case["shapes"]]
    n_mla = sum(sh["is_mla"])
    mla_page = sh["n"] * _WIDTH * sh["mla_bytes"]
    kda_conv = sh["conv_dim"] * (_KERNEL - 1) * 2
    g = dict(sh, mla_page=mla_page, kda_conv=kda_conv, row=_WIDTH * sh["mla_bytes"])
    g["blocks"] = _blocks(case, sh["n"])
    if sh["path"] == 1:  # packed: a block holds every layer of its group
        g["stride"] = n_mla * mla_page
        g["pool_bytes"] = g["blocks"] * g["stride"]
        g["mla_step"], g["kda_step"] = mla_page, kda_conv + sh["heads"] * sh["head_dim"] ** 2 * 4
    else:  # one tensor of padded pages for the s-th layer of every group
        g["stride"] = mla_page
        g["pool_bytes"] = g["blocks"] * mla_page * n_mla
        g["mla_step"] = g["kda_step"] = g["blocks"] * mla_page
    return g


def _batch(case):
    """(tokens already cached, new tokens) of every sequence: new ones between a
    quarter of the longest run and the longest, the longest first; a batch of
    eight or more holds one with nothing to do."""
    n, top = case["seqs"], case["new"]
    new = [top] + [max(1, int(top * (0.25 + 0.75 * ((i * 0.6180339887) % 1.0)))) for i in range(1, n)]
    if n >= 8:
        new[n // 2] = 0
    # sequences that decode one token beside the prompts of the same call
    new += [1] * case.get("riders", 0)
    old = [int(case["old"] * ((0.3 + i * 0.7548776662) % 1.0)) for i in range(len(new))]
    if case["op"] == "prefill" and case["aligned"]:  # prefixes end where blocks do
        block = _SHAPES[case["shapes"]]["n"]
        old = [x // block * block for x in old]
    return old, new


def _touched(old, new, n):
    """Blocks that the new tokens lie in: first, one past the last."""
    return old // n, (-(-(old + new) // n) if new else old // n)


def _blocks(case, n):
    old, new = _batch(case)
    spans = [_touched(o, t, n) for o, t in zip(old, new)]
    sources = len(old) if case["op"] == "prefill" else 0
    return sum(b - a for a, b in spans) + sources + 1


def _mla_rows(pool, g, dtype):
    """[blocks][N][width] view of the second MLA layer's pages."""
    es = dtype.itemsize
    return pool.view(dtype).as_strided((g["blocks"], g["n"], _WIDTH), (g["stride"] // es, _WIDTH, 1),
                                       g["mla_step"] // es)


def _kda_pages(pool, g, dtype):
    """The conv states [blocks][conv_dim][kernel-1] and recurrent states
    [blocks][heads][d][d] of the second layer of KDA group 0."""
    d, off = g["head_dim"], g["kda_step"]
    conv = pool.view(dtype).as_strided((g["blocks"], g["conv_dim"], _KERNEL - 1),
                                       (g["stride"] // 2, _KERNEL - 1, 1), off // 2)
    rec = pool.view(torch.float32).as_strided((g["blocks"], g["heads"], d, d),
                                              (g["stride"] // 4, d * d, d, 1),
                                              (off + g["kda_conv"]) // 4)
    return conv, rec


# ---------------------------------------------------------------- cases
def listed():
    return [
        # one request's next token: latency
        dict(name="append_one", op="append", shapes="kl_tp2", seqs=1, new=1, old=333, heads=16,
             dtype="bf16", halves=False),
        # a large decode batch
        dict(name="append_decode", op="append", shapes="kl_tp2", seqs=256, new=1, old=3000, heads=16,
             dtype="fp16", halves=False),
        # the prompts of a serving step with a large token budget
        dict(name="append_prompt", op="append", shapes="kl_tp1", seqs=6, new=4001, old=9000, heads=32,
             dtype="bf16", halves=True),
        # an fp8 cache, prompts beside decoding sequences
        dict(name="append_fp8", op="append", shapes="k3_tp8", seqs=5, new=1500, old=20000, heads=64,
             dtype="bf16", halves=False, riders=40),
        # a few drafted tokens checked for each of a batch of requests
        dict(name="prefill_draft", op="prefill", shapes="k3_tp8", seqs=61, new=5, old=9000,
             dtype="fp16", misses=False, aligned=False),
        # one request's prompt after a prefix hit, at the rank's token budget
        dict(name="prefill_rank", op="prefill", shapes="k3_tp8", seqs=1, new=1500, old=8000,
             dtype="bf16", misses=False, aligned=True),
        # a budget of 2N - 1 tokens, one prompt that crosses a block
        dict(name="prefill_budget", op="prefill", shapes="kl_tp2", seqs=1, new=1887, old=5000,
             dtype="bf16", misses=False, aligned=True),
        # a budget shared by prompts, new requests among them, and decoding sequences
        dict(name="prefill_mixed", op="prefill", shapes="kl_tp1", seqs=4, new=1400, old=4000,
             dtype="fp16", misses=True, aligned=False, riders=24),
        # one long prompt on a rank with few heads
        dict(name="prefill_long", op="prefill", shapes="k3_tp8", seqs=1, new=16384, old=4000,
             dtype="bf16", misses=False, aligned=True),
        # the largest: many prompts at once
        dict(name="prefill_batch", op="prefill", shapes="kl_tp1", seqs=16, new=2000, old=6000,
             dtype="bf16", misses=True, aligned=True),
        # one long document over all heads
        dict(name="prefill_document", op="prefill", shapes="kl_tp1", seqs=1, new=20011, old=3000,
             dtype="bf16", misses=False, aligned=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "prefill", "prefill"])
    shapes = rng.choice(["kl_tp1", "kl_tp2", "k3_tp8"])
    seqs = _log(rng, 1, 48)
    riders = rng.choice([0, 0, rng.randint(1, 30)])
    if op == "append":
        return dict(op=op, shapes=shapes, seqs=seqs, new=_log(rng, 1, max(2, 12000 // seqs)),
                    old=rng.randint(0, 20000), heads=rng.choice([rng.randint(1, 32), 16, 32]),
                    dtype=rng.choice(["bf16", "fp16"]), halves=rng.random() < 0.5, riders=riders)
    heads = _SHAPES[shapes]["heads"]
    return dict(op=op, shapes=shapes, seqs=seqs,
                new=_log(rng, 1, max(2, min(16384, 480000 // heads) // seqs)), old=rng.randint(0, 9000),
                dtype=rng.choice(["bf16", "fp16"]), misses=rng.random() < 0.5,
                aligned=rng.random() < 0.5, riders=riders)


# ---------------------------------------------------------------- inputs
def prepare(case, seed):
    g = _geometry(case)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rng = np.random.default_rng(seed)
    pool = torch.zeros(g["pool_bytes"], dtype=torch.uint8, device="cuda")
    old, new = _batch(case)
    n, tokens, dt = len(old), sum(new), _TYPES[case["dtype"]]

    def normal(*shape, std=1.0):
        return torch.randn(*shape, device="cuda", generator=gen) * std

    def ints(a):
        return torch.from_numpy(np.asarray(a, np.int32)).cuda()

    # block tables: ids drawn from a shuffled pool for the blocks that the new
    # tokens lie in; no other entry is read
    spans = [_touched(o, t, g["n"]) for o, t in zip(old, new)]
    table = np.full((n, max(1, max(b for _, b in spans))), -1, np.int32)
    ids = rng.permutation(g["blocks"] - 1).astype(np.int32)
    at = 0
    for s, (a, b) in enumerate(spans):
        table[s, a:b] = ids[at:at + b - a]
        at += b - a
    starts = np.concatenate([[0], np.cumsum(new)])
    st = dict(case=case, g=g, pool=pool, old=old, new=new, table=ints(table), starts=ints(starts),
              host_table=table, host_starts=starts)
    if case["op"] == "append":
        cache = _TYPES["e4m3"] if g["mla_bytes"] == 1 else dt
        rows = _mla_rows(pool, g, torch.uint8 if g["mla_bytes"] == 1 else dt)
        for b in range(0, g["blocks"], 64):  # what earlier tokens left
            part = normal(*rows[b:b + 64].shape).to(cache)
            rows[b:b + 64] = part.view(torch.uint8) if cache.itemsize == 1 else part
        # a third of the sequences were cut to a budget before: their slots lie below
        # their tokens' positions
        shift = np.where(np.arange(n) % 3 == 2, 4096, 0)
        positions = np.concatenate([o + k + np.arange(t) for o, k, t in zip(old, shift, new)])
        top = int(positions.max()) + 1
        angle = torch.arange(top, dtype=torch.float64, device="cuda").unsqueeze(1) * \
            10000.0 ** (-torch.arange(0, _ROTARY, 2, dtype=torch.float64, device="cuda") / _ROTARY)
        st.update(cache=cache, lens=ints(np.add(old, new)), positions=ints(positions),
                  cos_sin=torch.cat([angle.cos(), angle.sin()], 1).float(),
                  kv=normal(tokens, _WIDTH).to(dt), norm=(1 + normal(_LATENT, std=0.1)).to(dt),
                  q=normal(tokens, case["heads"], _ROTARY, std=3.0).to(dt),
                  q_out=torch.zeros(tokens, case["heads"], _WIDTH, dtype=dt, device="cuda"))
        return st
    h, d = g["heads"], g["head_dim"]
    conv, rec = _kda_pages(pool, g, dt)
    conv.copy_(normal(*conv.shape).to(dt))
    rec.copy_(normal(*rec.shape, std=0.1))
    src = ids[at:at + n].copy()
    start = np.asarray(old)
    if case["misses"]:  # requests with no cached prefix start from zeros
        src[::5] = -1
    st.update(x=normal(tokens, g["conv_dim"]).to(dt),
              conv_weight=normal(g["conv_dim"], _KERNEL, std=0.5).to(dt),
              log_decay=-torch.rand(tokens, h * d, device="cuda", generator=gen) ** 4,
              beta=torch.rand(tokens, h, device="cuda", generator=gen),
              src=ints(src), host_src=src, positions=ints(start),
              out=torch.zeros(tokens, h * d, dtype=dt, device="cuda"))
    return st


# ---------------------------------------------------------------- plain forms
def _plain_append(st):
    case, g, dt = st["case"], st["g"], st["kv"].dtype
    new = torch.diff(st["starts"].long())
    tokens = st["kv"].shape[0]
    seq = torch.repeat_interleave(torch.arange(new.numel(), device="cuda"), new, output_size=tokens)
    slot = (st["lens"].long() - st["starts"][1:])[seq] + torch.arange(tokens, device="cuda")
    block = st["table"].long()[seq, slot // g["n"]]
    cos, sin = st["cos_sin"][st["positions"].long()].chunk(2, 1)

    def turned(x, cos, sin):
        x = x.float()
        if case["halves"]:
            a, b = x.chunk(2, -1)
            return torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
        a, b = x[..., 0::2], x[..., 1::2]
        return torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)

    c = st["kv"][:, :_LATENT].float()
    c = c * torch.rsqrt(c.square().mean(1, keepdim=True) + _EPS) * st["norm"].float()
    row = torch.cat([c, turned(st["kv"][:, _LATENT:], cos, sin)], 1)
    rows = _mla_rows(st["pool"], g, torch.uint8 if g["mla_bytes"] == 1 else dt)
    if g["mla_bytes"] == 1:
        row = (row / _CACHE_SCALE).clamp(-448, 448).to(st["cache"]).view(torch.uint8)
    rows[block, slot % g["n"]] = row.to(rows.dtype)
    st["q_out"][:, :, _LATENT:] = turned(st["q"], cos.unsqueeze(1), sin.unsqueeze(1)).to(dt)
    return dict(rows=rows.view(st["cache"]), q=st["q_out"])


_CHUNK = 16


def _chunks(st):
    """The prompts in chunks of 16 tokens that end where their positions are
    multiples of 16 (block sizes are): token rows [chunks][16] (-1: none), each
    chunk's sequence and its place in it, and the block whose state it ends
    (-1: none).  Chunks are ordered by their place."""
    out = []
    for s, (old, new) in enumerate(zip(st["old"], st["new"])):
        for i, lo in enumerate(range(old // _CHUNK * _CHUNK, old + new, _CHUNK)):
            hi = min(lo + _CHUNK, old + new)
            rows = [st["host_starts"][s] + p - old if old <= p < hi else -1 for p in range(lo, lo + _CHUNK)]
            ends = hi == old + new or hi % st["g"]["n"] == 0
            out.append((i, s, st["host_table"][s, lo // st["g"]["n"]] if ends else -1, rows, hi - 1))
    out.sort(key=lambda c: c[0])
    return out


def _conv_taps(st, conv, seq, at, k):
    """The values k tokens before those at offset `at` of their sequences: from
    the call's rows, or from the source pages' conv states where they lie before."""
    back = at - k
    x = st["x"][(st["starts"].long()[seq] + back.clamp(min=0))]
    src = st["src"].long()[seq]
    old = conv[src.clamp(min=0), :, (_KERNEL - 1 + back).clamp(0, _KERNEL - 2)]
    old = torch.where((src < 0).unsqueeze(1), torch.zeros_like(old), old)
    return torch.where((back < 0).unsqueeze(1), old, x)


def _plain_prefill(st):
    g = st["g"]
    h, d, dt = g["heads"], g["head_dim"], st["x"].dtype
    conv, rec = _kda_pages(st["pool"], g, dt)
    tokens = st["x"].shape[0]
    if "chunks" not in st:  # the schedule: made once for a batch's lengths
        st["chunks"] = _chunks(st)
    chunks = st["chunks"]
    new = torch.diff(st["starts"].long())
    seq = torch.repeat_interleave(torch.arange(new.numel(), device="cuda"), new, output_size=tokens)
    at = torch.arange(tokens, device="cuda") - st["starts"].long()[seq]
    # the conv, for all tokens; zeros behind the last row stand for absent tokens
    y = torch.zeros(tokens + 1, 3 * h * d, device="cuda")
    for lo in range(0, tokens, 8192):
        part = slice(lo, min(tokens, lo + 8192))
        sum_ = sum(_conv_taps(st, conv, seq[part], at[part], _KERNEL - 1 - j).float()
                   * st["conv_weight"][:, j].float() for j in range(_KERNEL))
        y[part] = sum_ * torch.sigmoid(sum_)
    # the pages' new conv states
    ends = [(c[2], c[1], c[4] - st["old"][c[1]]) for c in chunks if c[2] >= 0]
    if ends:
        block, s, last = (torch.tensor(v, device="cuda") for v in zip(*ends))
        conv[block] = torch.stack([_conv_taps(st, conv, s, last, _KERNEL - 2 - j)
                                   for j in range(_KERNEL - 1)], 2)
    y = y.view(tokens + 1, 3, h, d)
    y[:, :2] *= torch.rsqrt(y[:, :2].square().sum(3, keepdim=True) + _EPS)
    gates = torch.cat([st["log_decay"], torch.zeros(1, h * d, device="cuda")]).view(-1, h, d)
    beta = torch.cat([st["beta"], torch.zeros(1, h, device="cuda")])
    rows = torch.tensor([c[3] for c in chunks], device="cuda")
    place = [c[0] for c in chunks]
    state = torch.zeros(new.numel(), h, d, d, device="cuda")
    hit = st["src"] >= 0
    state[hit] = rec[st["src"][hit].long()]
    tri = torch.ones(_CHUNK, _CHUNK, device="cuda").tril()
    eye = torch.eye(_CHUNK, device="cuda")
    step = max(1, (1 << 29) // (h * _CHUNK * _CHUNK * d))
    lo = 0
    while lo < len(chunks):
        # all that does not depend on the state, for as many places as fit
        hi = lo
        while hi < len(chunks) and (hi - lo < step or place[hi] == place[hi - 1]):
            hi += 1
        r = rows[lo:hi]
        q, k, v = (y[r, j].transpose(1, 2) for j in range(3))  # [chunks][h][16][d]
        b = beta[r].transpose(1, 2).unsqueeze(3)
        cum = gates[r].transpose(1, 2).cumsum(2)
        decay = torch.exp(cum.unsqueeze(3) - cum.unsqueeze(2)) * tri.unsqueeze(2)
        kd = decay * k.unsqueeze(2)
        a = (kd * k.unsqueeze(3)).sum(4) * b * (tri - eye)
        p = (kd * q.unsqueeze(3)).sum(4)
        del decay, kd
        inv = eye - a
        power = torch.matmul(a, a)
        for _ in range(3):  # (1 + a)^-1 = (1 - a)(1 + a^2)(1 + a^4)(1 + a^8): a^16 = 0
            inv = inv + torch.matmul(inv, power)
            power = torch.matmul(power, power)
        w, u0 = torch.matmul(inv, b * k * cum.exp()), torch.matmul(inv, b * v)
        q = q * cum.exp()
        k = (k * torch.exp(cum[:, :, -1:] - cum)).transpose(2, 3).contiguous()
        end = cum[:, :, -1].exp().unsqueeze(3)
        o = torch.empty_like(v)
        i = lo
        while i < hi:  # places in order, all sequences that have one at once
            j = i
            while j < hi and place[j] == place[i]:
                j += 1
            c, s = slice(i - lo, j - lo), [x[1] for x in chunks[i:j]]
            s = slice(s[0], s[0] + 1) if len(s) == 1 else torch.tensor(s, device="cuda")
            old = state[s]
            u = u0[c] - torch.matmul(w[c], old)
            o[c] = torch.matmul(q[c], old) + torch.matmul(p[c], u)
            now = end[c] * old + torch.matmul(k[c], u)
            state[s] = now
            done = [(m, x[2]) for m, x in enumerate(chunks[i:j]) if x[2] >= 0]
            if done:
                m, block = (torch.tensor(z, device="cuda") for z in zip(*done))
                rec[block] = now[m]
            i = j
        live = r >= 0
        st["out"].view(tokens, h, d)[r[live]] = (o.transpose(1, 2)[live] * d ** -0.5).to(dt)
        lo = hi
    return dict(out=st["out"], recurrent=rec, conv=conv)


# ---------------------------------------------------------------- the library
def _plan(st):
    """What a serving program sets up once for its buffers: the layout, the
    argument block and the workspace."""
    import retrieve_store_chunk_amd as hkv

    case, g = st["case"], st["g"]
    lay = hkv.Layout(dict(is_mla=g["is_mla"], kda_heads=g["heads"], kda_head_dim=g["head_dim"],
                          kda_state_bytes=4, conv_dim=g["conv_dim"], conv_kernel=_KERNEL,
                          conv_bytes=2, mla_width=_WIDTH, mla_bytes=g["mla_bytes"],
                          block_size=g["n"], path=g["path"], pool_bytes=g["pool_bytes"]))
    dtype = hkv.HKV_BF16 if case["dtype"] == "bf16" else hkv.HKV_FP16
    common = dict(n_seqs=len(st["old"]), n_tokens=sum(st["new"]), dtype=dtype,
                  max_blocks=st["table"].shape[1], block_table=st["table"].data_ptr(),
                  table_stride=st["table"].stride(0), seq_starts=st["starts"].data_ptr(),
                  positions=st["positions"].data_ptr())
    if case["op"] == "append":
        q_out = st["q_out"][:, :, _LATENT:]
        a = hkv.hkv_mla_append_args(
            layer=[i for i, m in enumerate(g["is_mla"]) if m][1], n_heads=case["heads"],
            cache_dtype=hkv.HKV_E4M3 if g["mla_bytes"] == 1 else dtype, latent_width=_LATENT,
            rotary_dim=_ROTARY, rotary_halves=int(case["halves"]), n_positions=st["cos_sin"].shape[0],
            eps=_EPS, cache_scale=_CACHE_SCALE if g["mla_bytes"] == 1 else 1.0,
            kv=st["kv"].data_ptr(), kv_stride=st["kv"].stride(0), norm_weight=st["norm"].data_ptr(),
            cos_sin=st["cos_sin"].data_ptr(), seq_lens=st["lens"].data_ptr(),
            q_in=st["q"].data_ptr(), q_in_token_stride=st["q"].stride(0),
            q_in_head_stride=st["q"].stride(1), q_out=q_out.data_ptr(),
            q_out_token_stride=q_out.stride(0), q_out_head_stride=q_out.stride(1), **common)
        rows = _mla_rows(st["pool"], g, torch.uint8 if g["mla_bytes"] == 1 else st["kv"].dtype)
        return lay, a, None, dict(rows=rows.view(st["cache"]), q=st["q_out"])
    a = hkv.hkv_kda_prefill_args(
        layer=1, max_seq_tokens=max(st["new"]), scale=g["head_dim"] ** -0.5, eps=_EPS,
        x=st["x"].data_ptr(), x_stride=st["x"].stride(0), conv_weight=st["conv_weight"].data_ptr(),
        log_decay=st["log_decay"].data_ptr(), decay_stride=st["log_decay"].stride(0),
        beta=st["beta"].data_ptr(), beta_stride=st["beta"].stride(0), src_blocks=st["src"].data_ptr(),
        out=st["out"].data_ptr(), out_stride=st["out"].stride(0), **common)
    conv, rec = _kda_pages(st["pool"], g, st["x"].dtype)
    ws = torch.empty(max(16, lay.kda_prefill_workspace(a)), dtype=torch.uint8, device="cuda")
    return lay, a, ws, dict(out=st["out"], recurrent=rec, conv=conv)


def _library(st):
    if "plan" not in st:
        st["plan"] = _plan(st)
    lay, a, ws, res = st["plan"]
    stream = torch.cuda.current_stream().cuda_stream
    if ws is None:
        lay.mla_append(st["pool"].data_ptr(), a, stream)
    else:
        lay.kda_prefill(st["pool"].data_ptr(), a, ws.data_ptr(), ws.numel(), stream)
    return res


def run(state):
    if own:
        return _library(state)
    return _plain_append(state) if state["case"]["op"] == "append" else _plain_prefill(state)


# ---------------------------------------------------------------- work
def work(case):
    g = _geometry(case)
    old, new = _batch(case)
    tokens = sum(new)
    if case["op"] == "append":
        moved = tokens * (_WIDTH * 2 + g["row"] + 4 + 2 * case["heads"] * _ROTARY * 2)
        table = min(tokens, max(old) + max(new) + 4096) * _ROTARY * 4
        return {"bytes": moved + table, "flops": tokens * (4 * _LATENT + 3 * _ROTARY * (1 + case["heads"]))}
    h, d, c = g["heads"], g["head_dim"], g["conv_dim"]
    page = h * d * d * 4 + c * (_KERNEL - 1) * 2
    live = [(o, t, i) for i, (o, t) in enumerate(zip(old, new)) if t]
    reads = sum(1 for _, _, i in live if not (case["misses"] and i % 5 == 0))
    writes = sum(b - a for a, b in (_touched(o, t, g["n"]) for o, t, _ in live))
    return {"bytes": (reads + writes) * page + tokens * (c * 2 + h * d * 4 + h * 4 + h * d * 2) + c * _KERNEL * 2,
            "flops": tokens * (h * d * d * 7 + c * (2 * _KERNEL + 4))}


# ---------------------------------------------------------------- 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    return _exact_append(st) if case["op"] == "append" else _exact_prefill(st)


def _exact_append(st):
    case, g = st["case"], st["g"]
    es = st["cache"].itemsize
    rows = _mla_rows(st["pool"], g, torch.uint8 if es == 1 else st["cache"])
    rows = rows.contiguous().view(st["cache"]).double()
    kv, pos = st["kv"].double(), st["positions"].long()
    scale = _CACHE_SCALE if es == 1 else 1.0
    freq = st["cos_sin"].double()[pos]
    turn = torch.complex(freq[:, :_ROTARY // 2], freq[:, _ROTARY // 2:])

    def rotate(x, by):
        if case["halves"]:
            z = torch.complex(x[..., :_ROTARY // 2].contiguous(), x[..., _ROTARY // 2:].contiguous()) * by
            return torch.cat([z.real, z.imag], -1)
        z = torch.view_as_complex(x.reshape(*x.shape[:-1], -1, 2).contiguous()) * by
        return torch.view_as_real(z).flatten(-2)

    rms = torch.sqrt((kv[:, :_LATENT] ** 2).sum(1, keepdim=True) / _LATENT + _EPS)
    kv = torch.cat([kv[:, :_LATENT] / rms * st["norm"].double(), rotate(kv[:, _LATENT:], turn)], 1)
    for s, (old, new) in enumerate(zip(st["old"], st["new"])):
        at = old
        while at < old + new:
            stop = min((at // g["n"] + 1) * g["n"], old + new)
            first = st["host_starts"][s] + at - old
            rows[int(st["host_table"][s, at // g["n"]]), at % g["n"]:at % g["n"] + stop - at] = \
                kv[first:first + stop - at] / scale
            at = stop
    q = torch.zeros(st["q_out"].shape, dtype=torch.float64, device=kv.device)
    q[:, :, _LATENT:] = rotate(st["q"].double(), turn.unsqueeze(1))
    return dict(rows=rows, q=q)


def _exact_prefill(st):
    """Token by token, all sequences side by side."""
    g = st["g"]
    h, d, n = g["heads"], g["head_dim"], len(st["old"])
    conv, rec = (x.double() for x in _kda_pages(st["pool"], g, st["x"].dtype))
    dev = rec.device
    src, first = st["src"].long(), st["starts"].long()[:-1]
    state = torch.where((src < 0).view(n, 1, 1, 1), 0.0, rec[src.clamp(min=0)])
    taps = torch.where((src < 0).view(n, 1, 1), 0.0, conv[src.clamp(min=0)])
    weight = st["conv_weight"].double()
    out = torch.zeros(st["x"].shape[0], h * d, dtype=torch.float64, device=dev)
    order = sorted(range(n), key=lambda s: -st["new"][s])  # those still running lead
    by = torch.tensor(order, device=dev)
    state, taps, first = state[by], taps[by], first[by]
    steps = [st["new"][s] for s in order]
    live = n
    for t in range(max(steps)):
        while live and steps[live - 1] <= t:
            live -= 1
        row = first[:live] + t
        window = torch.cat([taps[:live], st["x"][row].double().unsqueeze(2)], 2)
        taps[:live] = window[:, :, 1:]
        y = (window * weight).sum(2)
        y = (y / (1 + torch.exp(-y))).view(live, 3, h, d)
        q, k = (y[:, j] / torch.sqrt((y[:, j] ** 2).sum(2, keepdim=True) + _EPS) for j in (0, 1))
        s = state[:live]
        s *= torch.exp(st["log_decay"][row].double()).view(live, h, d, 1)
        seen = torch.matmul(k.unsqueeze(2), s).squeeze(2)
        u = st["beta"][row].double().unsqueeze(2) * (y[:, 2] - seen)
        s += k.unsqueeze(3) * u.unsqueeze(2)
        out[row] = torch.matmul(q.unsqueeze(2), s).reshape(live, h * d) * d ** -0.5
        for m in range(live):
            at = st["old"][order[m]] + t
            if t == steps[m] - 1 or (at + 1) % g["n"] == 0:
                b = int(st["host_table"][order[m], at // g["n"]])
                rec[b], conv[b] = s[m], taps[m]
    return dict(out=out, recurrent=rec, conv=conv)
