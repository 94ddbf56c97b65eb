"""The decode-step operators over the hybrid KDA+MLA pool, in plain torch and
through the library: MLA attention of one new token per sequence
(hkv_mla_attend), eviction by accumulated attention weight (hkv_mla_evict) and
the KDA layers' recurrent step (hkv_kda_step).

A case names one rank's shapes ("kl_tp1", "kl_tp2", "k3_tp8": the workloads of
the same names) and a batch.  The pool is laid out as the library's planner
does for those shapes; only the pages of the layers a case uses hold values.
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
_WIDTH, _VALUES, _KERNEL = 576, 512, 4
_TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "e4m3": torch.float8_e4m3fn}


# ---------------------------------------------------------------- geometry
def _geometry(case):
    """Block size, page sizes and where the MLA layers (and KDA group 0) sit."""
    sh = _SHAPES[case["shapes"]]
    n_mla = sum(sh["is_mla"])
    mla_page = sh["n"] * _WIDTH * sh["mla_bytes"]
    kda_conv = sh["conv_dim"] * (_KERNEL - 1) * 2
    g = dict(sh, n_mla=n_mla, mla_page=mla_page, kda_conv=kda_conv, row=_WIDTH * sh["mla_bytes"])
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


def _lens(case):
    """Ragged lengths between a quarter of the longest and the longest, the
    longest first; a batch of eight or more holds an idle (empty) sequence."""
    n, top = case["seqs"], case["len"]
    out = [top] + [max(1, int(top * (0.25 + 0.75 * ((i * 0.6180339887) % 1.0)))) for i in range(1, n)]
    if n >= 8:
        out[n // 2] = 0
    return out


def _blocks(case, n):
    if case["op"] == "kda":
        return 2 * case["seqs"] + 1
    return sum(-(-x // n) for x in _lens(case)) + 1


def _tables(case, g, rng):
    """[seqs][max_blocks] block ids drawn from a shuffled pool (the last block
    stays spare), -1 past a sequence's end."""
    lens = _lens(case)
    need = [-(-x // g["n"]) for x in lens]
    ids = rng.permutation(g["blocks"] - 1).astype(np.int32)
    table = np.full((len(lens), max(1, max(need))), -1, np.int32)
    at = 0
    for s, k in enumerate(need):
        table[s, :k] = ids[at:at + k]
        at += k
    return lens, table


def _mla_rows(pool, g, dtype):
    """[n_mla][blocks][N][width] view of the MLA layers' pages."""
    es = dtype.itemsize
    return pool.view(dtype).as_strided((g["n_mla"], g["blocks"], g["n"], _WIDTH),
                                       (g["mla_step"] // es, g["stride"] // es, _WIDTH, 1))


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
        # one request just past its first tokens: latency
        dict(name="attend_one_short", op="attend", shapes="kl_tp2", seqs=1, len=333, heads=16,
             dtype="bf16", cache="bf16", weights=False, holes=False),
        # an ordinary ragged serving batch
        dict(name="attend_batch", op="attend", shapes="kl_tp1", seqs=64, len=14001, heads=32,
             dtype="bf16", cache="bf16", weights=False, holes=False),
        # one request over a million-token prefix
        dict(name="attend_long", op="attend", shapes="kl_tp1", seqs=1, len=1000000, heads=32,
             dtype="bf16", cache="bf16", weights=False, holes=False),
        # an fp8 cache whose older blocks were partly dropped (null ids)
        dict(name="attend_fp8_holes", op="attend", shapes="k3_tp8", seqs=24, len=40000, heads=64,
             dtype="bf16", cache="e4m3", weights=False, holes=True),
        # the pass before an eviction: the attention weights are accumulated
        dict(name="attend_weights", op="attend", shapes="kl_tp1", seqs=16, len=9000, heads=32,
             dtype="fp16", cache="fp16", weights=True, holes=False),
        # a few requests over a small budget: latency
        dict(name="evict_small", op="evict", shapes="kl_tp2", seqs=4, len=1500, layers=1,
             budget=1024, sinks=4, recent=128, cache="bf16"),
        # every MLA layer of a batch cut to half its length
        dict(name="evict_batch", op="evict", shapes="kl_tp1", seqs=16, len=8192, layers=7,
             budget=4096, sinks=4, recent=512, cache="bf16"),
        # a long fp8 context, all 24 layers
        dict(name="evict_long", op="evict", shapes="k3_tp8", seqs=1, len=262144, layers=24,
             budget=100000, sinks=16, recent=4096, cache="e4m3"),
        # one request's step: latency
        dict(name="kda_one", op="kda", shapes="kl_tp2", seqs=1, dtype="bf16", misses=False),
        # a rank with few heads, some requests starting from nothing
        dict(name="kda_rank", op="kda", shapes="k3_tp8", seqs=61, dtype="fp16", misses=True),
        # a large decode batch
        dict(name="kda_batch", op="kda", shapes="kl_tp1", seqs=256, dtype="bf16", misses=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attend", "attend", "evict", "kda"])
    shapes = rng.choice(["kl_tp1", "kl_tp2", "k3_tp8"])
    if op == "kda":
        return dict(op=op, shapes=shapes, seqs=_log(rng, 1, 256), dtype=rng.choice(["bf16", "fp16"]),
                    misses=rng.random() < 0.5)
    if op == "evict":
        cap = 1000000 // (24 if shapes == "k3_tp8" else 7)
        seqs = _log(rng, 1, 32)
        top = _log(rng, 2, cap // seqs)
        budget = max(1, int(top * rng.uniform(0.2, 1.1)))
        recent = int(budget * rng.uniform(0, 0.5))
        layers = rng.randint(1, 24 if shapes == "k3_tp8" else 7)
        return dict(op=op, shapes=shapes, seqs=seqs, len=top, layers=layers, budget=budget,
                    sinks=min(rng.randint(0, 8), budget - recent), recent=recent,
                    cache="e4m3" if shapes == "k3_tp8" else rng.choice(["bf16", "fp16"]))
    heads = rng.choice([rng.randint(1, 128), 16, 32, 64])
    seqs = _log(rng, 1, 64)
    top = _log(rng, 1, max(2, min(900000, 28000000 // heads) // seqs))
    dtype = rng.choice(["bf16", "fp16"])
    return dict(op=op, shapes=shapes, seqs=seqs, len=top, heads=heads, dtype=dtype,
                cache="e4m3" if shapes == "k3_tp8" else dtype, weights=rng.random() < 0.3,
                holes=rng.random() < 0.3)


# ---------------------------------------------------------------- inputs
def prepare(case, seed):
    g = _geometry(case)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rng = np.random.default_rng(seed)
    pool = torch.zeros(g["pool_bytes"], dtype=torch.uint8, device="cuda")
    st = dict(case=case, g=g, pool=pool)

    def normal(*shape, std=1.0):
        return torch.randn(*shape, device="cuda", generator=gen) * std

    if case["op"] == "kda":
        n, h, d, dt = case["seqs"], g["heads"], g["head_dim"], _TYPES[case["dtype"]]
        conv, rec = _kda_pages(pool, g, dt)
        conv.copy_(normal(*conv.shape).to(dt))
        rec.copy_(normal(*rec.shape, std=0.1))
        ids = rng.permutation(2 * n).astype(np.int32)
        src, dst = ids[:n].copy(), ids[n:].copy()
        if case["misses"]:  # requests with no state yet start from zeros
            src[::5] = -1
        st.update(x=normal(n, g["conv_dim"]).to(dt),
                  conv_weight=normal(g["conv_dim"], _KERNEL, std=0.5).to(dt),
                  log_decay=-torch.rand(n, h * d, device="cuda", generator=gen) ** 4,
                  beta=torch.rand(n, h, device="cuda", generator=gen),
                  src=torch.from_numpy(src).cuda(), dst=torch.from_numpy(dst).cuda(),
                  out=torch.zeros(n, h * d, dtype=dt, device="cuda"))
        return st

    lens, table = _tables(case, g, rng)
    n, cap = len(lens), table.shape[1] * g["n"]
    cache = _TYPES[case["cache"]]
    rows = _mla_rows(pool, g, torch.uint8 if cache.itemsize == 1 else cache)
    st.update(lens=torch.tensor(lens, dtype=torch.int32, device="cuda"), longest=max(lens))
    if case["op"] == "attend":
        layer = rows[1]  # the second MLA layer
        for b in range(0, g["blocks"], 64):
            part = normal(*layer[b:b + 64].shape)
            part = (part * 16).to(cache).view(torch.uint8) if cache.itemsize == 1 else part.to(cache)
            layer[b:b + 64] = part
        if case["holes"]:  # every third block of a sequence, its newest kept
            for s, x in enumerate(lens):
                table[s, 0:max(0, -(-x // g["n"]) - 1):3] = -1
        dt = _TYPES[case["dtype"]]
        st.update(table=torch.from_numpy(table).cuda(),
                  q=normal(n, case["heads"], _WIDTH, std=3.0).to(dt),
                  scale=_WIDTH ** -0.5, cache_scale=1 / 16 if cache.itemsize == 1 else 1.0,
                  out=torch.zeros(n, case["heads"], _VALUES, dtype=dt, device="cuda"),
                  lse=torch.zeros(n, case["heads"], device="cuda"))
        if case["weights"]:  # what earlier steps left
            st["weights_in"] = torch.rand(n, cap, device="cuda", generator=gen)
            st["weights"] = st["weights_in"].clone()
        return st

    k = case["layers"]
    for i in range(k):
        for b in range(0, g["blocks"], 64):
            part = normal(*rows[i, b:b + 64].shape)
            part = (part * 16).to(cache).view(torch.uint8) if cache.itemsize == 1 else part.to(cache)
            rows[i, b:b + 64] = part
    # weights fall off like attention's: most small, some large, many never looked at
    w = normal(k, n, cap, std=2.0).exp()
    w = torch.where(torch.rand(k, n, cap, device="cuda", generator=gen) < 0.2, 0.0, w)
    # slots are ordered by position where they were appended, shuffled where an
    # earlier eviction moved rows into freed slots
    pos = torch.randint(1, 3, (k, n, cap), device="cuda", generator=gen).cumsum(2).int() - 1
    old = max(1, case["len"] // 2)
    perm = torch.randperm(old, device="cuda", generator=gen)
    pos[:, :, :old] = pos[:, :, perm]
    # the position of the next token: past the newest slot's
    nxt = torch.where(torch.arange(cap, device="cuda") < st["lens"].view(1, n, 1), pos, -1)
    st.update(table=torch.from_numpy(table).cuda(), weights=w, positions=pos,
              next_positions=(nxt.amax(dim=(0, 2)) + 1).int(),
              weights_out=torch.zeros_like(w), positions_out=torch.zeros_like(pos),
              new_lens=torch.zeros(n, dtype=torch.int32, device="cuda"))
    return st


# ---------------------------------------------------------------- plain forms
def _gather(st, layer, slots):
    """Rows [seqs][slots][width] of one layer, as stored; null blocks read the
    spare block."""
    g = st["g"]
    cache = _TYPES[st["case"]["cache"]]
    rows = _mla_rows(st["pool"], g, torch.uint8 if cache.itemsize == 1 else cache)[layer]
    ids = st["table"].long()[:, slots // g["n"]]
    got = rows[torch.where(ids < 0, g["blocks"] - 1, ids), slots % g["n"]]
    return got.view(cache).float(), ids >= 0


def _plain_attend(st):
    case = st["case"]
    slots = torch.arange(max(1, st["longest"]), device="cuda")
    rows, there = _gather(st, 1, slots)
    live = (there & (slots < st["lens"].view(-1, 1))).unsqueeze(1)
    logits = torch.matmul(st["q"].float(), rows.transpose(1, 2)) * (st["scale"] * st["cache_scale"])
    logits = torch.where(live, logits, -math.inf)
    top = logits.amax(2, keepdim=True)
    p = torch.exp(logits - torch.where(top == -math.inf, 0.0, top))
    total = p.sum(2, keepdim=True)
    p = torch.where(total > 0, p / total, 0.0)
    out = torch.matmul(p, rows[:, :, :_VALUES]) * st["cache_scale"]
    res = dict(out=out.to(_TYPES[case["dtype"]]), lse=(top + total.log()).squeeze(2))
    if case["weights"]:
        w = st["weights_in"].clone()
        w[:, :slots.numel()] += p.sum(1)
        res["weights"] = w
    return res


def _plain_evict(st):
    case, g = st["case"], st["g"]
    w, pos, k, n, budget = st["weights"], st["positions"], case["layers"], case["seqs"], case["budget"]
    cap = w.shape[2]
    slot = torch.arange(cap, device="cuda")
    lens = st["lens"].view(1, n, 1)
    new = lens.clamp(max=budget)
    live = slot < lens
    held = (pos < case["sinks"]) | (pos >= st["next_positions"].view(1, n, 1) - case["recent"])
    key = torch.where(live, torch.where(held, math.inf, w), -math.inf)
    order = torch.sort(key, dim=2, descending=True, stable=True).indices
    rank = torch.empty_like(order).scatter_(2, order, slot.expand_as(order))
    keep = live & (rank < budget)
    hole, mover = live & ~keep & (slot < new), keep & (slot >= new)
    holes = torch.sort((~hole).to(torch.uint8), dim=2, stable=True).indices
    movers = torch.sort((~mover).to(torch.uint8), dim=2, stable=True).indices
    moved = slot < hole.sum(2, keepdim=True)
    src = slot.expand_as(pos).clone()
    src.scatter_(2, holes, torch.where(moved, movers, holes))
    # metadata: kept slots below the new length, then cleared ones
    gone = live & (slot >= new)
    st["weights_out"].copy_(torch.where(gone, 0.0, torch.where(live, w.gather(2, src), st["weights_out"])))
    st["positions_out"].copy_(torch.where(gone, -1, torch.where(live, pos.gather(2, src), st["positions_out"])))
    st["new_lens"].copy_(new.view(n))
    # rows: every slot below the budget takes its source's (most their own)
    top = min(budget, cap)
    last = (lens - 1).clamp(min=0)
    dst = torch.minimum(slot[:top].expand(k, n, top), last.expand(k, n, top))
    src = src.gather(2, dst)
    cache = _TYPES[case["cache"]]
    rows = _mla_rows(st["pool"], g, torch.uint8 if cache.itemsize == 1 else cache)
    layer = torch.arange(k, device="cuda").view(k, 1, 1)
    table = st["table"].long().expand(k, n, -1)
    spare = g["blocks"] - 1

    def ids(at):
        got = table.gather(2, at // g["n"])
        return torch.where(got < 0, spare, got)

    rows[layer, ids(dst), dst % g["n"]] = rows[layer, ids(src), src % g["n"]]
    return dict(rows=rows[:k], weights=st["weights_out"], positions=st["positions_out"],
                new_lens=st["new_lens"])


def _plain_kda(st):
    g, dt = st["g"], _TYPES[st["case"]["dtype"]]
    n, h, d = st["x"].shape[0], g["heads"], g["head_dim"]
    conv, rec = _kda_pages(st["pool"], g, dt)
    src, dst = st["src"].long(), st["dst"].long()
    hit = src >= 0
    old = conv[src.clamp(min=0)] * hit.view(n, 1, 1)
    window = torch.cat([old, st["x"].unsqueeze(2)], 2)
    y = (window.float() * st["conv_weight"].float()).sum(2)
    y = (y * torch.sigmoid(y)).view(n, 3, h, d)
    q = y[:, 0] * torch.rsqrt(y[:, 0].square().sum(2, keepdim=True) + 1e-6) * d ** -0.5
    k = y[:, 1] * torch.rsqrt(y[:, 1].square().sum(2, keepdim=True) + 1e-6)
    s = rec[src.clamp(min=0)] * hit.view(n, 1, 1, 1)
    s = s * torch.exp(st["log_decay"].view(n, h, d, 1))
    u = st["beta"].unsqueeze(2) * (y[:, 2] - (k.unsqueeze(3) * s).sum(2))
    s = s + k.unsqueeze(3) * u.unsqueeze(2)
    out = (q.unsqueeze(3) * s).sum(2)
    rec[dst] = s
    conv[dst] = window[:, :, 1:]
    return dict(out=out.reshape(n, h * d).to(dt), recurrent=rec, conv=conv)


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
    mla = [i for i, m in enumerate(g["is_mla"]) if m]
    types = {"bf16": hkv.HKV_BF16, "fp16": hkv.HKV_FP16, "e4m3": hkv.HKV_E4M3}
    if case["op"] == "kda":
        a = hkv.hkv_kda_step_args(
            layer=1, n_seqs=case["seqs"], dtype=types[case["dtype"]], scale=g["head_dim"] ** -0.5,
            eps=1e-6, x=st["x"].data_ptr(), x_stride=st["x"].stride(0),
            conv_weight=st["conv_weight"].data_ptr(), log_decay=st["log_decay"].data_ptr(),
            decay_stride=st["log_decay"].stride(0), beta=st["beta"].data_ptr(),
            beta_stride=st["beta"].stride(0), src_blocks=st["src"].data_ptr(),
            dst_blocks=st["dst"].data_ptr(), out=st["out"].data_ptr(), out_stride=st["out"].stride(0))
        conv, rec = _kda_pages(st["pool"], g, _TYPES[case["dtype"]])
        return lay, a, None, dict(out=st["out"], recurrent=rec, conv=conv)
    table = st["table"]
    if case["op"] == "attend":
        a = hkv.hkv_mla_attend_args(
            layer=mla[1], n_seqs=case["seqs"], n_heads=case["heads"], value_width=_VALUES,
            dtype=types[case["dtype"]], cache_dtype=types[case["cache"]],
            max_blocks=table.shape[1], scale=st["scale"], cache_scale=st["cache_scale"],
            q=st["q"].data_ptr(), q_seq_stride=st["q"].stride(0), q_head_stride=st["q"].stride(1),
            block_table=table.data_ptr(), table_stride=table.stride(0),
            seq_lens=st["lens"].data_ptr(), out=st["out"].data_ptr(),
            out_seq_stride=st["out"].stride(0), out_head_stride=st["out"].stride(1),
            lse=st["lse"].data_ptr())
        res = dict(out=st["out"], lse=st["lse"])
        if case["weights"]:
            a.weights, a.weights_stride = st["weights"].data_ptr(), st["weights"].stride(0)
            res["weights"] = st["weights"]
        size = lay.mla_attend_workspace(a)
    else:
        a = hkv.hkv_mla_evict_args(
            n_seqs=case["seqs"], max_blocks=table.shape[1], budget=case["budget"],
            sinks=case["sinks"], recent=case["recent"], block_table=table.data_ptr(),
            table_stride=table.stride(0), seq_lens=st["lens"].data_ptr(),
            next_positions=st["next_positions"].data_ptr(), weights=st["weights"].data_ptr(),
            positions=st["positions"].data_ptr(), weights_out=st["weights_out"].data_ptr(),
            positions_out=st["positions_out"].data_ptr(), layer_stride=st["weights"].stride(0),
            seq_stride=st["weights"].stride(1), new_lens=st["new_lens"].data_ptr())
        a.set_layers(mla[:case["layers"]])
        cache = _TYPES[case["cache"]]
        rows = _mla_rows(st["pool"], g, torch.uint8 if cache.itemsize == 1 else cache)
        res = dict(rows=rows[:case["layers"]], weights=st["weights_out"],
                   positions=st["positions_out"], new_lens=st["new_lens"])
        size = lay.mla_evict_workspace(a)
    return lay, a, torch.empty(max(16, size), dtype=torch.uint8, device="cuda"), res


def _library(st):
    if "plan" not in st:
        st["plan"] = _plan(st)
    lay, a, ws, res = st["plan"]
    stream = torch.cuda.current_stream().cuda_stream
    pool = st["pool"].data_ptr()
    if ws is None:
        lay.kda_step(pool, a, stream)
    elif "weights_in" in st:
        # a pass adds to what earlier steps left: start from the same sums
        st["weights"].copy_(st["weights_in"])
        lay.mla_attend(pool, a, ws.data_ptr(), ws.numel(), stream)
    elif st["case"]["op"] == "attend":
        lay.mla_attend(pool, a, ws.data_ptr(), ws.numel(), stream)
    else:
        lay.mla_evict(pool, a, ws.data_ptr(), ws.numel(), stream)
    return res


def run(state):
    if own:
        return _library(state)
    op = state["case"]["op"]
    return (_plain_attend if op == "attend" else _plain_evict if op == "evict" else _plain_kda)(state)


# ---------------------------------------------------------------- work
def work(case):
    g = _geometry(case)
    if case["op"] == "kda":
        n, h, d, c = case["seqs"], g["heads"], g["head_dim"], g["conv_dim"]
        page = h * d * d * 4 + c * (_KERNEL - 1) * 2
        hits = n - (-(-n // 5) if case["misses"] else 0)
        extra = n * (c * 2 + h * d * 4 + h * 4 + 8 + h * d * 2) + c * _KERNEL * 2
        return {"bytes": (n + hits) * page + extra, "flops": n * (h * d * d * 7 + c * (2 * _KERNEL + 4))}
    lens = _lens(case)
    if case["op"] == "attend":
        n, h = len(lens), case["heads"]
        tokens = sum(lens)
        if case["holes"]:
            for x in lens:
                dropped = len(range(0, max(0, -(-x // g["n"]) - 1), 3))
                tokens -= dropped * g["n"]
        extra = n * h * (_WIDTH * 2 + _VALUES * 2 + 4) + (tokens * 8 if case["weights"] else 0)
        return {"bytes": tokens * g["row"] + extra, "flops": tokens * h * 2 * (_WIDTH + _VALUES)}
    k, b = case["layers"], case["budget"]
    over = [x for x in lens if x > b]
    moved = sum(b * (x - b) / x for x in over)
    return {"bytes": int(k * (sum(lens) * 16 + moved * 2 * g["row"])), "flops": int(k * sum(lens) * 4)}


# ---------------------------------------------------------------- 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    g = st["g"]
    if case["op"] == "kda":
        return _exact_kda(st, g)
    n_slots = sum(_lens(case))
    if case["op"] == "attend":
        return _exact_attend(st, g) if n_slots * case["heads"] <= 40000000 else None
    return _exact_evict(st, g) if n_slots * case["layers"] <= 2000000 else None


def _row_at(st, layer, s, lo, hi):
    """Stored rows [lo, hi) of one sequence (one block's part), or None."""
    g = st["g"]
    cache = _TYPES[st["case"]["cache"]]
    b = int(st["host_table"][s, lo // g["n"]])
    if b < 0:
        return None
    rows = _mla_rows(st["pool"], g, torch.uint8 if cache.itemsize == 1 else cache)[layer, b]
    return rows[lo % g["n"]:lo % g["n"] + hi - lo].contiguous().view(cache).double()


def _exact_attend(st, g):
    case, dev = st["case"], st["pool"].device
    st["host_table"] = st["table"].cpu().numpy()
    n, h = case["seqs"], case["heads"]
    out = torch.zeros(n, h, _VALUES, dtype=torch.float64, device=dev)
    lse = torch.full((n, h), -math.inf, dtype=torch.float64, device=dev)
    w = st["weights_in"].double() if case["weights"] else None
    for s, length in enumerate(_lens(case)):
        parts = [(lo, min(lo + g["n"], length)) for lo in range(0, length, g["n"])]
        parts = [(lo, hi, r) for lo, hi in parts if (r := _row_at(st, 1, s, lo, hi)) is not None]
        if not parts:
            continue
        rows = torch.cat([r for _, _, r in parts]) * st["cache_scale"]
        z = st["q"][s].double() @ rows.t().contiguous() * st["scale"]
        lse[s] = torch.logsumexp(z, 1)
        p = torch.exp(z - lse[s].unsqueeze(1))
        out[s] = p @ rows[:, :_VALUES].contiguous()
        if w is not None:
            sums, at = p.sum(0), 0
            for lo, hi, _ in parts:
                w[s, lo:hi] += sums[at:at + hi - lo]
                at += hi - lo
    res = dict(out=out, lse=lse)
    if w is not None:
        res["weights"] = w
    return res


def _exact_evict(st, g):
    case = st["case"]
    w, pos = st["weights"].cpu().numpy().astype(np.float64), st["positions"].cpu().numpy()
    nxt, lens = st["next_positions"].cpu().numpy(), _lens(case)
    wo, po = np.zeros_like(w), np.zeros_like(pos)
    for i in range(case["layers"]):
        for s, length in enumerate(lens):
            new = min(length, case["budget"])
            held = [p < case["sinks"] or p >= nxt[s] - case["recent"] for p in pos[i, s, :length].tolist()]
            by = sorted(range(length), key=lambda t: (not held[t], 0.0 if held[t] else -w[i, s, t], t))
            keep = set(by[:new])
            movers = iter(sorted(t for t in keep if t >= new))
            for t in range(length):
                a = t if t in keep else next(movers) if t < new else None
                if t >= new:
                    wo[i, s, t], po[i, s, t] = 0.0, -1
                else:
                    wo[i, s, t], po[i, s, t] = w[i, s, a], pos[i, s, a]
    return dict(rows=None, weights=wo, positions=po, new_lens=np.minimum(lens, case["budget"]).astype(np.int32))


def _exact_kda(st, g):
    dt = _TYPES[st["case"]["dtype"]]
    conv, rec = (x.double() for x in _kda_pages(st["pool"], g, dt))
    h, d = g["heads"], g["head_dim"]
    n = st["x"].shape[0]
    out = torch.zeros(n, h * d, dtype=torch.float64, device=rec.device)
    src, dst = st["src"].tolist(), st["dst"].tolist()
    weight = st["conv_weight"].double()
    for s in range(n):
        taps = torch.zeros_like(conv[0]) if src[s] < 0 else conv[src[s]]
        taps = torch.cat([taps, st["x"][s].double().unsqueeze(1)], 1)
        y = (taps * weight).sum(1)
        y = (y / (1 + torch.exp(-y))).view(3, h, d)
        q = y[0] / torch.sqrt((y[0] ** 2).sum(1, keepdim=True) + 1e-6) * d ** -0.5
        k = y[1] / torch.sqrt((y[1] ** 2).sum(1, keepdim=True) + 1e-6)
        state = torch.zeros_like(rec[0]) if src[s] < 0 else rec[src[s]]
        state = torch.exp(st["log_decay"][s].double()).view(h, d, 1) * state
        seen = torch.matmul(k.unsqueeze(1), state).squeeze(1)
        delta = st["beta"][s].double().unsqueeze(1) * (y[2] - seen)
        state = state + k.unsqueeze(2) * delta.unsqueeze(1)
        out[s] = torch.matmul(q.unsqueeze(1), state).reshape(-1)
        rec[dst[s]], conv[dst[s]] = state, taps[:, 1:]
    return dict(out=out, recurrent=rec, conv=conv)
