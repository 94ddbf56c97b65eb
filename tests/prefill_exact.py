"""hkv_kda_prefill against the definition in 64 bits, with bounds as tight as fp32's:
column by column in norm, and by element for outputs that cancel.

A token (or a chunk of them) brings an error of at most E (|s_j| + 2 |v_j|) into column
j of a state (v only where beta lets it in), E = 2^-19: its products take operands that are off by at most 2^-21 each
(two fp16 terms, without the product of the low ones) or 2^-24, and its sums are fp32.
Errors of different tokens are independent, so their squares add up, and a token's
decays shrink what came before it by at least the largest of them: |M_t| <= max a_t."""
import torch

from tests.pool_cases import half_step

E = 2.0 ** -19


def columns(x):
    """[..., rows, columns] -> norms of the columns."""
    return (x * x).sum(-2).sqrt()


def follow(c, join=None):
    """The case's states behind the tokens that end a block or a run, by block, and its
    outputs by row, each with its tolerance: {block: (state, tol of a column)},
    {row: (out, tol of an element)}.  On c.x's device.  `join` = (token, factor): a mistake
    for tests of the checks, a state that goes on as `factor` times itself."""
    dev, h, d, n = c.x.device, c.heads, c.d, c.pool.n
    conv, rec, wt = c.conv().clone(), c.rec().clone(), c.weight.double()
    states, outs = {}, {}
    for s, tokens in enumerate(c.new):
        if tokens == 0 or s in c.ignored or s in c.refused:
            continue
        row0, src = int(c.starts[s]), int(c.src[s])
        old = conv[src].double() if src >= 0 else torch.zeros_like(conv[0], dtype=torch.float64)
        state = rec[src].double() if src >= 0 else torch.zeros(h, d, d, dtype=torch.float64, device=dev)
        win = torch.cat([old.t(), c.x[row0:row0 + tokens].double()]).unfold(0, c.taps, 1)
        y = (win * wt).sum(2)
        y = (y / (1 + torch.exp(-y))).view(tokens, 3, h, d)
        norm = torch.sqrt((y[:, :2] ** 2).sum(3, keepdim=True) + c.eps)
        q, k, v = y[:, 0] / norm[:, 0] * c.scale, y[:, 1] / norm[:, 1], y[:, 2]
        a = torch.exp(c.log_decay[row0:row0 + tokens].double().clamp(max=0)).view(tokens, h, d)
        most = a.amax(2, keepdim=True)
        qn = q.norm(dim=2, keepdim=True)
        beta = c.beta[row0:row0 + tokens].double().unsqueeze(2)
        err2 = torch.zeros(h, d, dtype=torch.float64, device=dev)
        for t in range(tokens):
            size, new = columns(state), 2 * v[t].abs()
            state = a[t].unsqueeze(2) * state
            u = beta[t] * (v[t] - (k[t].unsqueeze(2) * state).sum(1))
            state = state + k[t].unsqueeze(2) * u.unsqueeze(1)
            err2 = (most[t] ** 2) * err2 + (E * (size + new * (beta[t] != 0))) ** 2
            o = (q[t].unsqueeze(2) * state).sum(1)
            tol = qn[t] * (err2.sqrt() + E * (size + new + columns(state)))
            outs[row0 + t] = (o.reshape(-1), (tol + half_step(c.dt) * (o.abs() + tol)).reshape(-1)
                              + torch.finfo(c.dt).tiny)
            p = c.at[s] + t
            if (p + 1) % n == 0 or t == tokens - 1:
                b = int(c.table[s, p // n])
                if b >= 0:
                    states[b] = state.clone(), err2.sqrt() + E * columns(state)
            if join is not None and t == join[0]:
                state = state * join[1]
    return states, outs


def state_errors(got, want):
    """How far each column of the states is off, in units of its tolerance."""
    return torch.stack([columns(got[b].double() - w) / tol for b, (w, tol) in want.items()])


def check(c, outs=True):
    """Runs the case and checks it."""
    states, rows = follow(c)
    c.enqueue()
    torch.cuda.synchronize()
    off = state_errors(c.rec(), states)
    assert (off <= 1).all(), float(off.max())
    if outs:
        want, tol = (torch.stack([r[i] for r in rows.values()]) for i in (0, 1))
        got = c.out[torch.tensor(list(rows), device=c.out.device)].double()
        over = (got - want).abs() / tol
        assert (over <= 1).all(), float(over.max())
    return float(off.max())
