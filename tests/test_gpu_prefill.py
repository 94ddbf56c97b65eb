"""The KDA layers' prompt form on the pool's state pages (hkv_kda_prefill)
against the definition in 64 bits."""
import math

import numpy as np
import pytest
import torch

import retrieve_store_chunk_amd as hkv
from tests.pool_cases import stream
from tests.prefill_cases import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_head_dims_and_types(d, dtype):
    Case([5, 1, 0, 70, 130], at=[0, 3, 0, 40, 0], src=["other", "other", None, "own", None], heads=2, d=d,
         dtype=dtype, seed=d, path=d // 16 % 2, lead=3, tail=5).run()


@pytest.mark.parametrize("taps", [1, 2, 3, 4, 5, 8])
def test_conv_kernels(taps):
    """Taps from the source's page, from the call's rows, and from both."""
    Case([1, 2, 40, 90], heads=1, taps=taps, seed=taps).run()
    Case([1, 3, 33], src=["own", None, "own"], at=[5, 0, 20], heads=2, d=64, taps=taps, seed=taps).run()


@pytest.mark.parametrize("heads", [1, 6, 32])
def test_heads(heads):
    Case([66], heads=heads, seed=heads, path=1).run()


@pytest.mark.parametrize("tokens", [1, 2, 15, 16, 17, 31, 32, 33, 47, 48, 49, 63, 64, 65, 127, 128, 129, 200])
def test_lengths(tokens):
    Case([tokens], heads=1, seed=tokens).run()
    Case([tokens, tokens], at=[7, 0], src=["own", None], heads=1, seed=tokens, dtype="fp16").run()


@pytest.mark.parametrize("at", [0, 1, 5, 159, 160, 161])
@pytest.mark.parametrize("d", [64, 128])
def test_snapshots_at_block_ends(at, d):
    """Blocks that end between a chunk's tokens, at its end, and several in one run."""
    c = Case([1, 159, 160, 161, 400], at=[at] * 5, src=["other", "own", None, "other", "own"], heads=1, d=d, seed=at,
             block_size=160)
    c.run()


def test_snapshots_that_are_not_kept():
    Case([700, 300], at=[100, 0], heads=1, block_size=160, null=[(0, 1), (0, 2), (1, 1)], seed=3).run()
    Case([40], heads=1, null=[(0, 0)], seed=4).run()


def test_the_smallest_blocks():
    """Blocks smaller than a chunk."""
    Case([50, 33, 1, 16], at=[3, 0, 15, 16], heads=1, d=16, block_size=16, seed=5).run()


def test_the_source_may_be_a_later_block_of_its_own():
    c = Case([400], at=[0], heads=1, block_size=160, seed=6)
    c.src[0] = c.table[0, 2]
    c.upload()
    c.run()


def test_one_source_for_several_sequences():
    c = Case([70, 30, 90], heads=2, seed=7)
    c.src[:] = c.src[0]
    c.upload()
    c.run()


def test_bad_ids_are_refused():
    c = Case([70, 5, 90, 30, 40, 33], heads=1, block_size=160, seed=8)
    c.src[0], c.src[1] = c.pool.blocks, -2
    c.table[2, 0], c.table[3, 0] = c.pool.blocks, -3
    c.refused = {0, 1, 2, 3}
    c.upload()
    c.run()


def test_clashing_blocks_are_refused():
    c = Case([200, 200, 200, 200, 90, 10], heads=1, block_size=160, seed=9)
    c.table[1, 1] = c.table[0, 0]   # 0 and 1 write one block
    c.src[3] = c.table[2, 1]        # 2 would write what 3 reads; 3 may go on
    c.refused = {0, 1, 2}
    c.upload()
    c.run()
    c = Case([700, 40], heads=1, block_size=160, seed=10)
    c.table[0, 3] = c.table[0, 1]   # named twice by its own table
    c.refused = {0}
    c.upload()
    c.run()


def test_bad_lengths_and_positions_are_refused():
    c = Case([70, 70, 70, 40], heads=1, block_size=160, seed=11)
    c.at[0], c.at[1] = -1, 91       # 161 tokens in a table of 160
    c.refused = {0, 1}
    c.upload()
    c.run()
    c = Case([70, 30, 90], heads=1, seed=12)
    c.most = 70
    c.refused = {2}
    c.run()


def test_bad_starts_leave_their_sequences():
    c = Case([20, 30, 40, 50], heads=1, seed=13, tail=8)
    c.starts[:] = [0, 20, 10, 50, 100]
    # 1 goes backwards; 2 begins before 1 did, in rows that may be another's
    c.ignored = {1, 2}
    c.new[3] = 50
    c.upload()
    c.run()
    c = Case([20, 30], heads=1, seed=14, tail=8)
    c.starts[:] = [-1, 20, 59]      # before the first row, past the last
    c.ignored = {0, 1}
    c.upload()
    c.run()


@pytest.mark.parametrize("decay", [0.0, 5.0, 60.0, 300.0])
@pytest.mark.parametrize("tokens", [10, 150])
def test_decays(decay, tokens):
    """From none to states that vanish at once."""
    Case([tokens], heads=2, seed=15, decay=decay).run()


@pytest.mark.parametrize("tokens", [10, 100])
def test_decays_of_infinity_and_above_zero(tokens):
    c = Case([tokens], heads=2, seed=16)
    c.log_decay[3] = -math.inf            # a token that forgets everything
    c.log_decay[5, 7] = -math.inf
    c.log_decay[tokens - 2, ::3] = -math.inf
    c.log_decay[4, ::2] = 3.0             # counts as 0
    c.run()


@pytest.mark.parametrize("tokens", [10, 100])
def test_betas(tokens):
    for beta in ((0.0, 0.0), (1.0, 1.0), (2.0, 2.0), (0.0, 2.0)):
        Case([tokens], heads=1, seed=17, beta=beta, decay=0.2).run()


@pytest.mark.parametrize("tokens", [10, 100])
def test_the_same_key_again_and_again(tokens):
    """The system of a chunk at its worst: every key repeats the one before."""
    for beta in ((1.0, 1.0), (2.0, 2.0), (0.5, 1.0)):
        c = Case([tokens], heads=1, seed=18, decay=0.0, beta=beta)
        c.x[:, 128:256] = c.x[:1, 128:256]
        c.run()


@pytest.mark.parametrize("tokens", [10, 100])
def test_zeros(tokens):
    c = Case([tokens], heads=1, seed=19)
    c.x.zero_()
    c.conv().zero_()
    c.run()                               # q = k = v = 0: eps alone
    c = Case([tokens], heads=1, seed=20)
    c.x[:, 128:256] = 0                   # keys alone
    c.run()


@pytest.mark.parametrize("power", [-100, -40, 40, 100])
@pytest.mark.parametrize("tokens", [10, 150])
def test_values_of_any_size(power, tokens):
    """Columns of very different sizes stand side by side, each with its own
    precision; states as large and as small."""
    c = Case([tokens, tokens], heads=1, seed=21, src=["other", None], dtype="bf16")
    size = torch.ones(128, device="cuda")
    size[::3] = 2.0 ** power
    c.weight[256:] = (c.weight[256:].float() * size.unsqueeze(1)).to(c.dt)
    c.rec().mul_(size)
    if power < 0:
        c.x[:, 256:] = c.x[:, 256:].abs()  # silu of a tiny value is half of it
    want = c.expect()
    c.enqueue()
    c.compare(want)


def test_states_that_grow_and_fall_within_a_run():
    """Values that jump by 2^60 from one stretch of tokens to the next and back."""
    c = Case([330], heads=1, seed=22, dtype="bf16", decay=3.0)
    for lo, power in ((0, -30), (70, 30), (140, 0), (200, 60), (270, -60)):
        c.x[lo:lo + 70, 256:] = (c.x[lo:lo + 70, 256:].float().abs() * 2.0 ** power).to(c.dt)
    c.run()


def test_infinities_stay_in_their_column_and_sequence():
    for tokens in (10, 100):
        c = Case([tokens, tokens], heads=2, seed=23)
        c.rec()[int(c.src[0]), 0, 3, 5] = math.inf
        c.enqueue()
        torch.cuda.synchronize()
        out = c.out.float().cpu().view(2, tokens, 2, 128)
        assert not out[0, :, 0, 5].isfinite().any()
        out[0, :, 0, 5] = 0
        assert out.isfinite().all()
        c = Case([tokens, tokens], heads=2, seed=24)
        c.x[tokens // 2, 9] = math.nan    # a query of head 0: its own token, and the next three by the conv
        c.enqueue()
        torch.cuda.synchronize()
        out = c.out.float().cpu().view(2, tokens, 2, 128)
        assert out[0, tokens // 2, 0].isnan().all()
        assert out[0, :, 1].isfinite().all() and out[1].isfinite().all()
        last = c.rec()[int(c.table[0, 0])]
        assert last.isfinite().all()      # a query never reaches the state


def test_strides():
    c = Case([70, 9], heads=2, d=64, seed=25)
    hd, tokens = 128, 79
    x = torch.full((tokens, 3 * hd + 5), 9.0, dtype=c.dt, device="cuda")  # rows at odd elements
    x[:, 3:3 * hd + 3] = c.x
    c.x = x[:, 3:3 * hd + 3]
    g = torch.full((tokens, hd + 3), 9.0, device="cuda")
    g[:, 1:hd + 1] = c.log_decay
    c.log_decay = g[:, 1:hd + 1]
    c.beta = torch.cat([c.beta, c.beta], 1)[:, :2]
    out = torch.full((tokens, hd + 12), 7.0, dtype=c.dt, device="cuda")
    c.out = out[:, :hd]
    c.run()
    assert (out[:, hd:] == 7.0).all()
    c = Case([70], heads=1, seed=26)      # the same row for all tokens
    c.x, c.log_decay, c.beta = (v[:1].expand(70, v.shape[1]) for v in (c.x, c.log_decay, c.beta))
    c.run()


def test_as_the_step_does_it():
    """Against hkv_kda_step from token to token, within twice the definition's bounds."""
    c = Case([90, 7], at=[0, 30], heads=2, seed=27)
    res, pool, _ = c.expect()
    c.enqueue()
    torch.cuda.synchronize()
    mine, c.pool.bytes = c.pool.bytes, pool.clone()
    outs = {}
    for t in range(90):
        live = [s for s in range(2) if t < c.new[s]]
        rows = torch.tensor([int(c.starts[s]) + t for s in live], device="cuda")
        dst = torch.tensor([int(c.table[s, 0]) for s in live], dtype=torch.int32, device="cuda")
        src = dst if t else torch.tensor([int(c.src[s]) for s in live], dtype=torch.int32, device="cuda")
        x, g, b = c.x[rows], c.log_decay[rows], c.beta[rows]
        out = torch.empty(len(live), c.out.shape[1], dtype=c.dt, device="cuda")
        c.pool.layout.kda_step(c.pool.ptr, hkv.hkv_kda_step_args(
            layer=c.layer, n_seqs=len(live), dtype=c.dt_id, scale=c.scale, eps=c.eps, x=x.data_ptr(),
            x_stride=x.stride(0), conv_weight=c.weight.data_ptr(), log_decay=g.data_ptr(),
            decay_stride=g.stride(0), beta=b.data_ptr(), beta_stride=b.stride(0), src_blocks=src.data_ptr(),
            dst_blocks=dst.data_ptr(), out=out.data_ptr(), out_stride=out.stride(0)), stream())
        torch.cuda.synchronize()
        for i, r in enumerate(rows.tolist()):
            outs[r] = out[i].cpu().double()
    step_rec, step_conv = c.rec().cpu().double(), c.conv().cpu()
    c.pool.bytes = mine
    for r, (o, tol) in res["out"].items():
        assert (c.out[r].cpu().double() - outs[r]).abs().le(2 * tol).all(), r
    for b, (_, tol) in res["rec"].items():
        assert (c.rec()[b].cpu().double() - step_rec[b]).abs().le(2 * tol).all()
        assert torch.equal(c.conv()[b].cpu(), step_conv[b])


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_precision_of_long_runs(dtype):
    """Errors of single tokens are independent and forgotten with the state: in
    norm they stay near one token's.  A token's operands are off by at most 2^-21
    (two fp16 terms) to 2^-24, three of them meet in a product, and a state that
    remembers about 60 tokens adds up sqrt(60) of such errors at worst: 2^-21 x 3 x 8
    = 1.1e-5; outputs are rounded on top of that."""
    c = Case([1500], heads=1, dtype=dtype, seed=28, block_size=480)
    want = c.expect()
    c.enqueue()
    c.compare(want)
    out, rec = c.errors(want)
    assert rec < 1.1e-5
    assert out < 1.1e-5 + torch.finfo(c.dt).eps / 2


def test_the_same_call_twice_gives_the_same_bits():
    c = Case([100, 3, 64], heads=3, seed=29)
    before = c.pool.bytes.clone()
    c.enqueue()
    torch.cuda.synchronize()
    out, pool = c.out.clone(), c.pool.bytes.clone()
    c.pool.bytes.copy_(before)
    c.out.zero_()
    c.workspace.zero_()
    c.enqueue()
    torch.cuda.synchronize()
    assert torch.equal(out, c.out) and torch.equal(pool, c.pool.bytes)


def test_captured_and_replayed():
    """One captured call follows starts, positions, sources and tables."""
    c = Case([100, 40, 20], at=[0, 20, 0], heads=2, seed=30, tail=30, block_size=160)
    c.most = 190
    before = c.pool.bytes.clone()
    c.enqueue()
    torch.cuda.synchronize()
    g, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(g, stream=s):
        c.enqueue()
    for new, at, null in (([100, 40, 20], [0, 20, 0], False), ([1, 1, 1], [60, 59, 3], True),
                          ([0, 150, 3], [0, 10, 159 - 3], False), ([190, 0, 0], [0, 0, 0], True)):
        c.pool.bytes.copy_(before)
        c.new, c.at = list(new), list(at)
        c.starts = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        if at[0] == 0 and new[0] == 190:
            c.at[0], c.refused = 0, {0}   # past its table of one block
        src = c.src.copy()
        if null:
            src[1] = -1
        c.src, kept = src, c.src
        for t, v in ((c.d_starts, c.starts), (c.d_at, c.at), (c.d_src, c.src)):
            t.copy_(torch.from_numpy(np.array(v, np.int32)))
        c.out.fill_(7.0)
        torch.cuda.synchronize()
        want = c.expect()
        g.replay()
        c.compare(want)
        c.src, c.refused = kept, set()


def test_two_streams_at_once():
    cs = [Case([90, 200], heads=8, seed=31), Case([300], heads=2, d=64, seed=32, dtype="fp16")]
    want = [c.expect() for c in cs]
    for c in cs:
        c.workspace = torch.full((c.pool.layout.kda_prefill_workspace(c.args()),), 0xFF, dtype=torch.uint8,
                                 device="cuda")
    ss = [torch.cuda.Stream() for _ in cs]
    torch.cuda.synchronize()
    for c, s in zip(cs, ss):
        c.enqueue(s.cuda_stream)
    for c, w in zip(cs, want):
        c.compare(w)


def test_calls_share_a_workspace_one_after_another():
    cs = [Case([130], heads=4, seed=33), Case([20, 70, 5], heads=1, seed=34), Case([65] * 9, heads=2, seed=35)]
    size = max(c.pool.layout.kda_prefill_workspace(c.args()) for c in cs)
    ws = torch.full((size,), 0xFF, dtype=torch.uint8, device="cuda")
    want = [c.expect() for c in cs]
    for c in cs:
        c.workspace = ws
        c.enqueue()
    for c, w in zip(cs, want):
        c.compare(w)


def test_many_sequences():
    """Short and long ones side by side."""
    new = [(i * 5) % 4 for i in range(150)]
    new[10], new[77], new[149] = 90, 130, 66
    Case(new, src=[None if i % 4 == 0 else "other" for i in range(150)], heads=1, d=64, seed=36, block_size=96).run()


@pytest.mark.parametrize("heads", [1, 3, 16])
def test_long_runs_in_parts(heads):
    """Few heads and long runs: what parts of a run make of a state is joined."""
    Case([1300], heads=heads, seed=37, block_size=960 if heads == 16 else 480, at=[100], src=["own"]).run()


def test_parts_beside_short_runs():
    Case([1250, 0, 700, 3, 90, 1], at=[0, 5, 300, 0, 200, 7], src=["other", "other", None, "own", "own", None],
         heads=2, seed=38, block_size=320, null=[(0, 1), (2, 2)], lead=1, tail=9).run()


def test_parts_with_strong_and_no_decays():
    for decay, beta in ((0.0, (0.0, 2.0)), (40.0, (0.0, 1.0)), (0.0, (2.0, 2.0))):
        Case([1400], heads=1, seed=39, decay=decay, beta=beta).run()
    c = Case([1400], heads=1, seed=40, decay=0.05)
    c.log_decay[500] = -math.inf
    c.run()


def test_parts_of_refused_runs():
    c = Case([1300, 1250, 600, 40], heads=1, block_size=320, seed=41)
    c.src[0] = c.pool.blocks
    c.table[2, 1] = c.table[3, 0]
    c.refused = {0, 2, 3}
    c.upload()
    c.run()


def test_parts_keep_infinities_in_their_column():
    c = Case([1300], heads=2, seed=42)
    c.rec()[int(c.src[0]), 0, 3, 5] = math.inf
    c.enqueue()
    torch.cuda.synchronize()
    out = c.out.float().cpu().view(1300, 2, 128)
    assert not out[:, 0, 5].isfinite().any()
    out[:, 0, 5] = 0
    assert out.isfinite().all()


def test_many_pairs():
    """Enough heads that a workgroup scans two column tiles."""
    Case([70, 5, 130, 64], heads=12, seed=43, lead=2, tail=3).run()


def test_parts_captured_and_replayed():
    """A captured call whose lengths change: parts that were full are empty, and back."""
    c = Case([1300, 60], at=[0, 30], heads=1, seed=44, block_size=320, tail=200)
    for a in (c.x, c.log_decay, c.beta):
        a[1360:] = a[:200]
    before = c.pool.bytes.clone()
    g, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    c.enqueue()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=s):
        c.enqueue()
    for new in ([1300, 60], [30, 100], [700, 10], [1300, 200]):
        c.pool.bytes.copy_(before)
        c.new = list(new)
        c.starts = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        c.d_starts.copy_(torch.from_numpy(c.starts))
        c.out.fill_(7.0)
        torch.cuda.synchronize()
        want = c.expect()
        g.replay()
        c.compare(want)


def test_strides_of_chunks():
    """Rows at odd elements, one row for all, padded outputs, where runs go in chunks."""
    c = Case([90, 9], heads=2, seed=45)
    hd, tokens = 256, 99
    x = torch.full((tokens, 3 * hd + 5), 9.0, dtype=c.dt, device="cuda")
    x[:, 3:3 * hd + 3] = c.x
    c.x = x[:, 3:3 * hd + 3]
    g = torch.full((tokens, hd + 3), 9.0, device="cuda")
    g[:, 1:hd + 1] = c.log_decay
    c.log_decay = g[:, 1:hd + 1]
    c.beta = torch.cat([c.beta, c.beta], 1)[:, :2]
    out = torch.full((tokens, hd + 12), 7.0, dtype=c.dt, device="cuda")
    c.out = out[:, :hd]
    table = torch.full((2, 5), 0x7FFFFFFF, dtype=torch.int32, device="cuda")
    table[:, :c.columns] = c.d_table
    c.d_table = table
    c.run()
    assert (out[:, hd:] == 7.0).all()


def test_records_past_4_gib():
    """One call whose workspace passes 2^32 bytes against two calls that follow each
    other, cut where a block ends, so that both have the same chunks."""
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("needs 24 GiB")
    heads, n = 32, 1888
    first, second = 17 * n, 18 * n
    c = Case([8], heads=heads, seed=46, block_size=n, spare=3)
    hd, tokens = heads * 128, first + second
    gen = torch.Generator(device="cuda").manual_seed(46)
    c.x = torch.randn(tokens, 3 * hd, device="cuda", generator=gen, dtype=c.dt)
    c.log_decay = -torch.rand(tokens, hd, device="cuda", generator=gen) ** 3
    c.beta = torch.rand(tokens, heads, device="cuda", generator=gen)
    c.out = torch.zeros(tokens, hd, dtype=c.dt, device="cuda")
    c.columns = 35
    end, cut = int(c.table[0, 0]), [b for b in range(c.pool.blocks) if b not in (c.table[0, 0], c.src[0])][0]
    c.table = np.full((1, 35), -1, np.int32)   # only two snapshots are kept
    c.table[0, 16], c.table[0, 34] = cut, end
    before = c.pool.bytes.clone()

    def call(at, rows, src):
        c.at, c.src, c.starts, c.most = [at], np.array([src]), np.array(rows), rows[1] - rows[0]
        c.new = [c.most]
        c.upload()
        c.enqueue()
        torch.cuda.synchronize()

    src = int(c.src[0])
    call(0, [0, tokens], src)
    assert c.workspace.numel() > 1 << 32
    out, pool = c.out.clone(), c.pool.bytes.clone()
    c.pool.bytes.copy_(before)
    c.out.zero_()
    call(0, [0, first], src)
    call(first, [first, tokens], cut)
    mine, c.pool.bytes = c.pool.bytes, pool
    states = [c.rec()[b].double() for b in (cut, end)]
    c.pool.bytes = mine
    for want, b in zip(states, (cut, end)):
        got = c.rec()[b].double()
        assert float((got - want).norm() / want.norm()) < 2e-6, b   # two states' 2^-20 each
    off = (c.out.double() - out.double()).norm() / out.double().norm()
    assert float(off) < 2.0 ** -9
