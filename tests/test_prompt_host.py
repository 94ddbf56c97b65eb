"""Host-side checks of the operators that bring new tokens into the pool (no GPU
needed): argument validation rejects bad calls before any HIP call, workspace
sizes, and what the header says."""
import os
import re

import pytest

import retrieve_store_chunk_amd as hkv
import workloads as W
from tests.test_ops_host import POOL, WS, layout, needs_no_gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def append_args(**kw):
    a = dict(layer=2, n_seqs=3, n_tokens=20, n_heads=8, dtype=hkv.HKV_BF16, cache_dtype=hkv.HKV_BF16,
             latent_width=512, rotary_dim=64, rotary_halves=0, n_positions=100, max_blocks=4,
             eps=1e-6, cache_scale=1.0, kv=0x1000000, kv_stride=576, norm_weight=0x1100000,
             cos_sin=0x1200000, positions=0x1300000, seq_starts=0x1400000, seq_lens=0x1500000,
             block_table=0x1600000, table_stride=4, q_in=0x2000000, q_in_token_stride=8 * 64,
             q_in_head_stride=64, q_out=0x3000000, q_out_token_stride=8 * 576, q_out_head_stride=576)
    a.update(kw)
    return hkv.hkv_mla_append_args(**a)


def prefill_args(**kw):
    a = dict(layer=0, n_seqs=3, n_tokens=20, max_seq_tokens=20, max_blocks=4, dtype=hkv.HKV_BF16,
             scale=0.25, eps=1e-6, x=0x1000000, x_stride=96, conv_weight=0x2000000,
             log_decay=0x3000000, decay_stride=32, beta=0x4000000, beta_stride=2,
             seq_starts=0x5000000, positions=0x5100000, src_blocks=0x5200000, block_table=0x5300000,
             table_stride=4, out=0x7000000, out_stride=32)
    a.update(kw)
    return hkv.hkv_kda_prefill_args(**a)


def append_status(lay, pool=POOL, **kw):
    return hkv.status_of(lay.mla_append, pool, append_args(**kw), 0)


def prefill_status(lay, pool=POOL, ws=WS, ws_bytes=1 << 40, **kw):
    return hkv.status_of(lay.kda_prefill, pool, prefill_args(**kw), ws, ws_bytes, 0)


@needs_no_gpu
@pytest.mark.parametrize("bad,status", [
    (dict(layer=0), "ARG"), (dict(layer=5), "ARG"), (dict(n_seqs=-1), "ARG"), (dict(n_seqs=65536), "ARG"),
    (dict(n_tokens=-1), "ARG"), (dict(n_tokens=(1 << 20) + 1), "ARG"), (dict(n_heads=-1), "ARG"),
    (dict(n_heads=129), "ARG"), (dict(seq_starts=0), "ARG"), (dict(dtype=hkv.HKV_FP32), "ARG"),
    (dict(cache_dtype=hkv.HKV_FP16), "ARG"), (dict(cache_dtype=hkv.HKV_E4M3), "ARG"),
    (dict(latent_width=-8), "ARG"), (dict(latent_width=508), "ARG"), (dict(latent_width=520), "ARG"),
    (dict(rotary_dim=-16), "ARG"), (dict(rotary_dim=72), "ARG"), (dict(rotary_dim=592), "ARG"),
    (dict(rotary_halves=2), "ARG"), (dict(n_positions=-1), "ARG"), (dict(max_blocks=0), "ARG"),
    (dict(max_blocks=2**31 - 1), "ARG"), (dict(table_stride=-1), "ARG"), (dict(eps=-1.0), "ARG"),
    (dict(eps=float("nan")), "ARG"), (dict(cache_scale=0.0), "ARG"), (dict(cache_scale=-1.0), "ARG"),
    (dict(cache_scale=float("inf")), "ARG"), (dict(kv=0), "ARG"), (dict(cos_sin=0), "ARG"),
    (dict(positions=0), "ARG"), (dict(seq_lens=0), "ARG"), (dict(block_table=0), "ARG"),
    (dict(q_in=0), "ARG"), (dict(q_out=0), "ARG"), (dict(kv_stride=-8), "ARG"),
    (dict(q_in_head_stride=-8), "ARG"), (dict(q_out_token_stride=2**60), "ARG"), (dict(pool=0), "ARG"),
    (dict(kv=0x1000008), "ALIGN"), (dict(norm_weight=0x1100002), "ALIGN"), (dict(cos_sin=0x1200004), "ALIGN"),
    (dict(positions=0x1300002), "ALIGN"), (dict(seq_starts=0x1400001), "ALIGN"),
    (dict(seq_lens=0x1500002), "ALIGN"), (dict(block_table=0x1600002), "ALIGN"),
    (dict(q_in=0x2000002), "ALIGN"), (dict(q_out=0x3000008), "ALIGN"), (dict(kv_stride=580), "ALIGN"),
    (dict(q_in_token_stride=513), "ALIGN"), (dict(q_out_head_stride=578), "ALIGN"), (dict(pool=POOL + 8), "ALIGN"),
    (dict(q_out_head_stride=56), "ALIAS"), (dict(q_out_token_stride=0), "ALIAS"), (dict(q_out=0x2000010), "ALIAS"),
    (dict(q_out=0x2000000), "ALIAS"), (dict(q_out=0x1000000), "ALIAS"), (dict(q_out=0x1300000), "ALIAS"),
    (dict(kv=POOL), "ALIAS"), (dict(q_out=POOL + 4096), "ALIAS"), (dict(block_table=POOL), "ALIAS"),
])
def test_append_refusals(bad, status):
    lay = layout()
    assert append_status(lay, **bad) == getattr(hkv, "HKV_E_" + status), hkv.hkv_last_error()
    assert hkv.hkv_last_error()


@needs_no_gpu
def test_append_layout_refusals():
    narrow = dict(latent_width=0, rotary_dim=0, n_heads=0)
    assert append_status(layout(mla_width=24), **narrow) == hkv.HKV_E_ARG
    assert append_status(layout(mla_width=1040), **narrow) == hkv.HKV_E_ARG
    assert append_status(layout(mla_bytes=4)) == hkv.HKV_E_ARG
    assert append_status(layout(mla_bytes=1)) == hkv.HKV_E_ARG  # cache_dtype is bf16
    odd = layout(path=1, conv_dim=5, kv_group_of_layer=[0, 0, 0, 0, 0])
    assert odd.layers[2]["pool_offset"] % 16
    assert append_status(odd) == hkv.HKV_E_ALIGN


@needs_no_gpu
@pytest.mark.parametrize("bad,status", [
    (dict(layer=2), "ARG"), (dict(layer=-1), "ARG"), (dict(n_seqs=-1), "ARG"), (dict(n_seqs=4097), "ARG"),
    (dict(n_tokens=-1), "ARG"), (dict(n_tokens=(1 << 20) + 1), "ARG"), (dict(max_seq_tokens=-1), "ARG"),
    (dict(max_blocks=0), "ARG"), (dict(max_blocks=2**31 - 1), "ARG"), (dict(table_stride=-1), "ARG"),
    (dict(dtype=hkv.HKV_FP32), "ARG"), (dict(dtype=hkv.HKV_E4M3), "ARG"), (dict(scale=float("nan")), "ARG"),
    (dict(eps=-1e-6), "ARG"), (dict(x=0), "ARG"), (dict(conv_weight=0), "ARG"), (dict(log_decay=0), "ARG"),
    (dict(beta=0), "ARG"), (dict(seq_starts=0), "ARG"), (dict(positions=0), "ARG"), (dict(src_blocks=0), "ARG"),
    (dict(block_table=0), "ARG"), (dict(out=0), "ARG"), (dict(pool=0), "ARG"), (dict(x_stride=-1), "ARG"),
    (dict(decay_stride=2**60), "ARG"), (dict(beta_stride=-1), "ARG"), (dict(out_stride=28), "ALIAS"),
    (dict(out_stride=-32), "ALIAS"), (dict(out_stride=34), "ALIGN"), (dict(out=0x7000008), "ALIGN"),
    (dict(x=0x1000001), "ALIGN"), (dict(conv_weight=0x2000001), "ALIGN"), (dict(log_decay=0x3000002), "ALIGN"),
    (dict(seq_starts=0x5000002), "ALIGN"), (dict(positions=0x5100001), "ALIGN"),
    (dict(block_table=0x5300002), "ALIGN"), (dict(pool=POOL + 8), "ALIGN"), (dict(ws=WS + 4), "ALIGN"),
    (dict(out=0x1000000), "ALIAS"), (dict(out=0x5000000), "ALIAS"), (dict(x=POOL + 64), "ALIAS"),
    (dict(ws=0x1000000), "ALIAS"), (dict(ws=POOL), "ALIAS"), (dict(ws=0), "WORKSPACE"),
    (dict(ws_bytes=8), "WORKSPACE"),
])
def test_prefill_refusals(bad, status):
    lay = layout()
    ws_bytes = bad.pop("ws_bytes", lay.kda_prefill_workspace(prefill_args()))
    assert prefill_status(lay, ws_bytes=ws_bytes, **bad) == getattr(hkv, "HKV_E_" + status), hkv.hkv_last_error()
    assert hkv.hkv_last_error()


@needs_no_gpu
def test_prefill_layout_refusals():
    assert prefill_status(layout(head_dim=40, conv_dim=240)) == hkv.HKV_E_ARG
    assert prefill_status(layout(conv_dim=95)) == hkv.HKV_E_ARG
    assert prefill_status(layout(conv_kernel=9)) == hkv.HKV_E_ARG
    assert prefill_status(layout(state_bytes=2)) == hkv.HKV_E_ARG
    assert prefill_status(layout(conv_bytes=4)) == hkv.HKV_E_ARG  # wants fp32
    assert prefill_status(layout(conv_bytes=1)) == hkv.HKV_E_ARG


@needs_no_gpu
def test_empty_calls_do_nothing():
    lay = layout()
    for empty in (dict(n_seqs=0), dict(n_tokens=0)):
        assert append_status(lay, kv=0, q_out=0, pool=0, **empty) == hkv.HKV_OK
        assert prefill_status(lay, x=0, out=0, pool=0, ws=0, ws_bytes=0, **empty) == hkv.HKV_OK


def test_null_handles():
    assert hkv.status_of(hkv.hkv_mla_append, 0, POOL, hkv.hkv_mla_append_args()) == hkv.HKV_E_ARG
    assert hkv.status_of(hkv.hkv_kda_prefill_workspace, 0, hkv.hkv_kda_prefill_args()) == hkv.HKV_E_ARG
    assert hkv.status_of(hkv.hkv_kda_prefill, 0, POOL, hkv.hkv_kda_prefill_args(), WS, 0) == hkv.HKV_E_ARG
    assert hkv.lib.hkv_mla_append(None, None, None, None) == hkv.HKV_E_ARG
    assert hkv.lib.hkv_kda_prefill(None, None, None, None, 0, None) == hkv.HKV_E_ARG
    lay = layout()
    assert hkv.lib.hkv_kda_prefill_workspace(lay.handle, prefill_args(), None) == hkv.HKV_E_ARG


def test_workspaces_follow_the_call():
    lay = layout()
    size = lay.kda_prefill_workspace(prefill_args())
    assert size >= 3 * 4
    assert lay.kda_prefill_workspace(prefill_args(n_seqs=4096, n_tokens=1 << 20, max_seq_tokens=1 << 20)) >= size
    for bad in (dict(n_seqs=-1), dict(n_tokens=-1), dict(max_blocks=0)):
        assert hkv.status_of(lay.kda_prefill_workspace, prefill_args(**bad)) == hkv.HKV_E_ARG


def test_heads_that_no_launch_holds_are_refused():
    heads = 1024
    desc = W._desc([0, 1], heads, 128, 3 * heads * 128, 2, 0, 1 << 40)
    lay = hkv.Layout(desc)
    args = dict(n_tokens=1 << 20, max_seq_tokens=1 << 20, max_blocks=1)
    assert hkv.status_of(lay.kda_prefill_workspace, prefill_args(n_seqs=1, **args)) == hkv.HKV_E_ARG
    assert hkv.status_of(lay.kda_prefill_workspace, prefill_args(n_seqs=4096, n_tokens=9, max_seq_tokens=9)) == hkv.HKV_E_ARG
    assert lay.kda_prefill_workspace(prefill_args(n_seqs=8, n_tokens=5000, max_seq_tokens=900)) > 1 << 33


def test_the_header_declares_them():
    text = open(os.path.join(ROOT, "include", "hkv.h")).read()
    part = text[text.index("New tokens into the pool"):text.index("Object identity")]
    flat = re.sub(r"\s+", " ", re.sub(r"\n \*", " ", part))
    for name in ("hkv_mla_append", "hkv_kda_prefill", "hkv_kda_prefill_workspace"):
        assert re.search(r"hkv_status " + name + r"\(", flat), name
    for status in re.findall(r"HKV_E_\w+", flat):
        assert hasattr(hkv, status), status
