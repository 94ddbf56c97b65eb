"""Host-side checks of the decode-step operators (no GPU needed): argument
validation rejects bad calls before any HIP call, workspace sizes, and what the
header says.  Fake device addresses are used, so these run only where no GPU is
visible."""
import ctypes
import os
import re

import pytest
import torch

import retrieve_store_chunk_amd as hkv
import workloads as W

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

needs_no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="uses fake device addresses")

POOL = 1 << 40


def layout(**kw):
    desc = W._desc([0, 0, 1, 0, 1], kw.pop("heads", 2), kw.pop("head_dim", 16), kw.pop("conv_dim", 96),
                   kw.pop("mla_bytes", 2), kw.pop("path", 0), 1 << 22, **kw)
    return hkv.Layout(desc)


def attend_args(lay, **kw):
    a = dict(layer=2, n_seqs=3, n_heads=8, value_width=512, dtype=hkv.HKV_BF16,
             cache_dtype=hkv.HKV_BF16, max_blocks=4, scale=0.1, cache_scale=1.0, q=0x1000000,
             q_seq_stride=8 * 576, q_head_stride=576, block_table=0x2000000, table_stride=4,
             seq_lens=0x3000000, out=0x4000000, out_seq_stride=8 * 512, out_head_stride=512,
             lse=0x5000000, weights=0x6000000, weights_stride=4 * lay.info["block_size"])
    a.update(kw)
    return hkv.hkv_mla_attend_args(**a)


def evict_args(lay, layers=(2, 4), **kw):
    slots = 4 * lay.info["block_size"]
    a = dict(n_seqs=3, max_blocks=4, budget=20, sinks=2, recent=8, block_table=0x2000000,
             table_stride=4, seq_lens=0x3000000, next_positions=0x3800000, weights=0x4000000,
             positions=0x5000000, weights_out=0x6000000, positions_out=0x7000000,
             layer_stride=3 * slots, seq_stride=slots, new_lens=0x8000000)
    a.update(kw)
    args = hkv.hkv_mla_evict_args(**a)
    args.set_layers(list(layers))
    return args


def kda_args(lay, **kw):
    a = dict(layer=0, n_seqs=3, dtype=hkv.HKV_BF16, scale=0.25, eps=1e-6, x=0x1000000, x_stride=96,
             conv_weight=0x2000000, log_decay=0x3000000, decay_stride=32, beta=0x4000000,
             beta_stride=2, src_blocks=0x5000000, dst_blocks=0x6000000, out=0x7000000, out_stride=32)
    a.update(kw)
    return hkv.hkv_kda_step_args(**a)


WS = 0x7F0000000000


def attend_status(lay, ws=WS, ws_bytes=1 << 32, pool=POOL, **kw):
    return hkv.status_of(lay.mla_attend, pool, attend_args(lay, **kw), ws, ws_bytes, 0)


def evict_status(lay, ws=WS, ws_bytes=1 << 32, pool=POOL, layers=(2, 4), **kw):
    return hkv.status_of(lay.mla_evict, pool, evict_args(lay, layers, **kw), ws, ws_bytes, 0)


def kda_status(lay, pool=POOL, **kw):
    return hkv.status_of(lay.kda_step, pool, kda_args(lay, **kw), 0)


@needs_no_gpu
@pytest.mark.parametrize("bad,status", [
    (dict(layer=0), "ARG"), (dict(layer=-1), "ARG"), (dict(layer=5), "ARG"),
    (dict(n_seqs=-1), "ARG"), (dict(n_seqs=65536), "ARG"),
    (dict(n_heads=0), "ARG"), (dict(n_heads=129), "ARG"),
    (dict(value_width=0), "ARG"), (dict(value_width=24), "ARG"), (dict(value_width=528), "ARG"),
    (dict(dtype=hkv.HKV_FP32), "ARG"), (dict(cache_dtype=hkv.HKV_FP16), "ARG"),
    (dict(cache_dtype=hkv.HKV_E4M3), "ARG"), (dict(max_blocks=0), "ARG"),
    (dict(max_blocks=2**31 - 1), "ARG"), (dict(table_stride=-1), "ARG"),
    (dict(scale=float("nan")), "ARG"), (dict(cache_scale=float("inf")), "ARG"),
    (dict(q=0), "ARG"), (dict(block_table=0), "ARG"), (dict(seq_lens=0), "ARG"), (dict(out=0), "ARG"),
    (dict(q_seq_stride=-8), "ARG"), (dict(out_head_stride=-8), "ARG"),
    (dict(q_seq_stride=2**60), "ARG"), (dict(weights_stride=4), "ARG"),
    (dict(q=0x1000008), "ALIGN"), (dict(out=0x4000002), "ALIGN"), (dict(q_head_stride=580), "ALIGN"),
    (dict(out_seq_stride=8 * 512 + 4), "ALIGN"), (dict(lse=0x5000002), "ALIGN"),
    (dict(block_table=0x2000001), "ALIGN"), (dict(seq_lens=0x3000002), "ALIGN"),
    (dict(weights=0x6000001), "ALIGN"),
    (dict(out_head_stride=504), "ALIAS"), (dict(out_seq_stride=0), "ALIAS"),
    (dict(out_seq_stride=8), "ALIAS"), (dict(out=0x1000000), "ALIAS"), (dict(lse=0x4000000), "ALIAS"),
    (dict(weights=0x5000000), "ALIAS"), (dict(weights=POOL + 4096), "ALIAS"), (dict(lse=WS + 64), "ALIAS"),
    (dict(pool=POOL + 8), "ALIGN"), (dict(pool=0), "ARG"), (dict(ws=0), "WORKSPACE"),
    (dict(ws_bytes=1000), "WORKSPACE"), (dict(ws=WS + 8), "ALIGN"), (dict(ws=POOL), "ALIAS"),
])
def test_attend_refusals(bad, status):
    lay = layout()
    assert attend_status(lay, **bad) == getattr(hkv, "HKV_E_" + status), hkv.hkv_last_error()
    assert hkv.hkv_last_error()


@needs_no_gpu
def test_attend_layout_refusals():
    assert attend_status(layout(mla_width=9)) == hkv.HKV_E_ARG
    assert attend_status(layout(mla_width=48), value_width=32) == hkv.HKV_E_ARG
    assert attend_status(layout(mla_width=608), value_width=512) == hkv.HKV_E_ARG
    assert attend_status(layout(mla_width=64), value_width=80) == hkv.HKV_E_ARG
    assert attend_status(layout(mla_bytes=4)) == hkv.HKV_E_ARG
    fp8 = layout(mla_bytes=1)
    assert attend_status(fp8) == hkv.HKV_E_ARG  # cache_dtype is bf16
    assert attend_status(fp8, cache_dtype=hkv.HKV_FP16) == hkv.HKV_E_ARG
    # a group that mixes pages whose size is no 16-byte multiple (packed)
    odd = layout(path=1, conv_dim=5, kv_group_of_layer=[0, 0, 0, 0, 0])
    assert odd.layers[2]["pool_offset"] % 16
    assert attend_status(odd) == hkv.HKV_E_ALIGN


@needs_no_gpu
@pytest.mark.parametrize("bad,status", [
    (dict(layers=()), "ARG"), (dict(layers=(2,) * 65), "ARG"), (dict(layers=(0,)), "ARG"),
    (dict(layers=(2, 7)), "ARG"), (dict(layers=(2, 2)), "ALIAS"), (dict(n_seqs=-1), "ARG"),
    (dict(n_seqs=40000), "ARG"), (dict(max_blocks=0), "ARG"), (dict(max_blocks=1 << 25), "ARG"),
    (dict(budget=0), "ARG"), (dict(sinks=-1), "ARG"), (dict(recent=-1), "ARG"),
    (dict(sinks=13), "ARG"), (dict(table_stride=-4), "ARG"), (dict(layer_stride=-1), "ARG"),
    (dict(seq_stride=2**60), "ARG"), (dict(block_table=0), "ARG"), (dict(seq_lens=0), "ARG"),
    (dict(next_positions=0), "ARG"), (dict(weights=0), "ARG"), (dict(positions=0), "ARG"),
    (dict(weights_out=0), "ARG"), (dict(positions_out=0), "ARG"),
    (dict(seq_stride=8), "ALIAS"), (dict(layer_stride=8), "ALIAS"),
    (dict(weights_out=0x4000010), "ALIAS"), (dict(positions_out=0x5000010), "ALIAS"),
    (dict(new_lens=0x3000000), "ALIAS"), (dict(new_lens=0x2000000), "ALIAS"),
    (dict(weights_out=0x5000000), "ALIAS"), (dict(weights=POOL), "ALIAS"),
    (dict(weights=0x4000002), "ALIGN"), (dict(new_lens=0x8000001), "ALIGN"),
    (dict(pool=0), "ARG"), (dict(pool=POOL + 4), "ALIGN"), (dict(ws=0), "WORKSPACE"),
    (dict(ws_bytes=16), "WORKSPACE"), (dict(ws=WS + 4), "ALIGN"),
])
def test_evict_refusals(bad, status):
    lay = layout()
    assert evict_status(lay, **bad) == getattr(hkv, "HKV_E_" + status), hkv.hkv_last_error()


@needs_no_gpu
def test_evict_wants_one_kv_group():
    lay = layout(kv_group_of_layer=[0, 0, 1, 0, 2])
    assert evict_status(lay) == hkv.HKV_E_ARG
    args = evict_args(lay)
    args.layers = ctypes.POINTER(ctypes.c_int32)()
    assert hkv.status_of(lay.mla_evict, POOL, args, WS, 1 << 32, 0) == hkv.HKV_E_ARG


@needs_no_gpu
@pytest.mark.parametrize("bad,status", [
    (dict(layer=2), "ARG"), (dict(layer=9), "ARG"), (dict(n_seqs=-1), "ARG"), (dict(n_seqs=4097), "ARG"),
    (dict(dtype=hkv.HKV_FP32), "ARG"), (dict(dtype=hkv.HKV_E4M3), "ARG"), (dict(dtype=17), "ARG"),
    (dict(scale=float("inf")), "ARG"), (dict(eps=-1e-6), "ARG"), (dict(x=0), "ARG"),
    (dict(conv_weight=0), "ARG"), (dict(log_decay=0), "ARG"), (dict(beta=0), "ARG"),
    (dict(src_blocks=0), "ARG"), (dict(dst_blocks=0), "ARG"), (dict(out=0), "ARG"), (dict(pool=0), "ARG"),
    (dict(x_stride=-1), "ARG"), (dict(decay_stride=2**60), "ARG"), (dict(out_stride=28), "ALIAS"),
    (dict(out_stride=-32), "ALIAS"), (dict(out_stride=34), "ALIGN"), (dict(out=0x7000008), "ALIGN"),
    (dict(x=0x1000001), "ALIGN"), (dict(beta=0x4000002), "ALIGN"), (dict(pool=POOL + 8), "ALIGN"),
    (dict(out=0x1000000), "ALIAS"), (dict(out=0x5000000), "ALIAS"), (dict(x=POOL + 64), "ALIAS"),
])
def test_kda_refusals(bad, status):
    lay = layout()
    assert kda_status(lay, **bad) == getattr(hkv, "HKV_E_" + status), hkv.hkv_last_error()


@needs_no_gpu
def test_kda_layout_refusals():
    assert kda_status(layout(head_dim=40, conv_dim=240)) == hkv.HKV_E_ARG
    assert kda_status(layout(conv_dim=95)) == hkv.HKV_E_ARG
    assert kda_status(layout(conv_kernel=9)) == hkv.HKV_E_ARG
    assert kda_status(layout(state_bytes=2)) == hkv.HKV_E_ARG
    assert kda_status(layout(conv_bytes=4)) == hkv.HKV_E_ARG  # wants fp32
    assert kda_status(layout(conv_bytes=1)) == hkv.HKV_E_ARG


@needs_no_gpu
def test_empty_calls_do_nothing():
    lay = layout()
    assert attend_status(lay, n_seqs=0, q=0, out=0, ws=0, ws_bytes=0) == hkv.HKV_OK
    assert evict_status(lay, n_seqs=0, weights=0, ws=0, ws_bytes=0) == hkv.HKV_OK
    assert kda_status(lay, n_seqs=0, x=0) == hkv.HKV_OK


def test_null_handles():
    assert hkv.status_of(hkv.hkv_mla_attend_workspace, 0, hkv.hkv_mla_attend_args()) == hkv.HKV_E_ARG
    assert hkv.status_of(hkv.hkv_mla_attend, 0, POOL, hkv.hkv_mla_attend_args(), WS, 0) == hkv.HKV_E_ARG
    assert hkv.status_of(hkv.hkv_mla_evict_workspace, 0, hkv.hkv_mla_evict_args()) == hkv.HKV_E_ARG
    assert hkv.status_of(hkv.hkv_mla_evict, 0, POOL, hkv.hkv_mla_evict_args(), WS, 0) == hkv.HKV_E_ARG
    assert hkv.status_of(hkv.hkv_kda_step, 0, POOL, hkv.hkv_kda_step_args()) == hkv.HKV_E_ARG
    assert hkv.lib.hkv_kda_step(None, None, None, None) == hkv.HKV_E_ARG
    assert hkv.lib.hkv_mla_attend(None, None, None, None, 0, None) == hkv.HKV_E_ARG
    assert hkv.lib.hkv_mla_evict(None, None, None, None, 0, None) == hkv.HKV_E_ARG


def test_workspaces_grow_with_the_call():
    lay = layout()
    size = lay.mla_attend_workspace(attend_args(lay, weights=0))
    more = lay.mla_attend_workspace(attend_args(lay))
    assert more - size >= 3 * 4 * lay.info["block_size"] * 8 * 4  # one fp32 a head and token
    assert lay.mla_attend_workspace(attend_args(lay, n_seqs=500, max_blocks=500, weights=0)) > size
    assert lay.mla_evict_workspace(evict_args(lay)) < lay.mla_evict_workspace(evict_args(lay, max_blocks=4000))
    # at most 256 workgroups x 2 partial results x heads x values x 4 bytes, and little else
    big = lay.mla_attend_workspace(attend_args(lay, n_seqs=64, n_heads=128, max_blocks=100000, weights=0))
    assert 256 * 2 * 64 * 512 * 4 <= big < 256 * 2 * 64 * 520 * 4 + (1 << 20)


PAGES = ("vLLM hybrid KV-cache blog",)


def test_the_header_says_where_the_operators_layouts_come_from():
    text = open(os.path.join(ROOT, "include", "hkv.h")).read()
    part = text[text.index("The decode step over the pool"):text.index("Object identity")]
    flat = re.sub(r"\s+", " ", re.sub(r"\n \*", " ", part))
    for name in ("hkv_mla_attend", "hkv_mla_evict", "hkv_kda_step"):
        assert re.search(r"hkv_status " + name + r"\(", flat), name
    assert all(p in flat for p in PAGES)
    for status in re.findall(r"HKV_E_\w+", flat):
        assert hasattr(hkv, status), status
