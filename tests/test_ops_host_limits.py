"""Further host-side refusals of the decode-step operators (no GPU needed)."""
import os
import re

import pytest

import retrieve_store_chunk_amd as hkv
from tests.test_ops_host import attend_args, attend_status, evict_args, layout, needs_no_gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def header_comment(before):
    """The comment of include/hkv.h that ends right before `before`, on one line."""
    text = open(os.path.join(ROOT, "include", "hkv.h")).read()
    text = text[:text.index(before)]
    return re.sub(r"\s+", " ", re.sub(r"\n \*", " ", text[text.rindex("/*"):]))


@needs_no_gpu
@pytest.mark.parametrize("scale,cache_scale", [(1e30, 1e10), (-1e30, 1e10), (3e38, 1.5)])
def test_attend_scales_whose_product_overflows(scale, cache_scale):
    """Each is finite, but the logits' factor is not an fp32 number."""
    assert attend_status(layout(), scale=scale, cache_scale=cache_scale) == hkv.HKV_E_ARG
    assert "scale" in hkv.hkv_last_error()


def test_the_header_says_that_evicted_blocks_are_no_longer_the_prefixs():
    text = header_comment("typedef struct hkv_mla_evict_args")
    assert "hkv_chunk_keys" in text and "prefix" in text


def size_status(fn, args):
    return hkv.status_of(fn, args)


def test_the_largest_tables():
    """The limits that the header states, on both sides."""
    lay = layout()
    n = lay.info["block_size"]
    assert n == 16 and (1 << 28) % n == 0
    attend, evict = lay.mla_attend_workspace, lay.mla_evict_workspace
    most = (2**31 - 1) // n
    assert size_status(attend, attend_args(lay, n_seqs=1, max_blocks=most)) == hkv.HKV_OK
    assert size_status(attend, attend_args(lay, n_seqs=1, max_blocks=most + 1)) == hkv.HKV_E_ARG
    # 2^36 - 32 tokens in all
    assert size_status(attend, attend_args(lay, n_seqs=31, max_blocks=most)) == hkv.HKV_OK
    assert size_status(attend, attend_args(lay, n_seqs=32, max_blocks=most)) == hkv.HKV_E_ARG
    assert size_status(evict, evict_args(lay, n_seqs=1, max_blocks=(1 << 28) // n)) == hkv.HKV_OK
    assert size_status(evict, evict_args(lay, n_seqs=1, max_blocks=(1 << 28) // n + 1)) == hkv.HKV_E_ARG
    assert size_status(evict, evict_args(lay, (2,), n_seqs=65535)) == hkv.HKV_OK
    assert size_status(evict, evict_args(lay, (2, 4), n_seqs=32767)) == hkv.HKV_OK
    assert size_status(evict, evict_args(lay, (2, 4), n_seqs=32768)) == hkv.HKV_E_ARG


def test_the_header_states_the_limits():
    text = header_comment("#define HKV_BF16")
    assert "2^31 - 1 tokens" in text and "2^28 for an eviction" in text and "16-byte boundaries" in text
    header = open(os.path.join(ROOT, "include", "hkv.h")).read()
    assert "2^36 - 32 tokens" in header and "n_layers x n_seqs too" in header
