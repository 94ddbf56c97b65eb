"""Further host-side refusals of the decode-step operators (no GPU needed)."""
import os
import re

import pytest

import retrieve_store_chunk_amd as hkv
from tests.test_ops_host import attend_status, layout, needs_no_gpu

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
