"""Further host-side refusals of the decode-step operators (no GPU needed)."""
import pytest

import retrieve_store_chunk_amd as hkv
from tests.test_ops_host import attend_status, layout, needs_no_gpu


@needs_no_gpu
@pytest.mark.parametrize("scale,cache_scale", [(1e30, 1e10), (-1e30, 1e10), (3e38, 1.5)])
def test_attend_scales_whose_product_overflows(scale, cache_scale):
    """Each is finite, but the logits' factor is not an fp32 number."""
    assert attend_status(layout(), scale=scale, cache_scale=cache_scale) == hkv.HKV_E_ARG
    assert "scale" in hkv.hkv_last_error()
