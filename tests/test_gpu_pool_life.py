"""When a pool's memory goes."""
import gc
import weakref

import pytest

import gqa_decode_attention_paged_gb300 as pkv


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [pkv.BF16, pkv.FP8_E4M3, pkv.INT4])
def test_a_pool_goes_with_its_last_view_and_without_the_cycle_collector(dtype):
    """Nothing that a view leaves behind is a reference cycle: full GPU memory does not start the collector."""
    gc.collect()
    gc.disable()
    try:
        pool = pkv.kv_pool_create(3, 16, 2, 64, dtype)
        alive = weakref.ref(pool)
        views = [pool.k_view(), pool.v_view()[1:]] + ([pool.v_params_view()] if dtype == pkv.INT4 else [])
        del pool
        while views:
            assert alive() is not None
            views.pop()
        assert alive() is None
    finally:
        gc.enable()
