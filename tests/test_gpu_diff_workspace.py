"""The workspace of the differential decode: what a reservation covers."""
import pytest
import torch

import gqa_decode_attention_paged_gb300 as pkv
from diff_ref import BS, weights


def inputs(batch, n_q, d, W):
    q = torch.zeros(batch, n_q, d, dtype=torch.bfloat16, device="cuda")
    return q, torch.zeros(batch, W, dtype=torch.int32, device="cuda"), torch.full((batch,), BS, dtype=torch.int32, device="cuda")


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [pkv.BF16, pkv.FP8_E4M3])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("reserved,G,calls", [
    (2000, 8, [(2000, 8), (1025, 8), (1024, 8), (1000, 8), (1, 8), (1000, 1)]),
    (8192, 2, [(8192, 2), (4097, 2), (1000, 2), (300, 1)]),
])
def test_a_reservation_covers_every_smaller_call(dtype, d, reserved, G, calls):
    """More sequences leave fewer CTAs an SM (their lists share its memory), so a smaller call may need more."""
    n_kv, W = 2, 16
    with pkv.kv_pool_create(W, BS, n_kv, d, dtype) as pool:
        if dtype == pkv.FP8_E4M3:
            pool.set_fp8_scales([1.0] * n_kv, [1.0] * n_kv)
        pool.k_view().zero_()
        pool.v_view().zero_()
        params = weights(d)
        pool.reserve_diff_workspace(reserved, n_kv * G, W)
        before = pool.timing_read()["workspace_bytes"]
        for batch, g in calls:
            q, tables, lens = inputs(batch, n_kv * g, d, W)
            graph = torch.cuda.CUDAGraph()
            torch.cuda.synchronize()
            with torch.cuda.graph(graph):
                out = pkv.paged_diff_decode_attention(pool, q, tables, lens, 1.0, params)
            graph.replay()
            torch.cuda.synchronize()
            assert (out == 0).all()
        assert pool.timing_read()["workspace_bytes"] == before and pool.get_error() == 0
