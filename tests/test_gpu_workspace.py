"""How a pool's workspace grows: what it takes of the GPU's memory, and what a captured graph keeps."""
import pytest
import torch

import gqa_decode_attention_paged_gb300 as pkv
from diff_ref import BS, weights

MIB = 1 << 20
N_KV, G, D = 8, 8, 128


def pool_with(tokens=BS):
    pool = pkv.kv_pool_create(4, BS, N_KV, D, pkv.BF16)
    pool.set_partition_tokens(tokens)  # short slices: the workspace grows with the tables' width
    pool.k_view().zero_()
    pool.v_view().zero_()
    return pool


def used():
    torch.cuda.synchronize()
    free, total = torch.cuda.mem_get_info()
    return total - free


def reserve(pool, kind, W):
    (pool.reserve_workspace if kind == "decode" else pool.reserve_diff_workspace)(8, N_KV * G, W)
    return pool.timing_read()["workspace_bytes"]


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["decode", "diff"])
def test_a_workspace_that_no_graph_uses_is_freed_when_it_grows(kind):
    with pool_with() as pool:
        reserve(pool, kind, 256)
        base = used() - pool.timing_read()["workspace_bytes"]
        for W in (512, 600, 1024, 1100, 1300):  # steps smaller than a doubling, and one larger
            now = reserve(pool, kind, W)
            assert abs(used() - base - now) <= 4 * MIB  # nothing but the newest (in pages of 2 MiB)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["decode", "diff"])
@pytest.mark.parametrize("captured", [False, True])
def test_a_workspace_grows_where_its_headroom_does_not_fit(kind, captured):
    """With too little free memory for a quarter (or, beside one that a graph uses, the double) on top, the
    bytes that are needed are asked for."""
    with pool_with() as pool:
        first = reserve(pool, kind, 1024)
        with pool_with() as other:
            more = reserve(other, kind, 1600)  # 1.25 times what 1600 needs
        need = more * 4 // 5
        assert first < need and 2 * first > need + 24 * MIB and need // 4 > 24 * MIB
        if captured:
            q = torch.zeros(1, N_KV * G, D, dtype=torch.bfloat16, device="cuda")
            tables, lens = torch.zeros(1, 1024, dtype=torch.int32, device="cuda"), torch.ones(1, dtype=torch.int32, device="cuda")
            params = weights(D)
            g = torch.cuda.CUDAGraph()
            torch.cuda.synchronize()
            with torch.cuda.graph(g):
                if kind == "decode":
                    pkv.paged_decode_attention(pool, q, tables, lens, 1.0)
                else:
                    pkv.paged_diff_decode_attention(pool, q, tables, lens, 1.0, params)
        torch.cuda.synchronize()
        torch.cuda.empty_cache()
        free = torch.cuda.mem_get_info()[0]
        room = need + 12 * MIB if captured else need + 12 * MIB - first  # (the old one's place is free then, too)
        hog = torch.empty(free - room, dtype=torch.uint8, device="cuda")
        try:
            got = reserve(pool, kind, 1600)
        finally:
            del hog
            torch.cuda.empty_cache()
        # more is 5/4 of the bytes, rounded up to a MiB: the bytes are at most need and above need - 4/5 MiB, rounded up
        assert need - MIB < got <= need + MIB
        if captured:
            g.replay()
            torch.cuda.synchronize()
            assert pool.get_error() == 0


@pytest.mark.gpu
def test_a_captured_plain_decode_keeps_its_workspace():
    with pool_with(0) as pool:
        pool.k_view().copy_(torch.randn(4, N_KV, BS, D).to(torch.bfloat16).view(torch.uint8).cuda())
        pool.v_view().copy_(torch.randn(4, N_KV, BS, D).to(torch.bfloat16).view(torch.uint8).cuda())
        q = torch.randn(2, N_KV * G, D, device="cuda").to(torch.bfloat16)
        tables = torch.tensor([[0, 1, 2, 3] * 64, [3, 2, 1, 0] * 64], dtype=torch.int32, device="cuda")
        lens = torch.tensor([4000, 777], dtype=torch.int32, device="cuda")
        want = pkv.paged_decode_attention(pool, q, tables, lens, 0.1)
        g = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(g):
            out = pkv.paged_decode_attention(pool, q, tables, lens, 0.1)
        before = pool.timing_read()["workspace_bytes"]
        pool.set_partition_tokens(BS)
        assert reserve(pool, "decode", 4096) > before
        for _ in range(2):
            out.zero_()
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, want)
