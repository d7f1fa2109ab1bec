"""Calls that are given a stream: their outputs are that stream's memory."""
import pytest
import torch

import gqa_decode_attention_paged_gb300 as pkv
from diff_ref import BS, weights

N_KV, D, B = 2, 64, 3


def owner(t):
    """Handle of the stream whose memory t is."""
    for seg in torch.cuda.memory_snapshot():
        if seg["address"] <= t.data_ptr() < seg["address"] + seg["total_size"]:
            return seg["stream"]
    raise AssertionError("not memory of the caching allocator")


def calls(pool):
    """Every call that allocates its outputs, as f(**kw) -> outputs."""
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    q, kv = (torch.randn(B, h, D, device="cuda").to(torch.bfloat16) for h in (4, N_KV))
    tables, lens, indptr = i32([[0], [1], [2]]), i32([5, 16, 9]), i32([0, 1, 2, 3])
    positions, slots, prefix = i32([[4, 15, 8]]), torch.tensor([4, 31, 40], device="cuda"), i32([3])
    rope, params = pkv.Rope([1.0] * 16), weights(D)
    two = torch.cat((prefix.repeat(B, 1), tables), 1)
    return {
        "decode": lambda **k: pkv.paged_decode_attention(pool, q, tables, lens, 0.1, **k),
        "noalloc": lambda **k: pkv.paged_decode_attention_noalloc(pool, q, tables, lens, 0.1, **k),
        "csr": lambda **k: pkv.paged_decode_attention_csr(pool, q, indptr, tables.view(-1), lens, 0.1, **k),
        "prefill": lambda **k: pkv.paged_prefill_attention(pool, q, indptr, tables, lens, 0.1, **k),
        "prefix": lambda **k: pkv.paged_decode_attention_prefix(pool, q, prefix, two, lens + 16, 0.1, **k),
        "step": lambda **k: pkv.paged_decode_step(pool, q, kv, kv, tables, lens, 0.1, **k),
        "rope": lambda **k: pkv.paged_rope_append(pool, rope, q, kv, kv, positions, slots, **k),
        "gather": lambda **k: pkv.paged_kv_gather(pool, indptr, tables, n_rows=B, **k),
        "diff decode": lambda **k: pkv.paged_diff_decode_attention(pool, q, tables, lens, 0.1, params, **k),
        "diff prefill": lambda **k: pkv.paged_diff_prefill_attention(pool, q, indptr, tables, lens, 0.1, params, **k),
    }


@pytest.mark.gpu
@pytest.mark.parametrize("handle", [False, True], ids=["stream", "handle"])
def test_outputs_are_memory_of_the_given_stream(handle):
    """Memory of the current stream may be in use by kernels queued there, which the other stream does not wait for."""
    with pkv.kv_pool_create(8, BS, N_KV, D, pkv.BF16) as pool:
        pool.k_view().copy_(torch.randn(8, N_KV, BS, D).to(torch.bfloat16).view(torch.uint8).cuda())
        pool.v_view().copy_(torch.randn(8, N_KV, BS, D).to(torch.bfloat16).view(torch.uint8).cuda())
        todo = calls(pool)
        side = torch.cuda.Stream()
        torch.cuda.synchronize()
        for name, call in todo.items():
            outs = lambda x: x if isinstance(x, tuple) else (x,)  # noqa: E731
            want = outs(call())
            torch.cuda.synchronize()
            got = outs(call(stream=side.cuda_stream if handle else side))
            side.synchronize()
            for x, y in zip(want, got):
                assert torch.equal(x, y), name
                assert owner(x) == torch.cuda.current_stream().cuda_stream, name
                assert owner(y) == side.cuda_stream, name
            with torch.cuda.stream(side):  # the same stream by another name
                assert all(owner(y) == side.cuda_stream for y in outs(call(stream=side.cuda_stream)))
                here = torch.cuda.default_stream()
                got = outs(call(stream=here.cuda_stream if handle else here))  # back on the default stream
                assert all(owner(y) == here.cuda_stream for y in got)
            torch.cuda.synchronize()
            for x, y in zip(want, got):
                assert torch.equal(x, y), name
        assert pool.get_error() == 0
