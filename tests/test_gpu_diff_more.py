"""Differential attention where values are not finite, where its two maps nearly cancel, and captured."""
import math

import numpy as np
import pytest
import torch

import gqa_decode_attention_paged_gb300 as pkv
from diff_ref import BS, Cache, check, plain, weights
from test_gpu_diff_prefill import PAD, i32, prefill, ptr, queries


def decode(c, q, params, **kw):
    return pkv.paged_diff_decode_attention(c.pool, q, c.tables.cuda(), i32(c.lens), 1 / np.sqrt(c.d), params, **kw)


def at(c, b, pos):
    """(block, offset) of a position of sequence b."""
    return int(c.tables[b, pos // BS]), pos % BS


@pytest.mark.gpu
@pytest.mark.parametrize("part", [0, 16])
@pytest.mark.parametrize("G", [1, 8])
def test_visible_keys_with_scores_of_minus_infinity_weigh_nothing(part, G):
    """Keys of one channel at -infinity, among them the sequence's first 16 (a whole block) and all of one sequence."""
    d, lens, chunks = 64, [300, 40, 16, 5, 700], [33, 20, 16, 5, 120]
    low = [list(range(16)) + [100, 299], list(range(16)) + [20], range(16), [0, 4], list(range(64)) + list(range(500, 600))]
    with Cache("bf16", 2, d, lens, seed=21) as c:
        for b, keys in enumerate(low):
            for pos in keys:
                blk, off = at(c, b, pos)
                c.k[blk, :, off, 0] = -math.inf
        c.k64 = c.k.double()
        c.upload()
        c.pool.set_partition_tokens(part)
        params = weights(d)
        q = queries(len(lens), 2 * G, d)
        q[..., 0] = 1
        got = decode(c, q, params)
        torch.cuda.synchronize()
        check(got, *plain(c, q, np.arange(len(lens) + 1), lens, 1 / np.sqrt(d), params))
        q = queries(sum(chunks), 2 * G, d)
        q[..., 0] = 1
        for pad in (0, PAD):
            got = prefill(c, q, chunks, params, pad=pad)
            torch.cuda.synchronize()
            check(got, *plain(c, q, ptr(chunks), lens, 1 / np.sqrt(d), params))
        assert c.pool.get_error() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("which", ["key", "value"])
def test_a_nan_reaches_the_rows_that_see_it_and_no_other_heads_or_sequences(kv, which):
    """A NaN key reaches the rows from its position on.  A NaN value at position 0 is seen by every row."""
    d, lens, chunks = 64, [70, 300], [70, 130]
    pos = 41 if which == "key" else 0
    with Cache(kv, 4, d, lens, seed=22) as c:
        q, params = queries(sum(chunks), 8, d), weights(d)
        qd = queries(2, 8, d, 1)
        want = [prefill(c, q, chunks, params), prefill(c, q, chunks, params, pad=PAD), decode(c, qd, params)]
        blk, off = at(c, 0, pos)
        x = c.k if which == "key" else c.v
        x.view(torch.uint8)[blk, 1, off] = torch.full((d,), math.nan).to(x.dtype).view(torch.uint8)  # the first pair's second head
        c.upload()
        got = [prefill(c, q, chunks, params), prefill(c, q, chunks, params, pad=PAD), decode(c, qd, params)]
        torch.cuda.synchronize()
        for i, (x, y) in enumerate(zip(want, got)):
            nan = torch.zeros_like(x, dtype=torch.bool)
            nan[(pos if i < 2 else 0):(70 if i < 2 else 1), :2] = True  # the pair's two heads
            assert torch.equal(torch.isnan(y), nan)
            assert torch.equal(torch.where(nan, 0, y.float()), torch.where(nan, 0, x.float()))


@pytest.mark.gpu
@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("d", [64, 128])
def test_maps_that_nearly_cancel_keep_their_difference(kv, d):
    """Both maps on the same keys, the second's queries an eighth longer, lambda 1: what is left is about an eighth of
    either map.  With V and the scores as they are, roundings of each map's weights to one bf16 would move the result
    by 1.4e-2 in the 2-norm (a 64-bit simulation of each rounding), as decode's two bf16 or f16 they do by at most
    2.4e-3 with the result's own (1.7e-3), and one rounding of the difference, as chunks take it, by 2.2e-3: 2^-8."""
    lens, chunks = [700, 90], [64, 30]
    with Cache(kv, 2, d, lens, seed=23) as c:
        if kv == "fp8":
            c.pool.set_fp8_scales(*[np.full(2, 5 / 448, np.float32)] * 2)
        c.k[:, 1] = c.k[:, 0]
        f = 1.0 if kv == "bf16" else float(np.float32(5 / 448))
        c.k64, c.v64 = c.k.double() * f, c.v.double() * f
        c.upload()
        a = torch.zeros(4, d, device="cuda")
        a[0, 0], a[1, 0] = 1.0, math.log(1.5)
        params = pkv.DiffParams(a, 0.5)  # 1.5 - 1 + 0.5

        def pairs(rows, seed):
            q = queries(rows, 8, d, seed)
            q[:, 1::2] = (q[:, 0::2].float() * 1.125).to(torch.bfloat16)
            return q

        q = pairs(2, 0)
        outs = [(decode(c, q, params), plain(c, q, np.arange(3), lens, 1 / np.sqrt(d), params)[0])]
        q = pairs(sum(chunks), 1)
        ref = plain(c, q, ptr(chunks), lens, 1 / np.sqrt(d), params)[0]
        outs += [(prefill(c, q, chunks, params, pad=pad), ref) for pad in (0, PAD)]
        for got, ref in outs:
            rel = float((got.double().cpu() - ref).norm() / ref.norm())
            assert rel <= 2.0 ** -8, f"{rel:.2e}"


@pytest.mark.gpu
@pytest.mark.parametrize("lens,chunks", [([500, 40], [13, 4]), ([300] * 200, [2] * 200), ([900, 30], [800, 30])])
def test_captured_chunks_are_the_bits_of_eager_ones_and_take_no_workspace(lens, chunks):
    with Cache("bf16", 4, 128, lens, seed=24) as c:
        q, params = queries(sum(chunks), 8, 128), weights(128)
        args = (i32(ptr(chunks)), c.tables.cuda(), i32(lens), 1 / np.sqrt(128), params)
        want = pkv.paged_diff_prefill_attention(c.pool, q, *args)
        static = torch.zeros_like(q)
        g = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(g):
            out = pkv.paged_diff_prefill_attention(c.pool, static, *args)
        for _ in range(2):
            static.copy_(q)
            out.zero_()
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, want)
        assert c.pool.timing_read()["workspace_bytes"] == 0
