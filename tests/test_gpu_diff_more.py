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
