"""Attention of a tree of drafted tokens in plain 64-bit arithmetic, for the
GPU tests, with the bound that its roundings give.

The kernel rounds twice on the way: each weight w of the softmax to the type of
its product with V (bf16 pools: bf16, half a step 2^-8; FP8 pools: f16, 2^-11,
and below f16's normal range, where a weight is at most 2^-14 of 1, half its
smallest step, 2^-25, against a sum of at least 1/2), and the result to bf16
(2^-8).  With A the mean of |V| under the weights, o = sum w v / sum w, whether
the sum takes the rounded weights or not, moves by at most e (A + |o|),
  e = the half step + 2^-12
(2^-12 covers what 32-bit scores, exponentials and sums are off by, for scores
below about 2^5).  A tenth is added for the second order.
"""
from __future__ import annotations

import math
import random

import numpy as np
import torch

from diff_ref import BS, Cache  # noqa: F401  (a pool with known contents)


def parents_of(t, rng, wide=5):
    """A tree of t nodes (parents before children, -1: the context)."""
    return [-1 if i == 0 or rng.random() < 0.1 else max(0, i - rng.randint(1, wide)) for i in range(t)]


def tree_bits(parent):
    bits = []
    for i, p in enumerate(parent):
        bits.append((bits[p] if p >= 0 else 0) | 1 << i)
    return bits


def pack(bits, words):
    """Python integers (a bit per node) as the int64 rows the call takes."""
    rows = []
    for m in bits:
        w = [(m >> (64 * i)) & (2 ** 64 - 1) for i in range(words)]
        rows.append([x - 2 ** 64 if x >= 2 ** 63 else x for x in w])
    return torch.tensor(rows, dtype=torch.int64).reshape(len(bits), words)


def random_masks(nodes, seed=0, wide=5):
    rng = random.Random(seed)
    return [m for t in nodes for m in tree_bits(parents_of(t, rng, wide))]


def plain(cache, q, indptr, bits, lens, scale, skip=(), only=None):
    """(out, bound) [rows, n_q, d]; `bits`: a row's visible nodes as a number; `skip`: (sequence, block index) pairs
    that count as masked; `only`: of these sequences."""
    d, n_kv = cache.d, cache.n_kv
    rows, n_q, _ = q.shape
    G = n_q // n_kv
    half = 2.0 ** -8 if cache.kv == "bf16" else 2.0 ** -11
    e = half + 2.0 ** -12
    out = torch.zeros(rows, n_q, d, dtype=torch.float64)
    bound = torch.zeros_like(out)
    q = q.double().cpu()
    for b, c in enumerate(lens):
        lo, hi = int(indptr[b]), int(indptr[b + 1])
        t = hi - lo
        if t <= 0 or (only is not None and b not in only):
            continue
        ids = cache.tables[b, :(c + BS - 1) // BS].long().clamp(0, cache.blocks - 1)
        k = cache.k64[ids].transpose(0, 1).reshape(n_kv, -1, d)[:, :c]
        v = cache.v64[ids].transpose(0, 1).reshape(n_kv, -1, d)[:, :c]
        see = torch.ones(t, c, dtype=torch.bool)
        see[:, c - t:] = torch.tensor([[(bits[lo + i] >> j) & 1 for j in range(t)] for i in range(t)], dtype=torch.bool)
        for sb, sj in skip:
            if sb == b:
                see[:, sj * BS:(sj + 1) * BS] = False
        v = torch.where(see.any(0)[None, :, None], v, torch.zeros_like(v))
        for h in range(n_q):
            vv = v[h // G]
            s = (q[lo:hi, h] @ k[h // G].t()) * float(np.float32(scale))
            s = s.masked_fill(~see, -math.inf)
            w = (s - s.amax(-1, keepdim=True).clamp(min=-1e300)).exp()
            total = w.sum(-1, keepdim=True)
            p = torch.where(total > 0, w / total, torch.zeros_like(w))
            o, size = p @ vv, p @ vv.abs()
            if cache.kv != "bf16":
                size = size + 2 * 2.0 ** -25 / e * see.sum(-1, keepdim=True) * vv.abs().amax()
            out[lo:hi, h] = o
            bound[lo:hi, h] = 1.1 * e * (size + o.abs())
    return out, bound + 2.0 ** -8 * out.abs() + 1e-30


def check(got, ref, bound):
    got = got.double().cpu()
    assert torch.isfinite(got).all()
    err = (got - ref).abs()
    assert (err <= bound).all(), f"worst: {float((err / bound).max()):.3g} of the bound"
