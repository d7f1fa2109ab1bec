"""Differential attention in plain 64-bit arithmetic, for the GPU tests, with
the bound that its roundings give.

The kernels round twice on the way: the weights of a map to the type of its
product with V (bf16 pools: bf16, half a step 2^-8; FP8 pools: f16, 2^-11, and
below f16's normal range, where a weight is at most 2^-14 of the largest, half
its smallest step, 2^-25), and the result to bf16 (2^-8).  With A_m the mean
of |V| under map m, the weights' rounding moves o by at most
  d = e (A_1 + |lambda| A_2),   e = the half step + 2^-12
(2^-12 covers what 32-bit scores, exponentials, sums and lambda are off by, for
scores below about 2^5).  Through the norm, with r = 1 / sqrt(mean(o^2) + eps):
  |d out| <= |w| (1 - lambda_init) r (d + |o| r rms(d))
to first order; a tenth of it is added for the rest.  That is the worst case
element by element.  For independent roundings of inputs with mean zero the
two together stay below 2^-8 sqrt(2 / 3) of the result in the 2-norm (each
rounding is uniform within its half step: 2^-8 / sqrt(3)), so 2^-8 is asked.
"""
from __future__ import annotations

import math

import numpy as np
import torch

import gqa_decode_attention_paged_gb300 as pkv

BS = 16


class Cache:
    """A pool with known contents: keys and values drawn for every slot, tables of shuffled blocks."""

    def __init__(self, kv, n_kv, d, lens, seed=0, table_extra=1, sharp=1.0, shift=0.0):
        g = torch.Generator().manual_seed(seed)
        self.kv, self.n_kv, self.d, self.lens = kv, n_kv, d, list(lens)
        need = [(c + BS - 1) // BS for c in lens]
        self.blocks = sum(need) + 2
        self.W = max(need + [0]) + table_extra
        order = torch.randperm(self.blocks, generator=g).tolist()
        self.tables = torch.full((len(lens), self.W), -1, dtype=torch.int32)
        at = 0
        for b, n in enumerate(need):
            self.tables[b, :n] = torch.tensor(order[at:at + n], dtype=torch.int32)
            at += n
        shape = (self.blocks, n_kv, BS, d)
        k = torch.randn(shape, generator=g) * sharp
        v = torch.randn(shape, generator=g) + shift
        self.pool = pkv.kv_pool_create(self.blocks, BS, n_kv, d, pkv.BF16 if kv == "bf16" else pkv.FP8_E4M3)
        if kv == "bf16":
            self.k, self.v = k.to(torch.bfloat16), v.to(torch.bfloat16)
            self.k64, self.v64 = self.k.double(), self.v.double()
        else:
            ks, vs = ((0.8 + 0.4 * torch.rand(n_kv, generator=g)) * 5 * max(1.0, sharp) / 448 for _ in range(2))
            self.pool.set_fp8_scales(ks.numpy(), vs.numpy())
            ks, vs = ks.view(1, n_kv, 1, 1), vs.view(1, n_kv, 1, 1)
            self.k, self.v = ((x / s).clamp(-448, 448).to(torch.float8_e4m3fn) for x, s in ((k, ks), (v, vs)))
            self.k64, self.v64 = self.k.double() * ks.double(), self.v.double() * vs.double()
        self.upload()

    def upload(self):
        self.pool.k_view().copy_(self.k.view(torch.uint8).cuda())
        self.pool.v_view().copy_(self.v.view(torch.uint8).cuda())

    def poison(self, b):
        """NaN in every slot of sequence b's last block behind its length."""
        c = self.lens[b]
        if c % BS:
            blk = int(self.tables[b, c // BS])
            nan = torch.full((self.n_kv, BS - c % BS, self.d), math.nan).to(self.k.dtype)
            self.k.view(torch.uint8)[blk, :, c % BS:] = nan.view(torch.uint8)
            self.v.view(torch.uint8)[blk, :, c % BS:] = nan.view(torch.uint8)

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.pool.close()


def weights(d, seed=0, lambda_init=0.6, norm=True, eps=1e-5):
    g = torch.Generator().manual_seed(1000 + seed)
    lam = 0.2 * torch.randn(4, d, generator=g)
    w = 1.0 + 0.2 * torch.randn(2 * d, generator=g) if norm else None
    return pkv.DiffParams(lam.cuda(), lambda_init, norm_weight=None if w is None else w.cuda(), eps=eps)


def plain(cache, q, indptr, lens, scale, params, skip=()):
    """(out, bound) [rows, n_q / 2, 2 d] of the chunks' rows: token i of sequence b sees positions
    0 .. lens[b] - T_b + i; `skip`: (sequence, block index) pairs that count as masked."""
    d, n_kv = cache.d, cache.n_kv
    rows, n_q, _ = q.shape
    G = n_q // n_kv
    a = params.lambdas.double().cpu()
    lam = math.exp(float(a[0] @ a[1])) - math.exp(float(a[2] @ a[3])) + params.lambda_init
    w = torch.ones(2 * d, dtype=torch.float64) if params.norm_weight is None else params.norm_weight.double().cpu()
    half = 2.0 ** -8 if cache.kv == "bf16" else 2.0 ** -11
    out = torch.zeros(rows, n_q // 2, 2 * d, dtype=torch.float64)
    bound = torch.zeros_like(out)
    q = q.double().cpu()
    for b, c in enumerate(lens):
        lo, hi = int(indptr[b]), int(indptr[b + 1])
        t = hi - lo
        if t <= 0 or c <= 0:
            continue
        ids = cache.tables[b, :(c + BS - 1) // BS].long().clamp(0, cache.blocks - 1)
        k = cache.k64[ids].transpose(0, 1).reshape(n_kv, -1, d)[:, :c]
        v = cache.v64[ids].transpose(0, 1).reshape(n_kv, -1, d)[:, :c]
        see = torch.ones(t, c, dtype=torch.bool).tril(c - t)
        for sb, sj in skip:
            if sb == b:
                see[:, sj * BS:(sj + 1) * BS] = False
        hidden = ~see.any(0)
        for h in range(n_q // 2):
            p = h // G
            vv = torch.cat((v[2 * p], v[2 * p + 1]), -1)
            vv = torch.where(hidden[:, None], torch.zeros_like(vv), vv)
            o, size = 0.0, 0.0
            for m, f in ((0, 1.0), (1, -lam)):
                s = (q[lo:hi, 2 * h + m] @ k[2 * p + m].t()) * float(np.float32(scale))
                s = s.masked_fill(~see, -math.inf)
                e = (s - s.amax(-1, keepdim=True).clamp(min=-1e300)).exp()
                total = e.sum(-1, keepdim=True)
                pr = torch.where(total > 0, e / total, torch.zeros_like(e))
                o = o + f * (pr @ vv)
                size = size + abs(f) * (pr @ vv.abs())
                if cache.kv != "bf16":  # subnormal f16 weights, against a sum of at least 1
                    size = size + abs(f) * 2.0 ** -25 / half * see.sum(-1, keepdim=True) * vv.abs().amax()
            r = 1 / (o.square().mean(-1, keepdim=True) + params.eps).sqrt()
            err = (half + 2.0 ** -12) * size
            f = (1 - params.lambda_init) * w
            out[lo:hi, h] = o * r * f
            bound[lo:hi, h] = 1.1 * f.abs() * r * (err + o.abs() * r * err.square().mean(-1, keepdim=True).sqrt())
    return out, bound + 2.0 ** -8 * out.abs() + 1e-30


def check(got, ref, bound, norm2=True):
    got = got.double().cpu()
    assert torch.isfinite(got).all()
    err = (got - ref).abs()
    assert (err <= bound).all(), f"worst: {float((err / bound).max()):.3g} of the bound"
    if norm2 and ref.numel():
        rel = float((got - ref).norm() / ref.norm())
        assert rel <= 2.0 ** -8, f"2-norm: {rel:.2e}"
