"""The rotary cache write where numbers are far, large or shared with the plain append."""
import math

import numpy as np
import pytest
import torch

import gqa_decode_attention_paged_gb300 as pkv
from test_turn import BITS, TURNS

BS = 16


def radians(pos, f):
    """pos * f modulo a turn, from exact arithmetic."""
    num, den = float(f).as_integer_ratio()
    return float(((num * int(pos) * TURNS << 64) // (den << BITS)) % 2 ** 64) * 2.0 ** -64 * 2 * math.pi


@pytest.mark.gpu
def test_rope_append_turns_by_fast_frequencies_at_far_positions():
    """Frequencies up to 2^20 radians a position, positions up to 2^31: |angle error| <= 2^-32 turns (2^-29.3
    radians), so the tolerance of near positions holds, 2^-21 (|a| + |b|) + 2^-8 |y|."""
    T, n_q, d = 64, 2, 64
    rng = np.random.default_rng(8)
    inv = rng.uniform(0.5, 1, 32) * 2.0 ** np.linspace(-5, 20, 32)
    inv[-1] = 2.0 ** 20
    pos = (rng.integers(0, 2 ** 20, (1, T)) - 2 ** 31).astype(np.int64)
    pos[0, ::2] = 2 ** 31 - 1 - pos[0, ::2] % 997
    q, k, v = (torch.from_numpy(rng.normal(size=(T, h, d)).astype(np.float32)).to(torch.bfloat16).cuda() for h in (n_q, 1, 1))
    with pkv.kv_pool_create(T // BS, BS, 1, d, pkv.BF16) as pool:
        got = pkv.paged_rope_append(pool, pkv.Rope(inv), q, k, v, torch.from_numpy(pos.astype(np.int32)).cuda(),
                                    torch.arange(T, device="cuda"))
        keys = pool.k_view().view(torch.bfloat16).transpose(1, 2).reshape(T, 1, d).double().cpu().numpy()
    ang = np.array([[radians(p, f) for f in inv] for p in pos[0]])[:, None]
    c, s = np.cos(ang), np.sin(ang)
    for x, y in ((q.double().cpu().numpy(), got.double().cpu().numpy()), (k.double().cpu().numpy(), keys)):
        a, b = x[..., :32], x[..., 32:]
        ref = np.concatenate((a * c - b * s, b * c + a * s), -1)
        size = np.tile(np.abs(a) + np.abs(b), 2)
        assert (np.abs(y - ref) <= 2.0 ** -21 * size + 2.0 ** -8 * np.abs(ref)).all()


@pytest.mark.gpu
def test_rope_append_gives_every_bf16_key_the_4_bit_code_of_the_plain_append():
    """All 2^16 bit patterns as keys at position 0, with scales from one end of fp32's range to the other and zero
    points beside and far from them: the same bytes as the append's correctly rounded quotient."""
    d, free = 128, 112  # channels that turn (the first 16) hold 0: one that is not finite spoils its pair's other one
    scales = np.float32([1e-45, 1e-39, 2.0 ** -126, 1e-30, 0.01, 0.37, 1.0, 3.0, 1e30, 2.0 ** 125, 2.0 ** 126, 1.2e38, 3.4e38])
    n_kv = len(scales)
    ks = np.repeat(scales[:, None], d, 1)
    kz = np.clip(ks.astype(np.float64) * np.repeat([-7.5, 0.0, 1.0, -1e38], d // 4), -3e38, 3e38).astype(np.float32)
    # every pattern meets every zero point: rows of 112 patterns, four times, turned by 28 channels each time
    T = 592
    x = torch.arange(T * free, dtype=torch.int32).to(torch.int16).view(torch.bfloat16).view(T, free)
    k = torch.zeros(4 * T, n_kv, d, dtype=torch.bfloat16)
    for i in range(4):
        k[i * T:(i + 1) * T, :, 16:] = torch.roll(x, 28 * i, -1)[:, None]
    k = k.cuda()
    T *= 4
    v = torch.zeros_like(k)
    slots, pos = torch.arange(T, device="cuda"), torch.zeros(1, T, dtype=torch.int32, device="cuda")
    got = []
    for rotary in (False, True):
        with pkv.kv_pool_create(T // BS, BS, n_kv, d, pkv.INT4) as pool:
            pool.set_int4_key_params(ks, kz)
            if rotary:
                pkv.paged_rope_append(pool, pkv.Rope(np.ones(8)), None, k, v, pos, slots)
            else:
                pkv.paged_kv_append(pool, k, v, slots)
            got.append(pool.k_view().cpu().numpy())
    bad = [(float(scales[g]), int((got[0][:, g] != got[1][:, g]).sum())) for g in range(n_kv)]
    assert all(n == 0 for _, n in bad), bad


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
def test_rope_append_and_plain_append_store_4_bit_values_within_a_rounding_of_one_another(d):
    """The rows' scales are (max - min) * fp32(1/15) here and (max - min) / 15 there: fp32(1/15) is off by at most 2^-24
    of itself and each result by its rounding, 2^-24, so they differ by at most 3 * 2^-24 of the scale; the minimum
    is the same.  (v - min) / scale then differs by at most 15 * 5 * 2^-24 (each quotient is rounded, too) < 2^-17, so
    only a value that close to the border between two codes gets another one, the next, and both stand for it within
    half a step and that."""
    T, n_kv = 512, 3
    g = torch.Generator().manual_seed(d)
    v = torch.randn(T, n_kv, d, generator=g).to(torch.bfloat16)
    v[0], v[1] = 0, 2.5
    v[2] = torch.arange(d).to(torch.bfloat16)
    slots, pos = torch.arange(T, device="cuda"), torch.zeros(1, T, dtype=torch.int32, device="cuda")
    got = []
    for rotary in (False, True):
        with pkv.kv_pool_create(T // BS, BS, n_kv, d, pkv.INT4) as pool:
            pool.set_int4_key_params(np.ones((n_kv, d)), np.zeros((n_kv, d)))
            if rotary:
                pkv.paged_rope_append(pool, pkv.Rope(np.ones(8)), None, v.cuda(), v.cuda(), pos, slots)
            else:
                pkv.paged_kv_append(pool, v.cuda(), v.cuda(), slots)
            c = pool.v_view().cpu().transpose(1, 2).reshape(T, n_kv, d // 2)
            p = pool.v_params_view().cpu().transpose(1, 2).reshape(T, n_kv, 2).double()
            got.append((torch.stack((c & 15, c >> 4), -1).reshape(T, n_kv, d).double(), p[..., :1], p[..., 1:]))
    (c0, s0, z0), (c1, s1, z1) = got
    assert torch.equal(z0, z1)
    assert ((s0 - s1).abs() <= 3 * 2.0 ** -24 * s0).all()
    away = ((v.double() - z0) / s0 - (c0 + c1) / 2).abs()  # of the border between the two codes
    assert ((c0 == c1) | (((c0 - c1).abs() == 1) & (away <= 2.0 ** -17))).all()
    for c, s, z in got:
        assert ((c * s + z - v.double()).abs() <= s * (0.5 + 2.0 ** -17)).all()
