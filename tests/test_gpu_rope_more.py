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
