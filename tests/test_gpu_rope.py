"""The rotary cache write and the cache read-back against plain 64-bit forms.

Tolerances, elementwise, for a turned value y = a cos - b sin (or b cos + a sin):
* 32-bit arithmetic: the angle is off by at most 2^-32 turns (2^-29.3 rad) plus
  its conversion to 32 bits (half a step of a value below pi: 2^-23 rad), sine
  and cosine by 2 steps (2^-23), two products and a sum by 3 * 2^-24 of their
  size: together below 2^-21 (|a| + |b|).
* one rounding to bf16: 2^-8 |y|; to E4M3 of y / s: 2^-4 |y| or, below its
  normal range, half its smallest step, 2^-10 s.
* a 4-bit code: half a step s / 2 of the clamped value (and 2^-20 of the
  numbers that make it up, in 32 bits).
"""
import ctypes

import numpy as np
import pytest
import torch

import gqa_decode_attention_paged_gb300 as pkv
import oracle
import workloads as wl

BS = 16


def f32(t):
    return t.float().cpu().numpy().astype(np.float64)


def turned64(x, positions, inv_freq, axis, inter):
    """x [T, H, D] float64 turned, and |a| + |b| of each value's pair."""
    out, size = x.copy(), np.abs(x)
    n = len(inv_freq)
    ang = positions.astype(np.float64)[axis].T * inv_freq  # [T, pairs]
    c, s = np.cos(ang)[:, None], np.sin(ang)[:, None]
    i, j = (slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if inter else (slice(0, n), slice(n, 2 * n))
    a, b = x[..., i], x[..., j]
    out[..., i], out[..., j] = a * c - b * s, b * c + a * s
    size[..., i] = size[..., j] = np.abs(a) + np.abs(b)
    return out, size


def make(kv, n_kv, d, blocks, seed=0):
    rng = np.random.default_rng(seed)
    pool = pkv.kv_pool_create(blocks, BS, n_kv, d, {"bf16": pkv.BF16, "fp8": pkv.FP8_E4M3, "int4": pkv.INT4}[kv])
    ks = kz = vs = None
    if kv == "fp8":
        ks, vs = (rng.uniform(0.005, 0.02, n_kv).astype(np.float32) for _ in range(2))
        pool.set_fp8_scales(ks, vs)
    if kv == "int4":
        ks = rng.uniform(0.3, 0.5, (n_kv, d)).astype(np.float32)
        kz = (-7.5 * ks + rng.normal(size=(n_kv, d)) * 0.1).astype(np.float32)
        pool.set_int4_key_params(ks, kz)
    m = oracle.PoolMirror(blocks, BS, n_kv, d, {"bf16": oracle.BF16, "fp8": oracle.E4M3, "int4": oracle.INT4}[kv],
                          ks, vs, kz)
    return pool, m


def raw(pool):
    torch.cuda.synchronize()
    return pool.k_view().cpu().numpy(), pool.v_view().cpu().numpy()


def value_rows4(v):
    """Codes and (scale, zero point) of 4-bit value rows [T, n_kv, d] bf16, in 32-bit arithmetic:
    scale = (max - min) * fp32(1/15) (1 if 0), zero point = min, code = rint((v - min) / scale)."""
    x = v.float().cpu().numpy()
    z = x.min(-1, keepdims=True) + np.float32(0)
    s = (x.max(-1, keepdims=True) - z) * np.float32(1 / 15)
    s = np.where(s == 0, np.float32(1), s)
    c = np.clip(np.rint((x - z) / s), 0, 15).astype(np.uint8)
    return c[..., 0::2] | (c[..., 1::2] << 4), np.concatenate((s, z), -1)


def expect_values(m, v, slots):
    """The mirror's values after v went to slots, as paged_rope_append stores them."""
    if m.dtype != oracle.INT4:
        return
    codes, params = value_rows4(v)
    for t, s in enumerate(slots):
        if 0 <= s < m.num_blocks * BS:
            m.v[s // BS, :, s % BS], m.v_params[s // BS, :, s % BS] = codes[t], params[t]


def dev(a, dt):
    return torch.from_numpy(np.ascontiguousarray(a)).to("cuda").to(dt)


def bits(t):
    return t.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)


CASES = [  # kv, T, n_q, n_kv, d, rot, axes, inter
    ("bf16", 1, 8, 2, 64, 64, 1, False),
    ("bf16", 37, 7, 3, 128, 128, 3, False),
    ("bf16", 5, 64, 8, 128, 32, 1, True),
    ("bf16", 300, 1, 1, 64, 16, 2, False),
    ("fp8", 1, 32, 8, 128, 128, 1, False),
    ("fp8", 130, 12, 3, 64, 32, 3, True),
    ("fp8", 2000, 8, 2, 128, 96, 1, False),
    ("int4", 3, 8, 2, 128, 128, 3, True),
    ("int4", 129, 5, 5, 64, 48, 1, False),
    ("int4", 900, 16, 4, 128, 64, 1, True),
]


def _inputs(kv, T, n_q, n_kv, d, rot, axes, inter, seed=3, far=False):
    rng = np.random.default_rng([seed, T, n_q])
    x = [torch.from_numpy(rng.normal(size=(T, h, d)).astype(np.float32)).to(torch.bfloat16).cuda()
         for h in (n_q, n_kv, n_kv)]
    lim = 2 ** 31 - 1 if far else 200000
    pos = rng.integers(-lim if far else 0, lim, size=(axes, T)).astype(np.int32)
    inv = 10000.0 ** (-np.arange(rot // 2) / (rot // 2))
    axis = rng.integers(0, axes, rot // 2)
    axis[0] = axes - 1
    return x, pos, inv, axis


@pytest.mark.gpu
@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
@pytest.mark.parametrize("far", [False, True])
def test_rope_append_matches_the_64_bit_form(case, far):
    kv, T, n_q, n_kv, d, rot, axes, inter = case
    (q, k, v), pos, inv, axis = _inputs(*case, far=far)
    blocks = T // BS + 2
    rng = np.random.default_rng(5)
    slots = rng.permutation(blocks * BS)[:T].astype(np.int64)
    pool, m = make(kv, n_kv, d, blocks)
    with pool:
        rope = pkv.Rope(inv, axis, interleaved=inter, n_axes=axes)
        got = pkv.paged_rope_append(pool, rope, q, k, v, dev(pos, torch.int32), dev(slots, torch.int64))
        kb, vb = raw(pool)
        assert pool.get_error() == 0
        m.append(bits(k), bits(v), slots)  # values: what an append stores
        expect_values(m, v, slots)
        assert np.array_equal(vb, m.v.view(np.uint8).reshape(vb.shape))
        if kv == "int4":
            assert np.array_equal(pool.v_params_view().cpu().numpy(), m.v_params)
    for name, x, y in (("q", q, f32(got)), ("k", k, None)):
        ref, size = turned64(f32(x), pos, inv, axis, inter)
        tol = 2.0 ** -21 * size
        if name == "q" or kv == "bf16":
            tol = tol + 2.0 ** -8 * np.abs(ref)
        if name == "k":
            st = kb[slots // BS, :, slots % BS]  # [T, n_kv, row bytes]
            if kv == "bf16":
                y = f32(torch.from_numpy(st.copy()).view(torch.bfloat16))
            elif kv == "fp8":
                s = m.k_scale.astype(np.float64)[None, :, None]
                y = f32(torch.from_numpy(st.copy()).view(torch.float8_e4m3fn)) * s
                ref = np.clip(ref, -448 * s, 448 * s)
                tol = tol + np.maximum(2.0 ** -4 * np.abs(ref), 2.0 ** -10 * s)
            else:
                s, z = m.k_scale.astype(np.float64), m.k_zero.astype(np.float64)
                y = np.stack((st & 15, st >> 4), -1).reshape(T, n_kv, d) * s + z
                ref = np.clip(ref, z, z + 15 * s)
                tol = tol + s / 2 + 2.0 ** -20 * (np.abs(ref) + np.abs(z) + 15 * s)
        assert (np.abs(y - ref) <= tol).all(), (name, np.max(np.abs(y - ref) - tol))


@pytest.mark.gpu
@pytest.mark.parametrize("kv", ["bf16", "fp8", "int4"])
def test_rope_append_at_position_zero_is_the_plain_append(kv):
    T, n_kv, d = 70, 4, 128
    (q, k, v), pos, inv, axis = _inputs(kv, T, 6, n_kv, d, 128, 1, False)
    slots = np.random.default_rng(1).permutation(96)[:T].astype(np.int64)
    pool, m = make(kv, n_kv, d, 6)
    with pool:
        got = pkv.paged_rope_append(pool, pkv.Rope(inv), q, k, v, dev(pos * 0, torch.int32), dev(slots, torch.int64))
        kb, vb = raw(pool)
    m.append(bits(k), bits(v), slots)
    expect_values(m, v, slots)
    assert torch.equal(got, q)
    assert np.array_equal(kb, m.k.view(np.uint8).reshape(kb.shape))
    assert np.array_equal(vb, m.v.view(np.uint8).reshape(vb.shape))


@pytest.mark.gpu
def test_rope_append_rounds_every_bf16_value_to_the_e4m3_of_the_plain_append():
    """All 2^16 bit patterns (zeros of both signs, subnormals, infinities and NaN among them) as values, divided by
    scales from one end of fp32's range to the other: the same bytes as the append's correctly rounded division."""
    scales = np.float32([1e-37, 2.0 ** -61, 1.1e-18, 0.0078, 0.3, 1.0, 448.0 / 3, 1.1e18, 2.0 ** 61, 3e38, 1.9999999, 0.1])
    d, n_kv, T = 128, len(scales), 512
    v = torch.arange(2 ** 16, dtype=torch.int32).to(torch.int16).view(torch.bfloat16).view(T, 1, d).repeat(1, n_kv, 1).cuda()
    q, k = torch.zeros(T, 2 * n_kv, d, dtype=torch.bfloat16, device="cuda"), torch.zeros_like(v)
    slots, pos = torch.arange(T, device="cuda"), torch.zeros(1, T, dtype=torch.int32, device="cuda")
    rope = pkv.Rope(np.ones(16))
    got = []
    for rotary in (False, True):
        with pkv.kv_pool_create(T // BS, BS, n_kv, d, pkv.FP8_E4M3) as pool:
            pool.set_fp8_scales(scales, scales)
            if rotary:
                pkv.paged_rope_append(pool, rope, q, k, v, pos, slots)
            else:
                pkv.paged_kv_append(pool, k, v, slots)
            got.append(raw(pool)[1])
    assert np.array_equal(*got)


@pytest.mark.gpu
@pytest.mark.parametrize("kv", ["bf16", "int4"])
def test_rope_append_from_a_fused_projection_in_place(kv):
    """q, k and v as slices of one [T, heads, d] array, q turned in place: the same bytes as from
    separate arrays, and nothing else of the array is touched."""
    T, n_q, n_kv, d = 45, 6, 2, 64
    (q, k, v), pos, inv, axis = _inputs(kv, T, n_q, n_kv, d, 64, 1, True)
    slots = np.arange(T, dtype=np.int64) + 3
    pool, _ = make(kv, n_kv, d, 4)
    other, _ = make(kv, n_kv, d, 4)
    rope = pkv.Rope(inv, interleaved=True)
    with pool, other:
        p, s = dev(pos, torch.int32), dev(slots, torch.int64)
        want = pkv.paged_rope_append(pool, rope, q, k, v, p, s)
        fused = torch.cat((q, k, v, torch.full_like(v, 7.0)), dim=1)
        a, b, c = fused[:, :n_q], fused[:, n_q:n_q + n_kv], fused[:, n_q + n_kv:n_q + 2 * n_kv]
        got = pkv.paged_rope_append(other, rope, a, b, c, p, s, q_out=a)
        assert got is a
        for x, y in zip(raw(pool), raw(other)):
            assert np.array_equal(x, y)
        assert torch.equal(fused, torch.cat((want, k, v, torch.full_like(v, 7.0)), dim=1))
        # keys and values only
        pkv.paged_rope_append(other, rope, None, b, c, p, s)
        for x, y in zip(raw(pool), raw(other)):
            assert np.array_equal(x, y)


@pytest.mark.gpu
@pytest.mark.parametrize("kv", ["bf16", "fp8", "int4"])
def test_rope_append_skips_padding_and_flags_slots_past_the_pool(kv):
    T, n_kv, d = 20, 2, 64
    (q, k, v), pos, inv, axis = _inputs(kv, T, 4, n_kv, d, 64, 1, False)
    slots = np.arange(T, dtype=np.int64)
    slots[[0, 7]] = -1
    slots[[3, 19]] = [32, 2 ** 40]
    pool, m = make(kv, n_kv, d, 2)
    with pool:
        got = pkv.paged_rope_append(pool, pkv.Rope(inv), q, k, v, dev(pos, torch.int32), dev(slots, torch.int64))
        kb, vb = raw(pool)
        assert pool.get_error(clear=True) == pkv.DEVERR_SLOT_RANGE
        assert m.append(bits(k), bits(v), slots) == 2
        expect_values(m, v, slots)
        assert np.array_equal(vb, m.v.view(np.uint8).reshape(vb.shape))
        assert (kb[0, :, [0, 3, 7]] == 0).all() and (kb[1, :, 4:] == 0).all()  # rows no token wrote
        ref, size = turned64(f32(q), pos, inv, axis, False)
        assert (np.abs(f32(got) - ref) <= 2.0 ** -21 * size + 2.0 ** -8 * np.abs(ref)).all()  # all tokens' queries
        pkv.paged_rope_append(pool, pkv.Rope(inv), q[:0], k[:0], v[:0], dev(pos[:, :0], torch.int32),
                              dev(slots[:0], torch.int64))
        assert pool.get_error() == 0


@pytest.mark.gpu
def test_rope_append_refusals():
    T, n_kv, d = 4, 2, 64
    pool, _ = make("bf16", n_kv, d, 2)
    with pool:
        q, k, v = (torch.zeros(T, h, d, dtype=torch.bfloat16, device="cuda") for h in (4, 2, 2))
        pos, slots = dev(np.zeros((1, T)), torch.int32), dev(np.arange(T), torch.int64)
        rope = pkv.Rope(np.ones(32))
        ok = dict(q=q, k_new=k, v_new=v, positions=pos, slot_mapping=slots)
        both = torch.zeros(T + 1, 4, d, dtype=torch.bfloat16, device="cuda")
        for change, err in [
            (dict(q=q.float()), ValueError), (dict(k_new=k[:3]), ValueError), (dict(q=q.cpu()), ValueError),
            (dict(v_new=v[..., :32]), ValueError), (dict(positions=pos[0]), ValueError),
            (dict(positions=dev(np.zeros((2, T)), torch.int32)), ValueError),
            (dict(slot_mapping=slots.int()), ValueError), (dict(q=q.transpose(0, 1).contiguous().transpose(0, 1)), ValueError),
            (dict(q=None, q_out=q), ValueError),
            (dict(q=both[:T], q_out=both[1:]), pkv.PagedKVError),      # overlaps q without being q
            (dict(q_out=torch.cat((k, v), 1)[:, :4], k_new=both[:T, :2], q=both[1:]), None),
            (dict(q_out=both[:T], k_new=both[:T, :2]), pkv.PagedKVError),  # overwrites the keys
            (dict(k_new=torch.zeros(T * n_kv * d + 1, dtype=torch.bfloat16, device="cuda")[1:].view(T, n_kv, d)),
             pkv.PagedKVError),                                       # 2-byte aligned
        ]:
            if err is None:
                pkv.paged_rope_append(pool, rope, **{**ok, **change})
                continue
            with pytest.raises(err):
                pkv.paged_rope_append(pool, rope, **{**ok, **change})
        with pytest.raises(pkv.PagedKVError):
            pkv.paged_rope_append(pool, pkv.Rope(np.ones(64)), **ok)  # rot_dim 128 on 64-channel heads
        with pytest.raises(pkv.PagedKVError):
            with pkv.kv_pool_create(2, BS, n_kv, d, pkv.FP8_E4M3) as unset:
                pkv.paged_rope_append(unset, rope, **ok)
        torch.cuda.synchronize()
        assert pool.get_error() == 0


def test_rope_create_refusals():
    lib, out = pkv.load(), ctypes.c_void_p()
    f = np.ones(64)
    ax = np.zeros(64, np.int32)

    def st(rot=64, inter=0, axes=1, freq=f, axis=ax):
        return lib.pkv_rope_create(rot, inter, axes, None if freq is None else freq.ctypes.data,
                                   None if axis is None else axis.ctypes.data, ctypes.byref(out))

    assert [st(rot=r) for r in (0, -16, 24, 144)] == [5, 5, 5, 5]
    assert st(inter=2) == 1 and st(axes=0) == 1 and st(axes=9) == 1 and st(freq=None) == 1
    for bad in (np.nan, np.inf, -np.inf, 2.0 ** 21):
        g = f.copy()
        g[31] = bad
        assert st(freq=g) == 1
        g = f.copy()
        g[32] = bad  # past rot_dim / 2: not looked at
        assert st(freq=g) == 0
        lib.pkv_rope_destroy(out)
    assert st(axis=ax + 1) == 1 and st(axis=ax - 1) == 1
    assert st(axis=None) == 0
    lib.pkv_rope_destroy(out)
    lib.pkv_rope_destroy(None)
    assert lib.pkv_rope_create(64, 0, 1, f.ctypes.data, None, None) == 1
    with pytest.raises(ValueError):
        pkv.Rope(f[:32], ax)
    assert pkv.Rope(f[:32], [2, 0] * 16).n_axes == 3
    assert lib.paged_rope_append(None, None, None, 0, 0, None, 0, None, 0, None, None, 1, None, 0, None) == 1
    assert lib.paged_kv_gather(None, None, None, 1, None, 1, 1, None, None, None) == 1


# ------------------------------------------------------------------ read-back

def rows64(m, tables, starts, lens):
    """What sequence b's positions starts[b] .. starts[b] + lens[b] - 1 stand for, in 64 bits."""
    out = []
    for which, r in (("k", m.k), ("v", m.v)):
        if m.dtype == oracle.BF16:
            x = wl.bf16_bits_to_f32(r).astype(np.float64)
        elif m.dtype == oracle.E4M3:
            s = m.k_scale if which == "k" else m.v_scale
            x = torch.from_numpy(r).view(torch.float8_e4m3fn).double().numpy() * s.astype(np.float64)[:, None, None]
        else:
            c = np.stack((r & 15, r >> 4), -1).reshape(*r.shape[:3], -1).astype(np.float64)
            if which == "k":
                x = c * m.k_scale.astype(np.float64)[:, None] + m.k_zero.astype(np.float64)[:, None]
            else:
                p = m.v_params.astype(np.float64)
                x = c * p[..., :1] + p[..., 1:]
        rows = [x[tables[b, p // BS], :, p % BS] for b in range(len(lens)) for p in range(starts[b], starts[b] + lens[b])]
        out.append(np.stack(rows) if rows else np.zeros((0, m.n_kv, m.d_head)))
    return out


def as_bf16(x):
    return torch.from_numpy(x.astype(np.float32)).to(torch.bfloat16)


def _filled(kv, n_kv, d, blocks, seed=0):
    rng = np.random.default_rng([seed, n_kv])
    T = blocks * BS
    k, v = (wl.f32_to_bf16_bits(rng.normal(size=(T, n_kv, d)).astype(np.float32)) for _ in range(2))
    pool, m = make(kv, n_kv, d, blocks)
    slots = np.arange(T, dtype=np.int64)
    m.append(k, v, slots)
    to = lambda a: torch.from_numpy(a.view(np.int16)).view(torch.bfloat16).cuda()  # noqa: E731
    pkv.paged_kv_append(pool, to(k), to(v), dev(slots, torch.int64))
    return pool, m


@pytest.mark.gpu
@pytest.mark.parametrize("kv", ["bf16", "fp8", "int4"])
@pytest.mark.parametrize("n_kv,d,lens,starts", [
    (2, 64, [1, 17, 0, 100, 16], [0, 3, 5, 15, 16]),
    (8, 128, [300, 1, 33], [0, 0, 31]),
    (1, 128, [5], [0]),
    (3, 64, [0, 0, 7, 0], None),
    (5, 128, [64, 31], [1, 2]),
    (40, 64, [20, 9], [0, 40]),
])
def test_gather_gives_what_the_rows_stand_for(kv, n_kv, d, lens, starts):
    B = len(lens)
    st = np.zeros(B, np.int64) if starts is None else np.array(starts)
    need = [(a + b + BS - 1) // BS for a, b in zip(st, lens)]
    blocks, W = sum(need) + 1, max(need) + 1
    ids = np.random.default_rng(2).permutation(blocks)
    tables = np.full((B, W), -7, np.int32)
    at = 0
    for b, n in enumerate(need):
        tables[b, :n] = ids[at:at + n]
        at += n
    pool, m = _filled(kv, n_kv, d, blocks)
    with pool:
        indptr = np.concatenate([[0], np.cumsum(lens)])
        k, v = pkv.paged_kv_gather(pool, dev(indptr, torch.int32), dev(tables, torch.int32),
                                   None if starts is None else dev(st, torch.int32), n_rows=int(indptr[-1]))
        torch.cuda.synchronize()
        assert pool.get_error() == 0
        for got, want in zip((k, v), rows64(m, tables, st, lens)):
            assert torch.equal(got.cpu(), as_bf16(want))


@pytest.mark.gpu
@pytest.mark.parametrize("kv", ["bf16", "int4"])
def test_gather_leaves_uncovered_rows_and_zeroes_bad_ones(kv):
    n_kv, d = 2, 128
    pool, m = _filled(kv, n_kv, d, 8)
    with pool:
        tables = np.array([[3, 99], [-1, 5]], np.int32)
        indptr = np.array([2, 22, 60], np.int32)  # rows 0, 1 and 60.. belong to nobody
        k, v = (torch.full((70, n_kv, d), 9.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        pkv.paged_kv_gather(pool, dev(indptr, torch.int32), dev(tables, torch.int32), dev([0, -2], torch.int32),
                            k_out=k, v_out=v)
        torch.cuda.synchronize()
        assert pool.get_error(clear=True) == pkv.DEVERR_BLOCK_RANGE | pkv.DEVERR_CTX_RANGE
        want = rows64(m, np.array([[3, 3], [5, 5]]), [0, 0], [16, 16])
        for got, w in zip((k.cpu(), v.cpu()), want):
            assert (got[:2] == 9).all() and (got[60:] == 9).all()
            assert torch.equal(got[2:18], as_bf16(w[:16]))
            assert (got[18:22] == 0).all()            # block 99 of 8
            assert (got[22:40] == 0).all()            # positions -2, -1, then block -1
            assert torch.equal(got[40:56], as_bf16(w[16:]))
            assert (got[56:60] == 0).all()            # positions past the table
        # fewer rows than the indptr says: the rest is not written
        k2, v2 = (torch.full((10, n_kv, d), 9.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        pkv.paged_kv_gather(pool, dev(indptr, torch.int32), dev(tables, torch.int32), k_out=k2[:5], v_out=v2[:5])
        torch.cuda.synchronize()
        assert (k2[5:] == 9).all() and (v2[5:] == 9).all() and torch.equal(k2[2:5].cpu(), k[2:5].cpu())


@pytest.mark.gpu
def test_gather_refusals():
    pool, _ = make("bf16", 2, 64, 2)
    with pool:
        ip, tb = dev([0, 4], torch.int32), dev([[0, 1]], torch.int32)
        out = torch.zeros(8, 2, 64, dtype=torch.bfloat16, device="cuda")
        for args in [dict(), dict(k_out=out), dict(n_rows=3, k_out=out, v_out=out.clone()),
                     dict(k_out=out, v_out=out[:4]), dict(n_rows=4, starts=dev([0, 0], torch.int32))]:
            with pytest.raises(ValueError):
                pkv.paged_kv_gather(pool, ip, tb, **args)
        with pytest.raises(ValueError):
            pkv.paged_kv_gather(pool, ip, tb.long(), n_rows=4)
        with pytest.raises(pkv.PagedKVError):
            pkv.paged_kv_gather(pool, ip, tb, k_out=out[:4], v_out=out[3:7])  # overlapping outputs
        k, v = pkv.paged_kv_gather(pool, dev([0], torch.int32), tb[:0], n_rows=0)
        assert k.shape == (0, 2, 64)


@pytest.mark.gpu
@pytest.mark.parametrize("kv", ["bf16", "fp8", "int4"])
def test_write_and_read_back_on_a_side_stream_and_in_a_graph(kv):
    T, n_q, n_kv, d = 50, 4, 2, 128
    (q, k, v), pos, inv, axis = _inputs(kv, T, n_q, n_kv, d, 128, 1, False)
    slots = np.random.default_rng(4).permutation(64)[:T].astype(np.int64)
    tables = np.arange(4, dtype=np.int32)[None]
    a, _ = make(kv, n_kv, d, 4)
    b, _ = make(kv, n_kv, d, 4)
    rope = pkv.Rope(inv)
    with a, b:
        p, s, tb, ip = dev(pos, torch.int32), dev(slots, torch.int64), dev(tables, torch.int32), dev([0, 64], torch.int32)
        want = (pkv.paged_rope_append(a, rope, q, k, v, p, s), *pkv.paged_kv_gather(a, ip, tb, n_rows=64))
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        qs = torch.zeros_like(q)
        with torch.cuda.stream(side):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=side):
                o = pkv.paged_rope_append(b, rope, qs, k, v, p, s)
                kk, vv = pkv.paged_kv_gather(b, ip, tb, n_rows=64)
            del rope
            for _ in range(2):
                qs.copy_(q)
                g.replay()
        side.synchronize()
        for x, y in zip(want, (o, kk, vv)):
            assert torch.equal(x, y)


@pytest.mark.gpu
@pytest.mark.parametrize("kv", ["bf16", "int4"])
def test_a_view_keeps_its_pool_alive(kv):
    import gc
    import weakref

    pool, _ = make(kv, 2, 64, 3)
    alive = weakref.ref(pool)
    views = [pool.k_view(), pool.v_view()[1:].view(torch.int8)] + ([pool.v_params_view()] if kv == "int4" else [])
    del pool
    gc.collect()
    while views:
        assert alive() is not None
        views.pop()
    gc.collect()
    assert alive() is None
