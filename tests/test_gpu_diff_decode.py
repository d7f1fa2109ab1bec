"""Differential decode attention against the plain 64-bit form (diff_ref.py)."""
import ctypes

import numpy as np
import pytest
import torch

import gqa_decode_attention_paged_gb300 as pkv
from diff_ref import BS, Cache, check, plain, weights


def queries(B, n_q, d, seed=0):
    g = torch.Generator().manual_seed(77 + seed)
    return torch.randn(B, n_q, d, generator=g).to(torch.bfloat16).cuda()


def decode(c, q, params, lens=None, tables=None, **kw):
    lens = c.lens if lens is None else lens
    tables = c.tables if tables is None else tables
    return pkv.paged_diff_decode_attention(c.pool, q, tables.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(),
                                           1 / np.sqrt(c.d), params, **kw)


LENS = [1, 300, 0, 16, 17, 15, 2000, 0, 31]


@pytest.mark.gpu
@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("G", [1, 2, 4, 8])
@pytest.mark.parametrize("part", [0, 16, 128])
def test_diff_decode_matches_the_64_bit_form(kv, d, G, part):
    with Cache(kv, 4, d, LENS, seed=G) as c:
        for b in range(len(LENS)):
            c.poison(b)
        c.upload()
        c.pool.set_partition_tokens(part)
        q, params = queries(len(LENS), 4 * G, d, G), weights(d, G)
        out = torch.full((len(LENS), 2 * G, 2 * d), 5.0, dtype=torch.bfloat16, device="cuda")
        got = decode(c, q, params, out=out)
        torch.cuda.synchronize()
        assert got is out and c.pool.get_error() == 0
        check(got, *plain(c, q, np.arange(len(LENS) + 1), LENS, 1 / np.sqrt(d), params))
        assert (got[[2, 7]] == 0).all()
        assert torch.equal(got, decode(c, q, params))  # the same bits again


@pytest.mark.gpu
@pytest.mark.parametrize("kv,n_kv,G,lens", [
    ("bf16", 2, 4, [1]), ("bf16", 2, 1, [20000]), ("fp8", 2, 8, [9000]), ("bf16", 16, 2, [40] * 50),
    ("fp8", 6, 4, list(range(0, 200, 3))), ("bf16", 256, 1, [33, 5]), ("bf16", 2, 8, [700] * 300),
])
def test_diff_decode_shapes(kv, n_kv, G, lens):
    d = 128 if G != 8 else 64
    with Cache(kv, n_kv, d, lens, seed=5) as c:
        q, params = queries(len(lens), n_kv * G, d), weights(d, norm=G != 2, lambda_init=0.2)
        got = decode(c, q, params)
        torch.cuda.synchronize()
        assert c.pool.get_error() == 0
        check(got, *plain(c, q, np.arange(len(lens) + 1), lens, 1 / np.sqrt(d), params))


@pytest.mark.gpu
@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_diff_decode_sharp_maps_and_values_off_zero(kv):
    """Scores up to a few dozen (few positions weigh), rising along the sequence so that the reference
    maximum is raised again and again, and values whose mean is far from zero."""
    lens = [400, 1000]
    with Cache(kv, 2, 128, lens, seed=9, sharp=2.0, shift=1.5) as c:
        q, params = 2 * queries(2, 8, 128), weights(128)
        got = decode(c, q, params)
        torch.cuda.synchronize()
        check(got, *plain(c, q, np.arange(3), lens, 1 / np.sqrt(128), params), norm2=False)


@pytest.mark.gpu
@pytest.mark.parametrize("part", [0, 32])
def test_diff_decode_bad_blocks_are_masked_and_flagged(part):
    lens = [100, 64, 200]
    with Cache("bf16", 2, 64, lens, seed=2) as c:
        c.pool.set_partition_tokens(part)
        tables = c.tables.clone()
        tables[0, 2], tables[2, 0] = c.blocks, -5
        tables[1, :4] = 10 ** 6  # nothing of sequence 1 can be read
        q, params = queries(3, 4, 64), weights(64)
        got = decode(c, q, params, tables=tables)
        torch.cuda.synchronize()
        assert c.pool.get_error(clear=True) == pkv.DEVERR_BLOCK_RANGE
        skip = [(0, 2), (2, 0)] + [(1, j) for j in range(4)]
        check(got, *plain(c, q, np.arange(4), lens, 1 / np.sqrt(64), params, skip=skip))
        assert (got[1] == 0).all()


@pytest.mark.gpu
def test_diff_decode_lengths_out_of_range_are_clamped_and_flagged():
    lens = [50, 16, 10]
    with Cache("bf16", 2, 64, lens, table_extra=0) as c:  # tables of 4 blocks
        q, params = queries(3, 2, 64), weights(64)
        c.tables[0, :4] = torch.arange(4)
        got = decode(c, q, params, lens=[65, -1, 10])
        torch.cuda.synchronize()
        assert c.pool.get_error(clear=True) == pkv.DEVERR_CTX_RANGE
        check(got, *plain(c, q, np.arange(4), [64, 0, 10], 1 / np.sqrt(64), params))


@pytest.mark.gpu
def test_diff_decode_8192_sequences():
    lens = [(7 * i) % 41 for i in range(8192)]
    with Cache("bf16", 2, 64, lens, seed=3) as c:
        q, params = queries(8192, 2, 64), weights(64)
        got = decode(c, q, params)
        torch.cuda.synchronize()
        assert c.pool.get_error() == 0
        check(got, *plain(c, q, np.arange(8193), lens, 1 / np.sqrt(64), params))
        with pytest.raises(pkv.PagedKVError):
            decode(c, torch.cat((q, q[:1])), params, lens=lens + [1], tables=torch.cat((c.tables, c.tables[:1])))


@pytest.mark.gpu
def test_diff_decode_lambda_and_norm_follow_their_weights():
    """Without a second map (lambda 0) the result is the norm of plain decode attention; lambda_init
    scales, norm_weight weighs, eps holds tiny outputs down."""
    lens = [70, 9]
    with Cache("bf16", 2, 64, lens, seed=4) as c:
        q = queries(2, 4, 64)
        zero = torch.zeros(4, 64, device="cuda")
        w = torch.linspace(-1, 2, 128, device="cuda")
        for params in (pkv.DiffParams(zero, 0.0), pkv.DiffParams(zero, 0.9, norm_weight=w),
                       pkv.DiffParams(zero, -0.5, norm_weight=w, eps=10.0)):
            got = decode(c, q, params)
            check(got, *plain(c, q, np.arange(3), lens, 1 / np.sqrt(64), params))
        d = pkv.paged_decode_attention(c.pool, q, c.tables.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), 0.125)
        # Head 0's first query on the first half of its channels is query row 0 on KV head 0: with o the 64-bit
        # attention and r the norm's factor (ref = r o), |first - r x| <= |first - ref| + r |x - o|, where the
        # first term is within plain()'s bound and the second within the weights' and the result's rounding,
        # (2^-8 + 2^-12) sum p |v| + 2^-8 |o|
        params = pkv.DiffParams(zero, 0.0)
        first = decode(c, q, params).double().cpu()[:, 0, :64]
        ref, bound = plain(c, q, np.arange(3), lens, 0.125, params)
        x = d.double().cpu()[:, 0]
        for b, n in enumerate(lens):
            ids = c.tables[b, :(n + BS - 1) // BS].long()
            k, v = (y[ids, 0].reshape(-1, 64)[:n] for y in (c.k64, c.v64))
            pr = torch.softmax(k @ q[b, 0].double().cpu() * 0.125, 0)
            o, size = pr @ v, pr @ v.abs()
            r = float(ref[b, 0, :64] @ o / (o @ o))
            tol = bound[b, 0, :64] + r * ((2.0 ** -8 + 2.0 ** -12) * size + 2.0 ** -8 * o.abs())
            assert ((first[b] - r * x[b]).abs() <= tol).all()


@pytest.mark.gpu
def test_diff_decode_captured_and_replayed_while_other_calls_grow_the_workspace():
    lens = [3000, 40, 513]
    with Cache("bf16", 4, 128, lens, seed=6) as c:
        params = weights(128)
        q = queries(3, 8, 128)
        want = decode(c, q, params)
        static = torch.zeros_like(q)
        tables, ln = c.tables.cuda(), torch.tensor(lens, dtype=torch.int32).cuda()
        side = torch.cuda.Stream()
        c.pool.reserve_diff_workspace(3, 8, c.W)
        before = c.pool.timing_read()["workspace_bytes"]
        g = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(g, stream=side):
            out = pkv.paged_diff_decode_attention(c.pool, static, tables, ln, 1 / np.sqrt(128), params)
        assert c.pool.timing_read()["workspace_bytes"] == before
        for _ in range(2):
            static.copy_(q)
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, want)
            # a call that needs a far larger workspace replaces it; the graph keeps its own
            c.pool.set_partition_tokens(16)
            decode(c, queries(3, 32, 128), weights(128))
            c.pool.set_partition_tokens(0)
            out.zero_()
        assert c.pool.timing_read()["workspace_bytes"] > before


@pytest.mark.gpu
def test_diff_decode_that_would_grow_inside_a_capture_is_refused():
    lens = [300]
    with Cache("bf16", 2, 64, lens) as c:
        q, params = queries(1, 4, 64), weights(64)
        tables, ln = c.tables.cuda(), torch.tensor(lens, dtype=torch.int32).cuda()
        out = torch.zeros(1, 2, 128, dtype=torch.bfloat16, device="cuda")
        x = torch.zeros(4, device="cuda")
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            x += 1
            with pytest.raises(pkv.PagedKVError) as e:
                pkv.paged_diff_decode_attention(c.pool, q, tables, ln, 0.125, params, out=out)
        assert e.value.status == 1 and "captured" in str(e.value)
        g.replay()  # the capture itself was not harmed
        torch.cuda.synchronize()
        assert (x == 1).all()


@pytest.mark.gpu
def test_diff_decode_refusals():
    with Cache("bf16", 2, 64, [20]) as c:
        q, params = queries(1, 4, 64), weights(64)
        tables, ln = c.tables.cuda(), torch.tensor([20], dtype=torch.int32).cuda()

        def call(q=q, tables=tables, ln=ln, scale=0.125, params=params, **kw):
            return pkv.paged_diff_decode_attention(c.pool, q, tables, ln, scale, params, **kw)

        for bad in (dict(q=q.float()), dict(q=q[..., :32]), dict(q=q.transpose(1, 2)), dict(ln=ln.long()),
                    dict(tables=tables[0]), dict(params=weights(128)), dict(out=q), dict(q=q.cpu())):
            with pytest.raises((ValueError, TypeError)):
                call(**bad)
        with pytest.raises(TypeError):
            call(params=None)
        lam = params.lambdas
        for bad in (dict(scale=float("nan")), dict(q=queries(1, 6, 64)), dict(q=queries(1, 5, 64)),
                    dict(params=pkv.DiffParams(lam, float("inf"))), dict(params=pkv.DiffParams(lam, 0.5, eps=0.0)),
                    dict(params=pkv.DiffParams(lam, 0.5, eps=float("nan")))):
            with pytest.raises(pkv.PagedKVError):
                call(**bad)
        with pytest.raises(ValueError):
            pkv.DiffParams(lam.half(), 0.5)
        with pytest.raises(ValueError):
            pkv.DiffParams(lam, 0.5, norm_weight=lam[0])
        assert call(q=q[:0], tables=tables[:0], ln=ln[:0]).shape == (0, 2, 128)
    for dtype, n_kv in ((pkv.INT4, 2), (pkv.BF16, 3)):
        with pkv.kv_pool_create(4, BS, n_kv, 64, dtype) as pool:
            if dtype == pkv.INT4:
                pool.set_int4_key_params(np.ones((2, 64)), np.zeros((2, 64)))
            with pytest.raises(pkv.PagedKVError) as e:
                pkv.paged_diff_decode_attention(pool, queries(1, 2 * n_kv, 64), tables, ln, 0.125, params)
            assert e.value.status == 5
            with pytest.raises(pkv.PagedKVError):
                pool.reserve_diff_workspace(1, 2 * n_kv, 2)


def test_diff_calls_with_null_pool_fail_cleanly():
    lib = pkv.load()
    prm = pkv._DiffParams(None, None, 0.5, 1e-5)
    assert lib.paged_diff_decode_attention(None, None, 4, None, 1, None, 1, 1.0, ctypes.byref(prm), None, None) == 1
    assert lib.paged_diff_reserve_workspace(None, 1, 4, 1) == 1


def test_diff_params_matches_the_header(tmp_path):
    import os
    import shutil
    import subprocess

    if shutil.which("gcc") is None:
        pytest.skip("gcc not found")
    inc = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include")
    fields = [f for f, _ in pkv._DiffParams._fields_]
    prints = "".join(f'printf("%zu ", offsetof(pkv_diff_params, {f}));' for f in fields)
    src, exe = tmp_path / "p.c", tmp_path / "p"
    src.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "pagedkv.h"\nint main(void) {' + prints
                   + 'printf("%zu", sizeof(pkv_diff_params)); return 0; }\n')
    subprocess.run(["gcc", "-I", inc, str(src), "-o", str(exe)], check=True)
    got = [int(x) for x in subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split()]
    assert got == [getattr(pkv._DiffParams, f).offset for f in fields] + [ctypes.sizeof(pkv._DiffParams)]
