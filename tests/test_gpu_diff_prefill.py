"""Differential attention of chunks of new tokens against the plain 64-bit
form (diff_ref.py), and a layer's calls run together."""
import ctypes

import numpy as np
import pytest
import torch

import gqa_decode_attention_paged_gb300 as pkv
from diff_ref import BS, Cache, check, plain, weights


def queries(rows, n_q, d, seed=0):
    g = torch.Generator().manual_seed(177 + seed)
    return torch.randn(rows, n_q, d, generator=g).to(torch.bfloat16).cuda()


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32).cuda()


PAD = 160  # sequences without rows behind the others: so many tiles may follow that the call runs whole


def prefill(c, q, chunks, params, lens=None, tables=None, indptr=None, pad=0, **kw):
    indptr = np.concatenate([[0], np.cumsum(chunks)]) if indptr is None else indptr
    if pad:
        indptr = np.concatenate([indptr, np.full(pad, indptr[-1])])
        lens = list(c.lens if lens is None else lens) + [0, 5] * (pad // 2)
        tables = c.tables if tables is None else tables
        tables = torch.cat((tables, torch.full((pad, tables.shape[1]), -1, dtype=torch.int32)))
    return pkv.paged_diff_prefill_attention(c.pool, q, i32(indptr), (c.tables if tables is None else tables).cuda(),
                                            i32(c.lens if lens is None else lens), 1 / np.sqrt(c.d), params, **kw)


def ptr(chunks):
    return np.concatenate([[0], np.cumsum(chunks)])


CASES = [  # n_kv, G, d, lens, chunks
    (2, 1, 64, [1], [1]),
    (2, 4, 128, [128], [32]),
    (2, 4, 128, [1, 40, 300, 1000], [1, 17, 300, 64]),
    (4, 8, 128, [200, 33, 700], [200, 0, 5]),
    (2, 2, 64, [90, 5, 257, 16], [90, 5, 100, 16]),
    (6, 1, 64, [100, 31, 0, 129], [60, 31, 0, 128]),
    (4, 2, 128, [64, 512, 3, 130], [33, 512, 2, 1]),
    (2, 8, 64, [515, 127], [515, 127]),
]


@pytest.mark.gpu
@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c[:3])) + f"-{len(c[3])}")
@pytest.mark.parametrize("pad", [0, PAD])
def test_diff_prefill_matches_the_64_bit_form(kv, case, pad):
    n_kv, G, d, lens, chunks = case
    with Cache(kv, n_kv, d, lens, seed=G) as c:
        for b in range(len(lens)):
            c.poison(b)
        c.upload()
        rows = sum(chunks)
        q, params = queries(rows, n_kv * G, d, G), weights(d, G, norm=G != 2)
        out = torch.full((rows, n_kv * G // 2, 2 * d), 5.0, dtype=torch.bfloat16, device="cuda")
        got = prefill(c, q, chunks, params, out=out, pad=pad)
        torch.cuda.synchronize()
        assert got is out and c.pool.get_error() == 0
        check(got, *plain(c, q, ptr(chunks), lens, 1 / np.sqrt(d), params))
        assert torch.equal(got, prefill(c, q, chunks, params, pad=pad))  # the same bits again


@pytest.mark.gpu
@pytest.mark.parametrize("kv,n_kv,G,d,lens,chunks", [
    ("bf16", 2, 4, 128, [2300], [2300]),                            # many steps, more tiles than one wave's worth of a pair
    ("fp8", 8, 4, 64, list(range(3, 203, 5)), list(range(1, 201, 5))),   # more than 32 sequences, all odd
    ("bf16", 16, 2, 64, [150] * 70, [7] * 70),
    ("bf16", 64, 1, 128, [260, 40], [130, 40]),
    ("fp8", 2, 8, 128, [1900, 10], [64, 10]),
    ("bf16", 2, 4, 128, [20000], [9]),                              # a few drafted tokens on a long cache
    ("fp8", 4, 2, 64, [9000, 17, 3], [3, 17, 1]),
    ("bf16", 4, 1, 64, [1030], [1030]),
    ("fp8", 16, 4, 128, [129] * 24, [100] * 24),                    # whole: single tiles of their pairs
    ("bf16", 64, 1, 64, [600, 520, 700, 513, 1, 640], [600, 520, 700, 513, 1, 640]),  # windows of four sequences
])
def test_diff_prefill_shapes(kv, n_kv, G, d, lens, chunks):
    with Cache(kv, n_kv, d, lens, seed=8) as c:
        q, params = queries(sum(chunks), n_kv * G, d), weights(d, lambda_init=0.3)
        got = prefill(c, q, chunks, params)
        torch.cuda.synchronize()
        assert c.pool.get_error() == 0
        check(got, *plain(c, q, ptr(chunks), lens, 1 / np.sqrt(d), params))


@pytest.mark.gpu
@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("lam", ["zero", "negative", "large", "tiny"])
@pytest.mark.parametrize("pad", [0, PAD])
def test_diff_prefill_lambdas(kv, lam, pad):
    """lambda 0, below 0, far above 1 (the second map's factor is then the larger) and far below 1."""
    d, lens, chunks = 64, [70, 300], [70, 33]
    a = torch.zeros(4, d, device="cuda")
    init = {"zero": 0.0, "negative": -0.75, "large": 0.0, "tiny": 1e-6}[lam]
    if lam == "large":
        a[0, 0] = a[1, 0] = 2.0  # e^4 - 1
    with Cache(kv, 2, d, lens, seed=1) as c:
        q, params = queries(sum(chunks), 8, d), pkv.DiffParams(a, init)
        got = prefill(c, q, chunks, params, pad=pad)
        torch.cuda.synchronize()
        check(got, *plain(c, q, ptr(chunks), lens, 1 / np.sqrt(d), params))


@pytest.mark.gpu
@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("scale", [-0.1, 0.0])
def test_diff_prefill_and_decode_scales_at_or_below_zero(kv, scale):
    d, lens, chunks = 64, [140, 20], [40, 20]
    with Cache(kv, 2, d, lens, seed=11) as c:
        q, params = queries(sum(chunks), 4, d), weights(d)
        got = pkv.paged_diff_prefill_attention(c.pool, q, i32(ptr(chunks)), c.tables.cuda(), i32(lens), scale, params)
        check(got, *plain(c, q, ptr(chunks), lens, scale, params))
        got = pkv.paged_diff_decode_attention(c.pool, q[:2].contiguous(), c.tables.cuda(), i32(lens), scale, params)
        check(got, *plain(c, q[:2], [0, 1, 2], lens, scale, params))


@pytest.mark.gpu
@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("pad", [0, PAD])
def test_diff_prefill_one_map_sharp_the_other_flat(kv, pad):
    """The two maps' sums differ by the whole length: one map's scores are 0 everywhere (its queries are
    0), the other's are dominated by single keys; both ways round."""
    d, lens, chunks = 64, [1500], [200]
    with Cache(kv, 2, d, lens, seed=12, sharp=3.0) as c:
        for flat in (0, 1):
            q = 3 * queries(200, 4, d)
            q[:, flat::2] = 0
            params = weights(d)
            got = prefill(c, q, chunks, params, pad=pad)
            torch.cuda.synchronize()
            check(got, *plain(c, q, ptr(chunks), lens, 1 / np.sqrt(d), params), norm2=False)


@pytest.mark.gpu
@pytest.mark.parametrize("pad", [0, PAD])
def test_diff_prefill_scores_of_large_magnitude(pad):
    """Scores of +-32768: a map's weights lie on a few equal keys, or on all of them, far below zero.

    The scores are exact, but four sums take place at their size in units of log2 (s - m, twice; the factor's
    exponent; m with the part of log2(l) that is not passed on): each is off by 2^-24 of it at most, and so is
    the exponent.  The bound's 2^-12 is for small scores; this is added to it."""
    d, lens, chunks = 64, [4000, 90], [20, 60]
    with Cache("bf16", 2, d, lens, seed=14) as c:
        c.k[..., 0] = -1
        for j in (3, 60, 200):
            c.k[int(c.tables[0, j]), :, j % BS, 0] = 1
        c.k64 = c.k.double()
        c.upload()
        q, params = torch.zeros(80, 8, d, dtype=torch.bfloat16, device="cuda"), weights(d)
        for h in range(8):
            q[:, h, 0] = 2.0 ** 18 * (-1 if h % 3 else 1)
        got = prefill(c, q, chunks, params, pad=pad)
        torch.cuda.synchronize()
        ref, bound = plain(c, q, ptr(chunks), lens, 1 / np.sqrt(d), params)
        exact = 2.0 ** -8 + 2.0 ** -12
        extra = 4 * 2.0 ** -24 * 32768  # (log2 units x ln 2)
        check(got, ref, bound * (exact + extra) / exact, norm2=False)


@pytest.mark.gpu
@pytest.mark.parametrize("pad", [0, PAD])
def test_diff_prefill_bad_blocks_are_masked_and_flagged(pad):
    lens, chunks = [300, 64, 200], [150, 20, 200]
    with Cache("bf16", 2, 64, lens, seed=2) as c:
        tables = c.tables.clone()
        tables[0, 2], tables[2, 0] = c.blocks, -5
        tables[1, :4] = 10 ** 6
        q, params = queries(sum(chunks), 4, 64), weights(64)
        got = prefill(c, q, chunks, params, tables=tables, pad=pad)
        torch.cuda.synchronize()
        assert c.pool.get_error(clear=True) == pkv.DEVERR_BLOCK_RANGE
        skip = [(0, 2), (2, 0)] + [(1, j) for j in range(4)]
        check(got, *plain(c, q, ptr(chunks), lens, 1 / np.sqrt(64), params, skip=skip))
        assert (got[150:170] == 0).all()  # sequence 1 sees nothing
        assert (got[170:186] == 0).all()  # the first 16 tokens of sequence 2 neither


@pytest.mark.gpu
def test_diff_prefill_rows_of_no_sequence_stay_as_they_were():
    lens, chunks = [50, 90], [20, 90]
    with Cache("bf16", 2, 64, lens, seed=3) as c:
        q, params = queries(130, 4, 64), weights(64)
        want = prefill(c, q[:110].contiguous(), chunks, params)
        out = torch.full((130, 2, 128), 3.0, dtype=torch.bfloat16, device="cuda")
        prefill(c, q, chunks, params, out=out)
        torch.cuda.synchronize()
        assert torch.equal(out[:110], want) and (out[110:] == 3).all()
        # sequences whose rows are not the caller's are skipped, the others are as before
        for bad in ([0, 20, 131], [-1, 20, 110], [0, 20, 10]):
            out.fill_(3.0)
            prefill(c, q, chunks, params, indptr=bad, out=out)
            torch.cuda.synchronize()
            assert c.pool.get_error(clear=True) == pkv.DEVERR_CTX_RANGE
            kept = slice(0, 20) if bad[0] == 0 else slice(20, 110)
            assert torch.equal(out[kept], want[kept])
            rest = torch.ones(130, dtype=torch.bool, device="cuda")
            rest[kept] = False
            assert (out[rest] == 3).all()


@pytest.mark.gpu
def test_diff_prefill_lengths_out_of_range():
    with Cache("bf16", 2, 64, [60, 60], table_extra=0, seed=4) as c:  # tables of 4 blocks
        q, params = queries(30 + 40, 4, 64), weights(64)
        # a length past the table is clamped to it, a chunk longer than its cache lengthens it
        got = prefill(c, q, [30, 40], params, lens=[1000, 12])
        torch.cuda.synchronize()
        assert c.pool.get_error(clear=True) == pkv.DEVERR_CTX_RANGE
        check(got, *plain(c, q, [0, 30, 70], [64, 40], 1 / np.sqrt(64), params))
        for pad in (0, PAD):
            out = torch.full((70, 2, 128), 3.0, dtype=torch.bfloat16, device="cuda")
            prefill(c, q, [65, 5], params, lens=[65, 60], out=out, pad=pad)  # 65 tokens in 4 blocks: skipped
            torch.cuda.synchronize()
            assert c.pool.get_error(clear=True) == pkv.DEVERR_CTX_RANGE
            assert (out[:65] == 3).all() and (out[65:] != 3).any()


@pytest.mark.gpu
def test_diff_prefill_on_a_side_stream_and_in_a_graph():
    lens, chunks = [500, 40], [130, 40]
    with Cache("bf16", 4, 128, lens, seed=6) as c:
        q, params = queries(170, 8, 128), weights(128)
        want = prefill(c, q, chunks, params)
        i32_kept = (i32(ptr(chunks)), c.tables.cuda(), i32(lens))
        args = (*i32_kept, 1 / np.sqrt(128), params)
        static = torch.zeros_like(q)
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            out = pkv.paged_diff_prefill_attention(c.pool, static, *args)
        with torch.cuda.stream(side):
            static.copy_(q)
            for _ in range(2):
                out.zero_()
                g.replay()
        side.synchronize()
        assert torch.equal(out, want)
    # a pool whose workspace would have to grow inside the capture: the call runs whole
    with Cache("bf16", 4, 128, lens, seed=6) as c:
        before = c.pool.timing_read()["workspace_bytes"]
        g = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(g, stream=side):
            out = pkv.paged_diff_prefill_attention(c.pool, static, *i32_kept, 1 / np.sqrt(128), params)
        assert c.pool.timing_read()["workspace_bytes"] == before
        g.replay()
        torch.cuda.synchronize()
        check(out, *plain(c, q, ptr(chunks), lens, 1 / np.sqrt(128), params))
        c.pool.reserve_diff_workspace(2, 8, c.W)
        assert c.pool.timing_read()["workspace_bytes"] > before
        got = pkv.paged_diff_prefill_attention(c.pool, static, *i32_kept, 1 / np.sqrt(128), params)
        assert torch.equal(got, want)


@pytest.mark.gpu
def test_diff_prefill_refusals():
    with Cache("bf16", 2, 64, [20]) as c:
        q, params = queries(4, 4, 64), weights(64)
        for bad in (dict(q=q.float()), dict(q=q[:, :, :32]), dict(params=weights(128)), dict(lens=[20, 20]),
                    dict(indptr=[0, 2, 4]), dict(out=q)):
            with pytest.raises((ValueError, TypeError)):
                prefill(c, **{**dict(q=q, chunks=[4], params=params), **bad})
        for bad in (dict(q=queries(4, 6, 64)), dict(params=pkv.DiffParams(params.lambdas, float("nan"))),
                    dict(params=pkv.DiffParams(params.lambdas, 0.5, eps=-1.0))):
            with pytest.raises(pkv.PagedKVError):
                prefill(c, **{**dict(q=q, chunks=[4], params=params), **bad})
        assert prefill(c, q[:0], [0], params).shape == (0, 2, 128)
    for dtype, n_kv in ((pkv.INT4, 2), (pkv.BF16, 1)):
        with pkv.kv_pool_create(4, BS, n_kv, 64, dtype) as pool:
            if dtype == pkv.INT4:
                pool.set_int4_key_params(np.ones((2, 64)), np.zeros((2, 64)))
            with pytest.raises(pkv.PagedKVError) as e:
                pkv.paged_diff_prefill_attention(pool, queries(4, 2 * n_kv, 64), i32([0, 4]), i32([[0, 1]]), i32([20]),
                                                 0.125, params)
            assert e.value.status == 5


def test_diff_prefill_with_null_pool_fails_cleanly():
    prm = pkv._DiffParams(None, None, 0.5, 1e-5)
    assert pkv.load().paged_diff_prefill_attention(None, None, 1, 4, None, None, 1, None, 1, 1.0, ctypes.byref(prm), None,
                                                   None) == 1


@pytest.mark.gpu
@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_a_layer_from_prompt_to_decode(kv):
    """A layer as it is served: prompts with image positions are rotated and written in two chunks, each
    attended with the differential prefill, then two decode steps; every output against the 64-bit
    form over what the pool holds, and the cache read back equal to it."""
    n_kv, G, d, prompts = 4, 2, 64, [37, 130, 5]
    B, n_q, steps = len(prompts), n_kv * G, 2
    lens_end = [p + steps for p in prompts]
    g = torch.Generator().manual_seed(5)
    rope = pkv.Rope(10000.0 ** (-np.arange(d // 2) / (d // 2)), np.arange(d // 2) % 3)
    params = weights(d)
    with Cache(kv, n_kv, d, lens_end, seed=7) as c:
        c.pool.k_view().zero_()
        c.pool.v_view().zero_()
        tables = c.tables.cuda()

        def feed(first, count):
            """Tokens first[b] .. first[b] + count[b] - 1 of every sequence; (outputs, queries)."""
            pos = np.concatenate([np.arange(f, f + n) for f, n in zip(first, count)])
            own = np.repeat(np.arange(B), count)
            slots = c.tables.numpy()[own, pos // BS].astype(np.int64) * BS + pos % BS
            q, k, v = (torch.randn(len(pos), h, d, generator=g).to(torch.bfloat16).cuda() for h in (n_q, n_kv, n_kv))
            axes = i32(np.stack((pos // 16, pos // 4 % 4, pos % 4)))
            turned = pkv.paged_rope_append(c.pool, rope, q, k, v, axes, torch.from_numpy(slots).cuda())
            now = [f + n for f, n in zip(first, count)]
            if max(count) == 1:
                out = pkv.paged_diff_decode_attention(c.pool, turned, tables, i32(now), 1 / np.sqrt(d), params)
            else:
                out = pkv.paged_diff_prefill_attention(c.pool, turned, i32(ptr(count)), tables, i32(now), 1 / np.sqrt(d),
                                                       params)
            torch.cuda.synchronize()
            assert c.pool.get_error() == 0
            # what the pool holds now, in 64 bits
            rk, rv = c.pool.k_view().view(c.k.dtype).cpu(), c.pool.v_view().view(c.v.dtype).cpu()
            lay = [1.0, 1.0] if kv == "bf16" else [torch.from_numpy(s).double().view(1, n_kv, 1, 1) for s in scales]
            c.k64, c.v64 = rk.double() * lay[0], rv.double() * lay[1]
            check(out, *plain(c, turned, ptr(count), now, 1 / np.sqrt(d), params))

        if kv == "fp8":
            scales = [np.full(n_kv, 6 / 448, np.float32), np.full(n_kv, 5.5 / 448, np.float32)]
            c.pool.set_fp8_scales(*scales)
        half = [p // 2 + 1 for p in prompts]
        feed([0] * B, half)
        feed(half, [p - h for p, h in zip(prompts, half)])
        for s in range(steps):
            feed([p + s for p in prompts], [1] * B)
        indptr = ptr(lens_end)
        k, v = pkv.paged_kv_gather(c.pool, i32(indptr), tables, n_rows=int(indptr[-1]))
        for got, want in ((k, c.k64), (v, c.v64)):
            rows = torch.cat([want[c.tables[b, :(n + BS - 1) // BS].long()].transpose(1, 2).reshape(-1, n_kv, d)[:n]
                              for b, n in enumerate(lens_end)])
            assert torch.equal(got.cpu(), rows.float().to(torch.bfloat16))
