"""Beam search's selection against 64-bit arithmetic: tokens and beams exactly, scores to their rounding.

Scores: v = score + x - lse is a double but for what lse is off by, and rounded once to 32 bits (2^-24 |v|).  lse
is the logarithm of a sum of 32-bit exponentials: each within 2^-21 of itself by the hardware's exponential, and
within |x - m| 2^-23 by its argument's two roundings, which in the mean over the sum is below 2^4 2^-23 (a row of
2^18 terms has none that counts further below its maximum); a thread adds at most 2^5 of them one after the other
in 32 bits, 2^-19 in the worst case.  2^-18 bounds the three together.
"""
import math

import pytest
import torch

import gqa_decode_attention_paged_gb300 as pkv

LSE = 2.0 ** -18


@pytest.fixture(scope="module")
def pool():
    with pkv.kv_pool_create(2, 16, 1, 64, pkv.BF16) as p:
        yield p


def expected(logits, scores, k):
    B, beams, V = logits.shape
    v = torch.log_softmax(logits.double().cpu(), -1) + scores.double().cpu()[..., None]
    v = torch.where(v.isnan(), torch.full_like(v, -math.inf), v).view(B, -1)
    if v.shape[1] < k:
        v = torch.cat((v, torch.full((B, k - v.shape[1]), -math.inf, dtype=torch.float64)), 1)
    best, at = v.sort(dim=-1, descending=True, stable=True)
    best, at = best[:, :k], at[:, :k]
    none = best == -math.inf
    return torch.where(none, -1, at % V), torch.where(none, -1, at // V), best


def check(pool, logits, scores, k, errors=0):
    got = pkv.paged_beam_select(pool, logits, scores, k)
    torch.cuda.synchronize()
    assert pool.get_error(clear=True) == errors
    tokens, parents, best = expected(logits, scores, k)
    assert [x.dtype for x in got] == [torch.int32, torch.int32, torch.float32]
    assert torch.equal(got[0].cpu().long(), tokens) and torch.equal(got[1].cpu().long(), parents)
    g = got[2].double().cpu()
    live = best > -math.inf
    assert torch.equal(g == -math.inf, ~live)
    err = (g - best).abs()[live]
    assert (err <= LSE + 2.0 ** -24 * best.abs()[live]).all(), float(err.max())
    return got


def draw(B, beams, V, dtype, seed=0, spread=3.0):
    g = torch.Generator().manual_seed(seed)
    x = (spread * torch.randn(B, beams, V, generator=g)).to(dtype).cuda()
    return x, (-10 * torch.rand(B, beams, generator=g)).cuda()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("B,beams,V,k", [(1, 1, 1, 1), (1, 1, 7, 4), (2, 3, 5, 15), (3, 4, 300, 8), (1, 4, 32000, 8), (5, 2, 8191, 4),
                                         (2, 5, 8193, 10), (4, 4, 16385, 5), (2, 16, 50257, 32), (1, 64, 4099, 64), (70, 5, 1001, 7),
                                         (1, 2, 262147, 17), (40, 10, 20000, 20), (300, 1, 129, 2)])
def test_selection_matches_64_bit_arithmetic(pool, dtype, B, beams, V, k):
    check(pool, *draw(B, beams, V, dtype, seed=V), k)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("kind", ["flat", "zeros", "rising", "falling", "two", "blocks", "tail"])
@pytest.mark.parametrize("V,k", [(40000, 3), (70001, 40), (513, 64)])
def test_equal_logits_and_orders_that_are_worst_for_a_scan(pool, dtype, kind, V, k):
    """Ties go to the lowest beam and token, whatever part of the row they are in; +0 and -0 are equal."""
    i = torch.arange(V)
    x = {"flat": torch.full((V,), 1.5), "zeros": torch.where(i % 2 == 0, -0.0, 0.0), "rising": i / V * 30, "falling": -(i / V) * 30,
         "two": torch.where(i % 1000 == 999, 4.0, 0.0), "blocks": (i // 700).float() / 8,
         "tail": torch.where(i >= V - 100, 5.0 + i / V, -1.0)}[kind]
    x = x.to(dtype).expand(2, 3, V).contiguous().cuda()
    scores = torch.tensor([[0.0, -1.0, 0.0], [-2.0, -2.0, -2.0]], device="cuda")
    check(pool, x, scores, k)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_forbidden_tokens_and_dead_beams(pool, dtype):
    x, scores = draw(6, 4, 20011, dtype, seed=1)
    x[0, :, ::3] = -math.inf
    x[1, 2] = -math.inf              # a beam without any token
    x[2] = -math.inf                 # a search without any
    x[3, :, 5:] = -math.inf          # 20 candidates for 30 places
    x[4, 1:, :] = math.nan           # ended beams: their logits may be anything
    x[4, 2, 0] = math.inf
    scores[4, 1:] = -math.inf
    scores[5, 0] = -math.inf
    x[0, 0, 7] = torch.finfo(dtype).min  # a mask of the type's lowest value is a value
    x[3, 0, 0] = torch.finfo(dtype).min
    check(pool, x, scores, 30)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("at", [0, 9000, 40010])
def test_beams_without_a_log_softmax_have_no_continuations_and_are_reported(pool, dtype, at):
    x, scores = draw(4, 3, 40011, dtype, seed=2)
    x[0, 1, at] = math.nan
    x[1, 0, at] = math.inf
    scores[2, 2] = math.nan
    scores[3, 1] = math.inf
    want = scores.clone()
    want[0, 1] = want[1, 0] = want[2, 2] = want[3, 1] = -math.inf
    got = pkv.paged_beam_select(pool, x, scores, 12)
    torch.cuda.synchronize()
    assert pool.get_error(clear=True) == pkv.DEVERR_NAN
    tokens, parents, best = expected(x, want, 12)
    assert torch.equal(got[0].cpu().long(), tokens) and torch.equal(got[1].cpu().long(), parents)
    assert (got[2].double().cpu() - best).abs().max() < 1e-4


@pytest.mark.gpu
def test_beams_that_differ_in_the_last_place(pool):
    """Two beams with the same logits, one score one step of 32 bits above the other, where score + logit is far larger."""
    g = torch.Generator().manual_seed(3)
    row = (3 * torch.randn(30000, generator=g)).cuda()
    x = row.expand(2, 2, 30000).contiguous()
    low = torch.tensor(-0.001)
    scores = torch.stack((torch.stack((low, torch.nextafter(low, torch.tensor(0.0)))), torch.stack((low, low)))).cuda()
    got = check(pool, x, scores, 20)
    assert got[1][0].tolist() == [1, 0] * 10 and got[1][1].tolist() == [0, 1] * 10


@pytest.mark.gpu
@pytest.mark.parametrize("scale", [1e-30, 1e3, 1e37])
def test_tiny_and_huge_logits(pool, scale):
    g = torch.Generator().manual_seed(4)
    x = (scale * torch.randn(2, 3, 30000, generator=g)).cuda()
    scores = torch.tensor([[0.0, -1e-3, -2e-3], [0.0, -1.0, -5.0]], device="cuda")
    if scale > 1e30:  # all but the greatest logit of a row are forbidden in effect; v of the rest is about -1e37
        got = pkv.paged_beam_select(pool, x, scores, 3)
        torch.cuda.synchronize()
        assert pool.get_error(clear=True) == 0
        assert got[1].tolist() == [[0, 1, 2]] * 2
        assert torch.equal(got[0].cpu().long(), x.cpu().argmax(-1))
        assert torch.equal(got[2], scores)
    elif scale < 1e-20:  # v is the same for all of a row's tokens to 64 bits, but their order is not
        got = pkv.paged_beam_select(pool, x, scores, 64)
        torch.cuda.synchronize()
        assert got[1].unique().tolist() == [0]
        assert torch.equal(got[0].cpu().long(), x[:, 0].cpu().sort(dim=-1, descending=True, stable=True).indices[:, :64])
    else:
        check(pool, x, scores, 5)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("lead,tail", [(0, 5), (1, 0), (3, 2), (7, 64)])
def test_rows_that_are_slices(pool, dtype, lead, tail):
    """Rows at any distance and alignment: what lies between them is not looked at."""
    wide, scores = draw(3, 4, lead + 12345 + tail, dtype, seed=5)
    wide[..., :lead] = math.nan
    wide[..., lead + 12345:] = 1e4
    check(pool, wide[..., lead:lead + 12345], scores, 9)
    check(pool, wide[:, :1, lead:lead + 12345], scores[:, :1].contiguous(), 9)
    check(pool, wide[:1, 1:2, lead:lead + 12345], scores[:1, 1:2].contiguous(), 9)


@pytest.mark.gpu
def test_on_another_stream_captured_and_again():
    x, scores = draw(9, 4, 33333, torch.bfloat16, seed=6)
    with pkv.kv_pool_create(2, 16, 1, 64, pkv.BF16) as pool:
        pool.reserve_beam_workspace(9, 4, 33333, 8)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = pkv.paged_beam_select(pool, x, scores, 8)
        for seed in (7, 8, 9):
            y, sc = draw(9, 4, 33333, torch.bfloat16, seed=seed)
            x.copy_(y)
            scores.copy_(sc)
            graph.replay()
            torch.cuda.synchronize()
            tokens, parents, _ = expected(x, scores, 8)
            assert torch.equal(got[0].cpu().long(), tokens) and torch.equal(got[1].cpu().long(), parents)
        s = torch.cuda.Stream()
        torch.cuda.synchronize()
        other = pkv.paged_beam_select(pool, x, scores, 8, stream=s)
        s.synchronize()
        for a, b in zip(got, other):
            assert torch.equal(a, b)
        bytes_now = pool.timing_read()["workspace_bytes"]
        for n in range(1, 10):  # fewer searches need no more
            pkv.paged_beam_select(pool, x[:n], scores[:n], 8)
        assert pool.timing_read()["workspace_bytes"] == bytes_now
    with pkv.kv_pool_create(2, 16, 1, 64, pkv.BF16) as fresh:
        graph = torch.cuda.CUDAGraph()
        with pytest.raises(pkv.PagedKVError):
            with torch.cuda.graph(graph):
                pkv.paged_beam_select(fresh, x, scores, 8)


@pytest.mark.gpu
def test_refusals(pool):
    x, scores = draw(2, 3, 100, torch.float32)
    call = lambda x=x, s=scores, k=4: pkv.paged_beam_select(pool, x, s, k)  # noqa: E731
    for bad in (dict(k=0), dict(k=65), dict(x=torch.zeros(2, 65, 10, device="cuda"), s=torch.zeros(2, 65, device="cuda")),
                dict(x=x[..., :0])):
        with pytest.raises(pkv.PagedKVError):
            call(**bad)
    for bad in (dict(x=x.half()), dict(x=x.cpu()), dict(s=scores.double()), dict(s=scores[:, :2]), dict(x=x.transpose(1, 2)),
                dict(x=x[..., ::2]), dict(x=x.transpose(0, 1))):
        with pytest.raises(ValueError):
            call(**bad)
    with pytest.raises(TypeError):
        call(x=x[0])
    none = call(x=x[:0], s=scores[:0])
    assert all(t.shape == (0, 4) for t in none)
    assert pool.get_error() == 0
