"""Attention of trees of drafted tokens over the paged cache, against 64-bit arithmetic."""
import math
import random

import numpy as np
import pytest
import torch

import gqa_decode_attention_paged_gb300 as pkv
from tree_ref import BS, Cache, check, pack, parents_of, plain, random_masks, tree_bits


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32).cuda()


def ptr(nodes, first=0):
    return np.cumsum([first] + list(nodes))


def queries(rows, n_q, d, seed=0):
    g = torch.Generator().manual_seed(50 + seed)
    return torch.randn(rows, n_q, d, generator=g).to(torch.bfloat16).cuda()


def words_of(nodes):
    return max(1, (max(list(nodes) + [0]) + 63) // 64)


def attend(c, q, nodes, bits, first=0, words=None, **kw):
    return pkv.paged_tree_attention(c.pool, q, i32(ptr(nodes, first)), pack(bits, words or words_of(nodes)).cuda(),
                                    c.tables.cuda(), i32(c.lens), 1 / math.sqrt(c.d), **kw)


def run(c, nodes, G, seed=0, bits=None, words=None):
    bits = random_masks(nodes, seed) if bits is None else bits
    q = queries(sum(nodes), c.n_kv * G, c.d, seed)
    got = attend(c, q, nodes, bits, words=words)
    torch.cuda.synchronize()
    check(got, *plain(c, q, ptr(nodes), bits, c.lens, 1 / math.sqrt(c.d)))
    assert c.pool.get_error() == 0
    return got


SHAPES = [
    # cache lengths, nodes: blocks that end inside a step, contexts of none, one node, none
    ([300], [8]),
    ([17, 1, 16, 64, 129], [1, 1, 16, 3, 5]),
    ([40, 40, 0, 128, 127, 500], [40, 7, 0, 33, 32, 0]),
    ([700, 130, 257, 1100], [64, 65, 128, 63]),
    ([2000, 31], [200, 31]),
]


@pytest.mark.gpu
@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("G", [1, 2, 4, 8])
@pytest.mark.parametrize("shape", range(len(SHAPES)))
def test_trees_match_64_bit_arithmetic(kv, d, G, shape):
    lens, nodes = SHAPES[shape]
    with Cache(kv, 2, d, lens, seed=shape) as c:
        run(c, nodes, G, seed=shape)


@pytest.mark.gpu
@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("n_kv,batch,C,T", [(1, 1, 9000, 13), (8, 3, 5000, 20), (4, 40, 600, 9), (1, 300, 33, 2), (3, 2, 3000, 90)])
def test_splits_of_long_and_many_sequences(kv, n_kv, batch, C, T):
    rng = random.Random(C)
    lens = [max(T, C - rng.randrange(C // 2)) for _ in range(batch)]
    nodes = [rng.randint(1, T) for _ in range(batch)]
    with Cache(kv, n_kv, 128 if n_kv < 4 else 64, lens, seed=3) as c:
        run(c, nodes, 4, seed=4)


@pytest.mark.gpu
@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_a_thousand_nodes_and_masks_of_sixteen_words(kv):
    with Cache(kv, 1, 64, [1500, 70], seed=5) as c:
        run(c, [1024, 70], 2, seed=5, words=16)


@pytest.mark.gpu
@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_masks_need_not_be_trees_and_may_leave_rows_empty(kv):
    """Any bits: a node that does not see itself, one that sees later nodes, none at all without a context (a row of
    zeros); bits behind the last node are not looked at."""
    nodes, lens = [9, 20, 5], [9, 200, 5]
    g = random.Random(7)
    bits = [g.getrandbits(64) for _ in range(sum(nodes))]
    bits[0] = 0
    bits[3] = 1 << 60  # behind the nodes: nothing
    bits[30] = 0
    bits[33] = (1 << 64) - 1
    with Cache(kv, 2, 128, lens, seed=6) as c:
        got = run(c, nodes, 2, bits=bits)
        assert (got[0] == 0).all() and (got[3] == 0).all() and (got[30] == 0).all()
        assert (got[33] != 0).any()


@pytest.mark.gpu
@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_rows_behind_the_end_are_never_used(kv):
    lens, nodes = [5, 130, 500, 1030], [5, 3, 40, 66]
    with Cache(kv, 2, 128, lens, seed=8) as c:
        for b in range(len(lens)):
            c.poison(b)
        c.upload()
        run(c, nodes, 4, seed=8)


@pytest.mark.gpu
@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("sharp", [6.0, 40.0])
def test_sharp_scores(kv, sharp):
    """Scores of tens: the running maximum rises step by step.  (Beyond 2^5 32-bit scores are off by more than the
    bound's 2^-12: 2^-24 * |s| * log2(e) each way for the product's and the reference's rounding, added here.)"""
    lens, nodes = [900, 257], [30, 12]
    with Cache(kv, 2, 64, lens, seed=9, sharp=sharp) as c:
        bits = random_masks(nodes, 9)
        q = queries(sum(nodes), 8, 64, 9)
        got = attend(c, q, nodes, bits)
        torch.cuda.synchronize()
        ref, bound = plain(c, q, ptr(nodes), bits, c.lens, 1 / 8)
        most = float((q.double().cpu().abs().amax() * c.k64.abs().amax() * 64 / 8))
        extra = 4 * 2.0 ** -24 * most * 2  # of |V|'s largest, relative weights
        check(got, ref, bound + extra * float(c.v64.abs().amax()))


@pytest.mark.gpu
def test_keys_rising_along_the_sequence():
    """Every step's scores are above the last one's by more than any slack."""
    lens, nodes = [1300], [10]
    with Cache("bf16", 1, 64, lens, seed=10) as c:
        for pos in range(1300):
            c.k[int(c.tables[0, pos // BS]), 0, pos % BS] = pos / 16.0
        c.k64 = c.k.double()
        c.upload()
        q = torch.full((10, 4, 64), 1 / 64).to(torch.bfloat16).cuda()
        bits = random_masks(nodes, 10)
        got = attend(c, q, nodes, bits)
        torch.cuda.synchronize()
        check(got, *plain(c, q, ptr(nodes), bits, lens, 1 / 8))


@pytest.mark.gpu
@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_rows_of_no_sequence_and_of_skipped_ones_stay_as_they_were(kv):
    lens = [100, 40, 70, 20, 30]
    nodes = [6, 50, 3, 2, 4]  # the second has more nodes than its cache holds
    first = 3
    rows = first + sum(nodes) + 5
    with Cache(kv, 2, 64, lens, seed=11) as c:
        q = queries(rows, 4, 64)
        bits = [0] * first + random_masks(nodes, 11) + [0] * 5
        out = torch.full((rows, 4, 64), 7.0, dtype=torch.bfloat16, device="cuda")
        attend(c, q, nodes, bits, first=first, out=out)
        torch.cuda.synchronize()
        assert c.pool.get_error(clear=True) == pkv.DEVERR_CTX_RANGE
        at = ptr(nodes, first)
        ref, bound = plain(c, q, at, bits, lens, 1 / 8, only=(0, 2, 3, 4))
        keep = torch.zeros(rows, dtype=torch.bool)
        keep[:first] = keep[at[1]:at[2]] = keep[at[-1]:] = True
        assert (out[keep.cuda()] == 7).all()
        check(out[~keep.cuda()], ref[~keep], bound[~keep])


@pytest.mark.gpu
@pytest.mark.parametrize("what", ["backwards", "outside", "negative", "table", "words", "lens"])
def test_sequences_that_do_not_fit_are_skipped(what):
    lens, nodes = [100, 200, 90], [10, 70, 8]
    with Cache("bf16", 2, 64, lens, seed=12) as c:
        q = queries(88, 4, 64)
        bits = random_masks(nodes, 12)
        at, ln, words = ptr(nodes), list(lens), 2
        good = [0, 2]
        if what == "backwards":
            at[1], at[2], at[3] = 10, 4, 4
            good = [0]
        elif what == "outside":
            at[3] = 95
            good = [0, 1]
        elif what == "negative":
            at[0] = -3
            good = [1, 2]
        elif what == "table":
            ln[1] = c.W * BS + 1
        elif what == "words":
            words = 1
        else:
            ln[1] = -5
        out = torch.full((88, 4, 64), 7.0, dtype=torch.bfloat16, device="cuda")
        pkv.paged_tree_attention(c.pool, q, i32(at), pack(bits, words).cuda(), c.tables.cuda(), i32(ln), 1 / 8, out=out)
        torch.cuda.synchronize()
        assert c.pool.get_error(clear=True) == pkv.DEVERR_CTX_RANGE
        ref, bound = plain(c, q, at, bits, lens, 1 / 8, only=good)
        for b in good:
            lo, hi = int(at[b]), int(at[b + 1])
            check(out[lo:hi], ref[lo:hi], bound[lo:hi])


@pytest.mark.gpu
@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_blocks_outside_the_pool_count_as_masked(kv):
    lens, nodes = [300, 50, 40], [20, 5, 40]
    with Cache(kv, 2, 128, lens, seed=13) as c:
        q = queries(65, 8, 128)
        bits = random_masks(nodes, 13)
        kept = c.tables.clone()
        c.tables[0, 3], c.tables[0, 12], c.tables[1, 3] = -1, c.blocks, 2 ** 31 - 1
        c.tables[2, :3] = -7
        got = attend(c, q, nodes, bits)
        torch.cuda.synchronize()
        assert c.pool.get_error(clear=True) == pkv.DEVERR_BLOCK_RANGE
        c.tables = kept
        skip = [(0, 3), (0, 12), (1, 3), (2, 0), (2, 1), (2, 2)]
        check(got, *plain(c, q, ptr(nodes), bits, lens, 1 / math.sqrt(128), skip))
        assert (got[25:] == 0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_nan_reaches_the_rows_that_see_it(kv):
    """A NaN key of one drafted node: its descendants' rows of the KV head, and no others."""
    lens, nodes = [200, 90], [40, 10]
    with Cache(kv, 2, 64, lens, seed=14) as c:
        bits = random_masks(nodes, 14)
        q = queries(50, 4, 64)
        want = attend(c, q, nodes, bits)
        node = 3
        pos = 160 + node
        blk = int(c.tables[0, pos // BS])
        c.k.view(torch.uint8)[blk, 1, pos % BS] = torch.full((64,), math.nan).to(c.k.dtype).view(torch.uint8)
        c.upload()
        got = attend(c, q, nodes, bits)
        torch.cuda.synchronize()
        hit = torch.tensor([r < 40 and (bits[r] >> node) & 1 == 1 for r in range(50)])
        nan = torch.zeros(50, 4, 64, dtype=torch.bool)
        nan[hit, 2:] = True
        assert torch.equal(got.isnan().cpu(), nan)
        assert torch.equal(got[~nan.cuda()], want[~nan.cuda()])


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 30])
def test_keys_whose_scores_are_minus_infinity_weigh_nothing(T):
    lens, nodes = [300, 40, 700], [T, T, T]
    low = [list(range(128)) + [299 - T], range(40), range(600)]
    with Cache("bf16", 2, 64, lens, seed=15) as c:
        for b, keys in enumerate(low):
            for pos in keys:
                c.k[int(c.tables[b, pos // BS]), :, pos % BS, 0] = -math.inf
        c.k64 = c.k.double()
        c.upload()
        q = queries(3 * T, 8, 64)
        q[..., 0] = 1
        bits = random_masks(nodes, 15)
        got = attend(c, q, nodes, bits)
        torch.cuda.synchronize()
        check(got, *plain(c, q, ptr(nodes), bits, lens, 1 / 8))


@pytest.mark.gpu
def test_scale_of_zero_and_negative_scales():
    lens, nodes = [300, 20], [20, 20]
    with Cache("bf16", 2, 64, lens, seed=16) as c:
        q = queries(40, 4, 64)
        bits = random_masks(nodes, 16)
        for scale in (0.0, -0.3):
            got = pkv.paged_tree_attention(c.pool, q, i32(ptr(nodes)), pack(bits, 1).cuda(), c.tables.cuda(), i32(lens), scale)
            torch.cuda.synchronize()
            check(got, *plain(c, q, ptr(nodes), bits, lens, scale))


@pytest.mark.gpu
def test_a_chain_is_the_chunked_prefill():
    """A tree that is one chain sees what a causal chunk sees."""
    lens, nodes = [1000, 333], [50, 61]
    with Cache("bf16", 4, 128, lens, seed=17) as c:
        q = queries(111, 16, 128)
        bits = [(1 << (i + 1)) - 1 for t in nodes for i in range(t)]
        got = attend(c, q, nodes, bits)
        other = pkv.paged_prefill_attention(c.pool, q, i32(ptr(nodes)), c.tables.cuda(), i32(lens), 1 / math.sqrt(128))
        torch.cuda.synchronize()
        ref, bound = plain(c, q, ptr(nodes), bits, lens, 1 / math.sqrt(128))
        check(got, ref, bound)
        assert ((got.double() - other.double()).abs().cpu() <= 2 * bound).all()


@pytest.mark.gpu
@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_blocks_beyond_four_gib(kv):
    """Entries whose offsets pass 32 bits."""
    n_kv, d = 8, 128
    entry = 16 * d * (4 if kv == "bf16" else 2)
    blocks = (2 ** 32 + 2 ** 28) // (n_kv * entry)
    lens, nodes = [200], [12]
    with Cache(kv, n_kv, d, lens, seed=18) as c:
        big = pkv.kv_pool_create(blocks, BS, n_kv, d, c.pool.dtype)
        if kv == "fp8":
            ks, vs = ((x64[0, :, 0, 0] / x[0, :, 0, 0].double()).float().numpy() for x64, x in ((c.k64, c.k), (c.v64, c.v)))
            big.set_fp8_scales(ks, vs)
        for view, x in ((big.k_view(), c.k), (big.v_view(), c.v)):
            view[blocks - c.blocks:] = x.view(torch.uint8).cuda()
        small, c.pool = c.pool, big
        bits = random_masks(nodes, 18)
        q = queries(12, 16, d)
        got = pkv.paged_tree_attention(big, q, i32(ptr(nodes)), pack(bits, 1).cuda(),
                                       torch.where(c.tables >= 0, c.tables + blocks - c.blocks, -1).cuda(), i32(lens), 1 / math.sqrt(d))
        torch.cuda.synchronize()
        check(got, *plain(c, q, ptr(nodes), bits, lens, 1 / math.sqrt(d)))
        assert big.get_error() == 0
        big.close()
        c.pool = small


@pytest.mark.gpu
def test_on_another_stream_and_captured():
    lens, nodes = [700, 90, 3000], [20, 9, 33]
    with Cache("bf16", 2, 128, lens, seed=19) as c:
        bits = random_masks(nodes, 19)
        q = queries(62, 8, 128)
        ref = plain(c, q, ptr(nodes), bits, lens, 1 / math.sqrt(128))
        want = attend(c, q, nodes, bits)  # (grows the workspace)
        torch.cuda.synchronize()
        check(want, *ref)
        s = torch.cuda.Stream()
        args = (i32(ptr(nodes)), pack(bits, 1).cuda(), c.tables.cuda(), i32(lens), 1 / math.sqrt(128))
        torch.cuda.synchronize()
        for handle in (s, s.cuda_stream):
            got = pkv.paged_tree_attention(c.pool, q, *args, stream=handle)
            s.synchronize()
            assert torch.equal(got, want)
        out = torch.zeros_like(q)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            pkv.paged_tree_attention(c.pool, q, *args, out=out)
        for _ in range(3):
            out.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, want)
        # the same graph on other lengths: shorter trees at the ends of shorter caches
        args[3].copy_(i32([650, 90, 100]))
        graph.replay()
        torch.cuda.synchronize()
        c.lens = [650, 90, 100]
        check(out, *plain(c, q, ptr(nodes), bits, c.lens, 1 / math.sqrt(128)))


@pytest.mark.gpu
def test_results_do_not_change_from_call_to_call():
    lens, nodes = [4000, 900, 2500], [33, 64, 7]
    with Cache("fp8", 4, 128, lens, seed=20) as c:
        bits = random_masks(nodes, 20)
        q = queries(104, 16, 128)
        want = attend(c, q, nodes, bits)
        for _ in range(5):
            assert torch.equal(attend(c, q, nodes, bits), want)


@pytest.mark.gpu
def test_refusals():
    lens, nodes = [50], [5]
    with Cache("bf16", 2, 64, lens, seed=21) as c:
        q = queries(5, 4, 64)
        m = pack(random_masks(nodes), 1).cuda()
        ip, t, ln = i32(ptr(nodes)), c.tables.cuda(), i32(lens)
        call = lambda **k: pkv.paged_tree_attention(*[{**dict(pool=c.pool, q=q, ip=ip, m=m, t=t, ln=ln, s=0.1), **k}[n]  # noqa: E731
                                                      for n in ("pool", "q", "ip", "m", "t", "ln", "s")])
        call()
        with pytest.raises(ValueError):
            call(m=m[:4])
        with pytest.raises(ValueError):
            call(m=m.to(torch.int32))
        with pytest.raises(ValueError):
            call(q=q.float())
        with pytest.raises(TypeError):
            call(q=q[0])
        with pytest.raises(ValueError):
            call(ip=ip.cpu())
        with pytest.raises(ValueError):
            call(ln=ln.long())
        with pytest.raises(pkv.PagedKVError):
            call(m=torch.zeros(5, 17, dtype=torch.int64, device="cuda"))
        with pytest.raises(pkv.PagedKVError):
            call(m=torch.zeros(5, 0, dtype=torch.int64, device="cuda"))
        with pytest.raises(pkv.PagedKVError):
            call(s=math.inf)
        with pytest.raises(pkv.PagedKVError):
            call(q=queries(5, 6, 64))  # three heads a KV head
        with pkv.kv_pool_create(4, 16, 2, 64, pkv.INT4) as p4, pytest.raises(pkv.PagedKVError):
            call(pool=p4)
        with pkv.kv_pool_create(4, 16, 2, 64, pkv.FP8_E4M3) as p8, pytest.raises(pkv.PagedKVError):
            call(pool=p8)  # no scales yet
        assert call(q=q[:0], m=m[:0], ip=i32([0, 0])).shape == (0, 4, 64)
        assert c.pool.get_error() == 0
