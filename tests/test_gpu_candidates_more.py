"""The edges of the calls for several candidates a sequence: memory that two arguments share, values that are not
finite, weights and scales at the ends of their types' ranges, beams that begin with one prompt."""
import math
import random

import numpy as np
import pytest
import torch

import gqa_decode_attention_paged_gb300 as pkv
from test_gpu_moves import Bytes, reorder
from tree_ref import BS, Cache, check, pack, parents_of, plain, tree_bits


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32).cuda()


def trees(c, nodes, G, seed):
    """Queries and what follows them in a call, the masks as numbers and the rows' offsets."""
    rng = random.Random(seed)
    bits = [m for n in nodes for m in tree_bits(parents_of(n, rng))]
    q = torch.randn(sum(nodes), G * c.n_kv, c.d, generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16).cuda()
    ip = np.cumsum([0] + list(nodes))
    words = (max(nodes) + 63) // 64
    return q, [i32(ip), pack(bits, words).cuda(), c.tables.cuda(), i32(c.lens), c.d ** -0.5], bits, ip


@pytest.mark.gpu
@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("lens,nodes,extra", [([3100, 200, 900, 16], [150, 3, 64, 1], 0), ([9000], [1000], 0), ([700, 900, 1000], [200, 70, 130], 0),
                                              ([700, 900, 1000], [200, 70, 130], 70)])
def test_several_units_of_a_head_may_write_over_their_queries(kv, lens, nodes, extra):
    """Eight query heads on a KV head: 256 rows are 32 nodes.  Tables of up to 64 blocks, whose units are whole, and
    wider ones, whose units are cut."""
    with Cache(kv, 2, 128, lens, seed=31, table_extra=extra) as c:
        q, args, bits, ip = trees(c, nodes, 8, 31)
        want = pkv.paged_tree_attention(c.pool, q, *args)
        check(want, *plain(c, q, ip, bits, lens, args[-1]))
        for _ in range(3):
            x = q.clone()
            assert pkv.paged_tree_attention(c.pool, x, *args, out=x) is x
            assert torch.equal(x, want)
        assert c.pool.get_error() == 0


@pytest.mark.gpu
def test_results_that_share_memory_with_an_input_are_refused():
    lens, nodes = [100, 40, 20], [6, 3, 1]
    with Cache("bf16", 2, 64, lens, seed=32) as c:
        q, args, bits, ip = trees(c, nodes, 4, 32)
        want = pkv.paged_tree_attention(c.pool, q, *args)
        n = q.numel()
        room = torch.zeros(3 * n + 512, dtype=torch.bfloat16, device="cuda")  # (the result's place is [n, 2 n))
        out = room[n:2 * n].view(q.shape)

        def put(x, at):
            """x's values at an offset (in bytes) of the room."""
            size = x.numel() * x.element_size()
            y = room.view(torch.uint8)[at:at + size].view(x.dtype).view(x.shape)
            y.copy_(x)
            return y

        row = 8 * 64 * 2
        lo, hi = 2 * n, 4 * n  # of the result, in bytes
        for at in (lo - row, lo + row, lo + 32, hi - row, lo - 2 * n + 16):  # (rows on and back, part of a row)
            with pytest.raises(pkv.PagedKVError, match="out overlaps q"):
                pkv.paged_tree_attention(c.pool, put(q, at), *args, out=out)
        for i in range(4):  # indptr, masks, tables, lengths: their last element in the result, and their first
            size = args[i].numel() * args[i].element_size()
            step = 8 if i == 1 else 4
            for at in (lo - size + step, lo + 64, hi - step):
                moved = [put(x, at) if j == i else x for j, x in enumerate(args[:4])]
                with pytest.raises(pkv.PagedKVError, match="out overlaps an input"):
                    pkv.paged_tree_attention(c.pool, q, *moved, args[4], out=out)
                with pytest.raises(pkv.PagedKVError, match="out overlaps an input"):  # and over the queries
                    pkv.paged_tree_attention(c.pool, out, *moved, args[4], out=out)
        inside = c.pool._alloc_bytes_view(c.pool.layout())[4096:][:q.numel() * 2].view(torch.bfloat16).view(q.shape)
        with pytest.raises(pkv.PagedKVError, match="out overlaps an input"):
            pkv.paged_tree_attention(c.pool, q, *args, out=inside)
        # next to one another is apart
        for at in (lo - 2 * n, hi):
            pkv.paged_tree_attention(c.pool, put(q, at), *args, out=out)
            assert torch.equal(out, want)
        for i in range(4):
            size = args[i].numel() * args[i].element_size()
            for at in (lo - size, hi):
                moved = [put(x, at) if j == i else x for j, x in enumerate(args[:4])]
                pkv.paged_tree_attention(c.pool, q, *moved, args[4], out=out)
                assert torch.equal(out, want)
        assert c.pool.get_error() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("gap", [9.0, 13.0, 15.0, 17.5])
@pytest.mark.parametrize("extra", [0, 200])
def test_what_little_weight_many_keys_have_next_to_one_that_has_most(kv, d, gap, extra):
    """The first key's score is `gap` above all others', and its value zero: the result is what the others add.
    Their weights, 2^-13 to 2^-25 of the first's, are bf16 on a bf16 pool (2^-8 of themselves, over its whole range).
    On an FP8 pool they are f16 after a factor of 2^7: 2^-11 of themselves down to 2^-21 of the first's, and half of
    f16's smallest step below, 2^-25 2^-7 of the first's.  The sum is at least the first's own weight."""
    lens, nodes = [1024, 1000, 17], [5, 40, 1]
    with Cache(kv, 2, d, lens, seed=33, table_extra=extra) as c:
        if kv == "fp8":
            c.pool.set_fp8_scales(np.ones(2, np.float32), np.ones(2, np.float32))
        c.k = torch.zeros(c.k.shape).to(c.k.dtype)
        c.v = (1 + torch.rand(c.v.shape, generator=torch.Generator().manual_seed(33))).to(c.v.dtype)
        for b in range(len(lens)):
            c.k[int(c.tables[b, 0]), :, 0, 0] = 16.0
            c.v[int(c.tables[b, 0]), :, 0] = 0.0
        c.k64, c.v64 = c.k.double(), c.v.double()
        c.upload()
        q, args, bits, ip = trees(c, nodes, 4, 33)
        q = torch.zeros_like(q)
        q[..., 0] = 1.0
        scale = float(np.float32(gap / 16.0))
        got = pkv.paged_tree_attention(c.pool, q, *args[:-1], scale)
        assert c.pool.get_error() == 0
        ref, _ = plain(c, q, ip, bits, lens, scale)
        e = (2.0 ** -8 if kv == "bf16" else 2.0 ** -11) + 2.0 ** -12
        small = 0.0 if kv == "bf16" else 2.0 ** -32 * max(lens) * 2  # (values are below 2)
        check(got, ref, 1.1 * (e * 2 * ref.abs() + small) + 2.0 ** -8 * ref.abs() + 1e-30)


@pytest.mark.gpu
@pytest.mark.parametrize("k_scale,scale", [(1e-16, 0.0), (1e-26, 1e-20), (1e-26, -1e-20), (1e-38, 1e-38), (1.0, 1e-45)])
def test_scales_whose_product_is_below_fp32(k_scale, scale):
    """Scores of zero to all that counts: what is visible weighs alike, what is not weighs nothing."""
    lens, nodes = [300, 20, 2100], [20, 20, 70]
    with Cache("fp8", 2, 64, lens, seed=34) as c:
        v_scale = np.array([0.01, 0.02], np.float32)
        c.pool.set_fp8_scales(np.full(2, k_scale, np.float32), v_scale)
        c.k64 = torch.zeros_like(c.k64)
        c.v64 = c.v.double() * torch.tensor(v_scale).double().view(1, 2, 1, 1)
        q, args, bits, ip = trees(c, nodes, 4, 34)
        got = pkv.paged_tree_attention(c.pool, q, *args[:-1], scale)
        assert c.pool.get_error() == 0
        check(got, *plain(c, q, ip, bits, lens, scale))


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("extra", [0, 200])
def test_values_that_are_not_finite_under_scores_of_minus_infinity(d, extra):
    """Of a key in the context, of a node, and where a sequence has no other scores: those channels are not finite in
    the rows that may see the key, and all else is as if the values were zero."""
    lens, nodes = [300, 2500, 40, 1000], [20, 40, 40, 9]
    # sequence, position, channels
    odd = [(0, 5, [3]), (0, 290, [7, 9]), (1, 2000, [0, 1, 2]), (1, 2461, [60]), (1, 2499, [4, 5]), (2, 3, [8]), (2, 39, range(20, 64)), (3, 998, [11])]
    with Cache("bf16", 2, d, lens, seed=35, table_extra=extra) as c:
        at = lambda b, pos: (int(c.tables[b, pos // BS]), slice(None), pos % BS)  # noqa: E731
        for b, pos, _ in odd + [(2, p, None) for p in range(40)]:  # (all scores of sequence 2 are)
            c.k[at(b, pos)] = c.k[at(b, pos)].index_fill(1, torch.tensor([0]), -math.inf)
        c.k64, c.v64 = c.k.double(), c.v.double()
        q, args, bits, ip = trees(c, nodes, 4, 35)
        q[..., 0] = 1
        hit = torch.zeros(sum(nodes), 8, d, dtype=torch.bool)
        for i, (b, pos, channels) in enumerate(odd):
            v = torch.zeros(2, d)
            v[:, list(channels)] = [math.inf, -math.inf, math.nan][i % 3]
            c.v[at(b, pos)] = torch.where(v == 0, c.v[at(b, pos)].float(), v).to(torch.bfloat16)
            c.v64[at(b, pos)] = torch.where(v == 0, c.v64[at(b, pos)], 0.0)
            node = pos - (lens[b] - nodes[b])
            for r in range(ip[b], ip[b + 1]):
                if node < 0 or (bits[r] >> node) & 1:
                    hit[r][:, list(channels)] = True
        c.upload()
        got = pkv.paged_tree_attention(c.pool, q, *args).cpu()
        assert c.pool.get_error() == 0
        assert hit.any() and not hit.all()
        assert torch.equal(~torch.isfinite(got), hit)
        ref, bound = plain(c, q, ip, bits, lens, args[-1])
        check(torch.where(hit, 0, got), torch.where(hit, 0, ref), bound)
        assert (got[ip[2]:ip[3]][~hit[ip[2]:ip[3]]] == 0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("kv", ["bf16", "fp8", "int4"])
@pytest.mark.parametrize("length", [1, 16, 37, 80])
def test_the_first_step_of_beams_that_share_a_prompt(kv, length):
    """Every beam's table is the prompt's, its unfilled block among them; one beam goes on, the others' scores are
    -infinity.  Afterwards each new beam has a block of its own to write."""
    searches, beams = 3, 4
    rng = random.Random(36)
    W = length // BS + 1
    ids = rng.sample(range(40), 40)
    table = np.array([ids[b * W:(b + 1) * W] for b in range(searches) for _ in range(beams)], np.int32)
    spare = ids[searches * W:searches * W + searches * beams]
    scores = torch.full((searches, beams), -math.inf)
    logits = torch.randn(searches, 1, 50, generator=torch.Generator().manual_seed(36)).expand(-1, beams, -1).contiguous()
    alive = [0, 2, 3]
    for b, j in enumerate(alive):
        scores[b, j] = 0.0
    with Bytes(kv, 2, 64, 40) as m:
        tokens, parents, _ = pkv.paged_beam_select(m.pool, logits.cuda(), scores.cuda(), beams)
        assert parents.tolist() == [[j] * beams for j in alive]
        assert tokens.tolist() == logits[:, 0].double().sort(dim=-1, descending=True, stable=True)[1][:, :beams].tolist()
        got, after = pkv.paged_beam_reorder(m.pool, parents, i32(table), i32([length] * len(table)), i32(spare))
        want, lens = reorder(m, parents.tolist(), table, [length] * len(table), spare, beams)
        m.check()
        assert got.tolist() == want and after.tolist() == lens == [length] * len(table)
        writes = [t[length // BS] for t in got.tolist()]
        assert len(set(writes)) == len(writes)
        assert m.pool.get_error() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("lens,nodes,G", [([131072], [2], 4), ([70000], [90], 4), ([66000, 40000], [3, 40], 1)])
def test_units_in_more_parts_than_a_warp_joins_at_once(kv, lens, nodes, G):
    """One KV head and few rows: a unit's parts are in tens of slices, up to all of them."""
    with Cache(kv, 1, 64, lens, seed=37) as c:
        q, args, bits, ip = trees(c, nodes, G, 37)
        got = pkv.paged_tree_attention(c.pool, q, *args)
        assert c.pool.get_error() == 0
        check(got, *plain(c, q, ip, bits, lens, args[-1]))
