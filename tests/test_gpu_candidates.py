"""The calls for several candidates a sequence, together as they are used: steps with trees of drafted tokens, and a
beam search, over pools of two layers; and their workspaces."""
import math
import random

import numpy as np
import pytest
import torch

import gqa_decode_attention_paged_gb300 as pkv
from test_gpu_beam_select import check as check_selection
from tree_ref import BS, Cache, check, pack, parents_of, plain, tree_bits

N_KV, G, D, LAYERS = 2, 4, 128, 2
KINDS = {"bf16": pkv.BF16, "fp8": pkv.FP8_E4M3}


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32).cuda()


class Layer:
    """A pool, and what it should hold: rows[sequence] is a list of (key, value), as they are stored, in 64 bits."""

    def __init__(self, kv, blocks, seed):
        self.kv, self.n_kv, self.d, self.blocks = kv, N_KV, D, blocks
        self.pool = pkv.kv_pool_create(blocks, BS, N_KV, D, KINDS[kv])
        self.scales = np.full(N_KV, 5 / 448, np.float32)
        if kv == "fp8":
            self.pool.set_fp8_scales(self.scales, self.scales)

    def stored(self, x):
        if self.kv == "bf16":
            return x.double()
        s = float(self.scales[0])
        return (x.float() / s).clamp(-448, 448).to(torch.float8_e4m3fn).double() * s

    def attention(self, q, indptr, bits, history, scale):
        """plain() over sequences whose rows are given one after the other."""
        n = [(len(h) + BS - 1) // BS for h in history]
        tables, at = torch.full((len(history), max(n)), 0, dtype=torch.int32), 0
        self.k64 = torch.zeros(max(1, sum(n)), N_KV, BS, D, dtype=torch.float64)
        self.v64 = torch.zeros_like(self.k64)
        for b, h in enumerate(history):
            tables[b, :n[b]] = torch.arange(at, at + n[b], dtype=torch.int32)
            for i, (k, v) in enumerate(h):
                self.k64[at + i // BS, :, i % BS], self.v64[at + i // BS, :, i % BS] = k, v
            at += n[b]
        self.tables, blocks = tables, self.blocks
        self.blocks = max(1, at)
        try:
            return plain(self, q, indptr, bits, [len(h) for h in history], scale)
        finally:
            self.blocks = blocks


def slots_of(table, first, n):
    return [int(table[p // BS]) * BS + p % BS for p in range(first, first + n)]


def append(layer, kv, slots):
    pkv.paged_kv_append(layer.pool, torch.stack([k for k, _ in kv]).cuda(), torch.stack([v for _, v in kv]).cuda(),
                        torch.tensor(slots, dtype=torch.int64).cuda())


def row(g):
    return tuple(torch.randn(N_KV, D, generator=g).to(torch.bfloat16) for _ in range(2))


@pytest.mark.gpu
@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_steps_with_drafted_tokens(kv):
    """Four steps of three sequences: draft a tree, attend, accept a path (none of it, a part, all), go on."""
    g, rng = torch.Generator().manual_seed(5), random.Random(5)
    scale, W = 1 / math.sqrt(D), 12
    layers = [Layer(kv, 3 * W, s) for s in range(LAYERS)]
    order = list(range(3 * W))
    rng.shuffle(order)
    tables = np.array(order, np.int32).reshape(3, W)
    history = [[[] for _ in range(3)] for _ in layers]
    lens = [0, 31, 70]
    for layer, h in zip(layers, history):
        for b, c in enumerate(lens):
            if not c:
                continue
            rows = [row(g) for _ in range(c)]
            append(layer, rows, slots_of(tables[b], 0, c))
            h[b] = [(layer.stored(k), layer.stored(v)) for k, v in rows]
    t = i32(tables)
    for step, nodes in enumerate(([5, 17, 33], [1, 20, 9], [12, 0, 40], [3, 26, 1])):
        parents = [parents_of(n, rng) for n in nodes]
        bits = [m for p in parents for m in tree_bits(p)]
        ip, total = np.cumsum([0] + nodes), sum(nodes)
        here = [c + n for c, n in zip(lens, nodes)]
        paths = []
        for b, p in enumerate(parents):
            path, i = [], rng.randrange(nodes[b]) if nodes[b] and (step + b) % 4 else -1
            while i >= 0:
                path.insert(0, i)
                i = p[i]
            paths.append(path)
        most = max(map(len, paths)) + 2
        accepted = i32([p + [-9] * (most - len(p)) for p in paths])
        count, after = i32([len(p) for p in paths]), []
        for layer, h in zip(layers, history):
            drafted = [[row(g) for _ in range(n)] for n in nodes]
            append(layer, [kv_ for d in drafted for kv_ in d],
                   [s for b, n in enumerate(nodes) for s in slots_of(tables[b], lens[b], n)])
            stored = [[(layer.stored(k), layer.stored(v)) for k, v in d] for d in drafted]
            q = torch.randn(total, N_KV * G, D, generator=g).to(torch.bfloat16).cuda()
            got = pkv.paged_tree_attention(layer.pool, q, i32(ip), pack(bits, 1).cuda(), t, i32(here), scale)
            check(got, *layer.attention(q, ip, bits, [h[b] + stored[b] for b in range(3)], scale))
            after.append(pkv.paged_tree_commit(layer.pool, i32(ip), accepted, count, t, i32(here)))
            for b, path in enumerate(paths):
                h[b] = h[b] + [stored[b][i] for i in path]
        lens = [len(x) for x in history[0]]
        for layer, h, a in zip(layers, history, after):
            assert a.tolist() == lens
            # what is cached now is the accepted text
            k, v = pkv.paged_kv_gather(layer.pool, i32(np.cumsum([0] + lens)), t, n_rows=sum(lens))
            want = [x for s in h for x in s]
            if kv == "bf16" and want:
                assert torch.equal(k.double().cpu(), torch.stack([x for x, _ in want]))
                assert torch.equal(v.double().cpu(), torch.stack([x for _, x in want]))
            # and a token behind it (here: the last one, again) attends to it
            q = torch.randn(3, N_KV * G, D, generator=g).to(torch.bfloat16).cuda()
            got = pkv.paged_decode_attention(layer.pool, q, t, a, scale)
            some = [b for b in range(3) if lens[b]]
            ref, bound = layer.attention(q, [0, 1, 2, 3], [1] * 3, [x if x else [(torch.zeros(N_KV, D).double(),) * 2] for x in h],
                                         scale)
            check(got[some], ref[some], bound[some])
            assert layer.pool.get_error() == 0
    assert all(c > first for c, first in zip(lens, (0, 31, 70)))
    for layer in layers:
        layer.pool.close()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("S,beams,steps", [(3, 4, 40), (1, 7, 20)])
def test_a_beam_search(dtype, S, beams, steps):
    """Decode, logits, selection and reordering in turn, with a block allocator: the selection is the one of 64-bit
    arithmetic on the same logits, and every beam's cache is its own text's."""
    g = torch.Generator().manual_seed(9)
    vocab, scale, n = 500, 1 / math.sqrt(D), S * beams
    W = (steps + BS - 1) // BS + 1
    blocks = n * (W + 3)
    layers = [Layer("bf16", blocks, s) for s in range(LAYERS)]
    kv = [[row(g) for _ in range(vocab)] for _ in layers]
    heads = [torch.randn(vocab, N_KV * G, D, generator=g).to(torch.bfloat16).cuda() for _ in layers]
    unembed = (torch.randn(N_KV * G * D, vocab, generator=g) * 0.5).cuda()
    with pkv.BlockAllocator(blocks) as alloc:
        tables = np.full((n, W), -1, np.int32)
        lens, text = [0] * n, [[i % vocab] for i in range(n)]
        scores = torch.full((S, beams), -math.inf)
        scores[:, 0] = 0  # one beam to begin with
        scores = scores.cuda()
        for step in range(steps):
            for r in range(n):  # the block that is written next
                if lens[r] >= 0 and tables[r, lens[r] // BS] < 0:
                    tables[r, lens[r] // BS] = alloc.take(1)[0]
            t, slots = i32(tables), [s for r in range(n) for s in slots_of(tables[r], lens[r], 1)]
            token = [x[-1] for x in text]
            lens = [c + 1 for c in lens]
            x = 0
            for layer, rows, q in zip(layers, kv, heads):
                append(layer, [rows[i] for i in token], slots)
                got = pkv.paged_decode_attention(layer.pool, q[token], t, i32(lens), scale)
                if step % 9 == 0 or step == steps - 1:
                    want = [[tuple(y.double() for y in rows[i]) for i in x_] for x_ in text]
                    check(got, *layer.attention(q[token], range(n + 1), [1] * n, want, scale))
                x = x + got.float().flatten(1) @ unembed
            logits = x.view(S, beams, vocab).to(dtype)
            tokens, parents, scores = check_selection(layers[0].pool, logits, scores, beams)
            spare = alloc.take(n)
            for layer in layers:
                new, after = pkv.paged_beam_reorder(layer.pool, parents, t, i32(lens), i32(spare))
                assert torch.equal(new, pkv.paged_beam_reorder(layers[0].pool, parents, t, i32(lens), i32(spare))[0])
            new = new.cpu().numpy()
            alloc.share(new[new >= 0])
            alloc.release(spare)
            alloc.release(tables[tables >= 0])
            at = [s * beams + p for s, ps in enumerate(parents.tolist()) for p in ps]
            assert min(at) >= 0
            text = [text[p] + [i] for p, i in zip(at, tokens.view(-1).tolist())]
            lens = [lens[p] for p in at]
            assert after.tolist() == lens
            tables = new.copy()
            for r in range(n):  # the block that is written next is no other beam's
                b = tables[r, lens[r] // BS]
                assert b < 0 or alloc.refcount(b) == 1
        assert len({tuple(x) for x in text}) == n
        alloc.release(tables[tables >= 0])
        assert alloc.free_blocks() == blocks
    for layer in layers:
        assert layer.pool.get_error() == 0
        layer.pool.close()


def tree_args(layer, nodes, lens, seed):
    rng, g = random.Random(seed), torch.Generator().manual_seed(seed)
    bits = [m for n in nodes for m in tree_bits(parents_of(n, rng))]
    q = torch.randn(sum(nodes), N_KV * G, D, generator=g).to(torch.bfloat16).cuda()
    W = max((c + BS - 1) // BS for c in lens)
    t = i32([[(b * W + e) % layer.blocks for e in range(W)] for b in range(len(lens))])
    return q, i32(np.cumsum([0] + nodes)), pack(bits, 1).cuda(), t, i32(lens), 1 / math.sqrt(D)


def fill(layer, seed):
    g = torch.Generator().manual_seed(seed)
    n = layer.blocks * BS
    k, v = (torch.randn(n, N_KV, D, generator=g).to(torch.bfloat16).cuda() for _ in range(2))
    pkv.paged_kv_append(layer.pool, k, v, torch.arange(n, dtype=torch.int64, device="cuda"))


@pytest.mark.gpu
def test_a_reserved_workspace_is_enough_for_smaller_calls_and_captures():
    layer = Layer("bf16", 64, 0)
    fill(layer, 1)
    args = tree_args(layer, [30, 7], [500, 90], 2)
    torch.cuda.synchronize()
    with pytest.raises(pkv.PagedKVError):  # nothing may be allocated there
        with torch.cuda.graph(torch.cuda.CUDAGraph()):
            pkv.paged_tree_attention(layer.pool, *args)
    layer.pool.reserve_tree_workspace(200, N_KV * G)
    have = layer.pool.timing_read()["workspace_bytes"]
    assert have > 0
    out = torch.zeros_like(args[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pkv.paged_tree_attention(layer.pool, *args, out=out)
    graph.replay()
    assert torch.equal(out, pkv.paged_tree_attention(layer.pool, *args))
    for nodes in ([64, 64, 64, 8], [1], [60] * 3, [0, 2]):
        pkv.paged_tree_attention(layer.pool, *tree_args(layer, nodes, [900] * len(nodes), 3))
    torch.cuda.synchronize()
    assert layer.pool.timing_read()["workspace_bytes"] == have
    for bad in ((-1, 8), (4, 3), (4, 0)):
        with pytest.raises(pkv.PagedKVError):
            layer.pool.reserve_tree_workspace(*bad)
    layer.pool.close()


@pytest.mark.gpu
def test_graphs_of_one_pool_take_turns():
    """A tree's, a selection's and a decode's graph use the same workspace, which grows between their captures."""
    layer = Layer("bf16", 64, 0)
    fill(layer, 4)
    pool, args = layer.pool, tree_args(layer, [40, 3, 25], [800, 700, 30], 5)
    g = torch.Generator().manual_seed(6)
    logits, scores = torch.randn(4, 5, 20001, generator=g).cuda(), torch.zeros(4, 5).cuda()
    wide, more = torch.randn(16, 8, 60000, generator=g).cuda(), torch.zeros(16, 8).cuda()
    calls = [lambda: (pkv.paged_beam_select(pool, logits, scores, 6)),
             lambda: (pkv.paged_tree_attention(pool, *args),),
             lambda: (pkv.paged_decode_attention(pool, args[0][:3].contiguous(), *args[3:]),),
             lambda: (pkv.paged_beam_select(pool, wide, more, 64))]
    graphs, outs = [], []
    for call in calls:
        call()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(call())
        graphs.append(graph)
    want = [call() for call in calls]
    for order in ((0, 1, 2, 3), (3, 1, 0, 2), (1, 1, 3, 0, 2)):
        for o in outs:
            for x in o:
                x.zero_()
        for i in order:
            graphs[i].replay()
        torch.cuda.synchronize()
        for w, o in zip(want, outs):
            assert all(torch.equal(x, y) for x, y in zip(w, o))
    assert pool.get_error() == 0
    layer.pool.close()


@pytest.mark.gpu
def test_eight_thousand_sequences():
    layer = Layer("fp8", 500, 0)
    fill(layer, 7)
    rng = random.Random(8)
    nodes = [rng.choice([0, 1, 1, 2, 3]) for _ in range(8192)]
    lens = [max(n, rng.choice([0, 1, 17, 40])) for n in nodes]
    args = tree_args(layer, nodes, lens, 9)
    got = pkv.paged_tree_attention(layer.pool, *args)
    # each sequence is one of few, as what it sees is: the same call with those that hold its nodes alone
    for at in (0, 1, 4000, 8191):
        lo, hi = sum(nodes[:at]), sum(nodes[:at + 1])
        if lo == hi:
            continue
        one = pkv.paged_tree_attention(layer.pool, args[0][lo:hi].contiguous(), i32([0, hi - lo]), args[2][lo:hi].contiguous(),
                                       args[3][at:at + 1].contiguous(), args[4][at:at + 1].contiguous(), args[5])
        assert torch.equal(got[lo:hi], one)  # (one step of keys: never cut)
    assert torch.isfinite(got).all() and (got.float().abs().amax((1, 2)) > 0).all()
    assert layer.pool.get_error() == 0
    layer.pool.close()


@pytest.mark.gpu
@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_a_block_that_a_table_names_twice(kv):
    """Shared and repeated blocks are read as often as tables name them."""
    layer = Layer(kv, 3, 0)
    g = torch.Generator().manual_seed(10)
    rows = [row(g) for _ in range(48)]
    append(layer, rows, list(range(48)))
    stored = [(layer.stored(k), layer.stored(v)) for k, v in rows]
    tables = [[0, 1, 0, 2], [2, 2, 2, 2]]
    lens, nodes = [60, 64], [5, 20]
    rng = random.Random(11)
    bits = [m for n in nodes for m in tree_bits(parents_of(n, rng))]
    q = torch.randn(25, N_KV * G, D, generator=g).to(torch.bfloat16).cuda()
    got = pkv.paged_tree_attention(layer.pool, q, i32([0, 5, 25]), pack(bits, 1).cuda(), i32(tables), i32(lens), 0.1)
    history = [[stored[t[p // BS] * BS + p % BS] for p in range(c)] for t, c in zip(tables, lens)]
    check(got, *layer.attention(q, [0, 5, 25], bits, history, 0.1))
    layer.pool.close()


@pytest.mark.gpu
def test_rows_in_one_piece_are_summed_as_exactly():
    """More rows than blocks run at once: a row is one piece of many parts, whose sums a thread adds one after the
    other.  Flat rows, so that every term counts: the sum of n exponentials of at most 0, each within 2^-21 of itself
    and in 16 terms' 32-bit additions within 2^-20, to which the other additions add 2^-40."""
    rows, vocab = 460, 1 << 19
    x = torch.empty(rows, 1, vocab, dtype=torch.bfloat16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(12)
    x.copy_((torch.rand(rows, 1, vocab, device="cuda", generator=g) - 1) * 0.5)
    with pkv.kv_pool_create(2, 16, 1, 64, pkv.BF16) as pool:
        tokens, parents, best = pkv.paged_beam_select(pool, x, torch.zeros(rows, 1, device="cuda"), 3)
        assert pool.get_error() == 0
    for r in (0, 1, 459):
        v, at = torch.log_softmax(x[r, 0].double(), -1).sort(descending=True, stable=True)
        assert torch.equal(tokens[r].long(), at[:3])
        err = (best[r].double() - v[:3]).abs()
        assert (err <= 2.0 ** -21 + 2.0 ** -20 + 2.0 ** -24 * v[:3].abs()).all(), err


@pytest.mark.gpu
@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lens,nodes", [([200, 90], [40, 10]), ([16, 300], [16, 129]), ([3000, 50], [100, 1]), ([9000, 1200], [90, 64])])
def test_what_hidden_nodes_hold_does_not_matter(kv, d, lens, nodes):
    """Keys and values of some nodes that are not finite (padding behind a tree, a branch that was not computed): rows
    that see a node have its channels' NaN and infinities, all else is as with zeros there."""
    rng = random.Random(13)
    with Cache(kv, 2, d, lens, seed=13) as c:
        bits = [m for n in nodes for m in tree_bits(parents_of(n, rng))]
        pads = {}  # (sequence, node): KV head, channels whose values are not finite
        for b, n in enumerate(nodes):
            for j in sorted({n - 1, n // 2, n // 3 + 1} - {0}):
                if j < n:
                    pads[b, j] = (rng.randrange(2), sorted(rng.sample(range(d), rng.choice([1, d]))))
        ip = np.cumsum([0] + nodes)
        nan = torch.zeros(sum(nodes), 8, d, dtype=torch.bool)
        for (b, j), (g, channels) in pads.items():
            pos = lens[b] - nodes[b] + j
            blk = int(c.tables[b, pos // BS])
            bad = torch.tensor([math.nan if kv == "fp8" or i % 3 else math.inf for i in channels]).to(c.v.dtype)
            c.v.view(torch.uint8).view(*c.v.shape, -1)[blk, g, pos % BS, channels] = bad.view(torch.uint8).view(len(channels), -1)
            c.v64[blk, g, pos % BS, channels] = 0.0
            for r in range(ip[b], ip[b + 1]):
                if (bits[r] >> j) & 1:
                    nan[r, 4 * g:4 * g + 4, channels] = True
        c.upload()
        q = torch.randn(sum(nodes), 8, d, generator=torch.Generator().manual_seed(14)).to(torch.bfloat16).cuda()
        words = (max(nodes) + 63) // 64
        call = lambda: pkv.paged_tree_attention(c.pool, q, i32(ip), pack(bits, words).cuda(), c.tables.cuda(), i32(lens), d ** -0.5)  # noqa: E731
        got = call().cpu()
        assert nan.any() and not nan.all()
        assert torch.equal(~torch.isfinite(got), nan)
        ref, bound = plain(c, q, ip, bits, lens, d ** -0.5)
        check(torch.where(nan, 0, got), torch.where(nan, 0, ref), bound)
        # and keys: NaN ones of nodes that no row sees change nothing
        unseen = [(b, n - 1) for b, n in enumerate(nodes) if n > 1]
        for b, j in unseen:
            for r in range(ip[b], ip[b + 1]):
                bits[r] &= ~(1 << j)
        want = call()
        for b, j in unseen:
            pos = lens[b] - nodes[b] + j
            c.k.view(torch.uint8)[int(c.tables[b, pos // BS]), :, pos % BS] = torch.full((d,), math.nan).to(c.k.dtype).view(torch.uint8)
        c.upload()
        assert torch.equal(call().nan_to_num(7, 8, 9), want.nan_to_num(7, 8, 9))
        assert c.pool.get_error() == 0


@pytest.mark.gpu
def test_the_result_may_replace_the_queries():
    layer = Layer("bf16", 200, 0)
    fill(layer, 15)
    args = tree_args(layer, [40, 3, 64, 1], [3100, 70, 900, 16], 16)
    want = pkv.paged_tree_attention(layer.pool, *args)
    for _ in range(3):
        q = args[0].clone()
        assert pkv.paged_tree_attention(layer.pool, q, *args[1:], out=q) is q
        assert torch.equal(q, want)
    layer.pool.close()


@pytest.mark.gpu
def test_the_widest_selection():
    """64 beams of 2^22 logits, 64 of their 2^28 continuations; more than that is refused."""
    beams, vocab, k = 64, 1 << 22, 64
    g = torch.Generator(device="cuda").manual_seed(17)
    x = torch.empty(1, beams, vocab, device="cuda")
    for j in range(beams):
        x[0, j] = torch.randn(vocab, device="cuda", generator=g)
    scores = -torch.rand(1, beams, device="cuda", generator=g)
    with pkv.kv_pool_create(2, 16, 1, 64, pkv.BF16) as pool:
        tokens, parents, best = pkv.paged_beam_select(pool, x, scores, k)
        assert pool.get_error() == 0
        for bad in (dict(logits=torch.zeros(1, 1, vocab + 1, device="cuda"), scores=scores[:, :1].contiguous(), k=1),
                    dict(logits=x, scores=scores, k=65)):
            with pytest.raises(pkv.PagedKVError):
                pkv.paged_beam_select(pool, **bad)
    lse = torch.stack([torch.logsumexp(x[0, j].double(), 0) for j in range(beams)])
    top = torch.stack([x[0, j].topk(k).values.double() for j in range(beams)]) - lse[:, None] + scores[0].double()[:, None]
    want = top.flatten().sort(descending=True).values[:k]
    p, t = parents[0].long(), tokens[0].long()
    mine = x[0, p, t].double() - lse[p] + scores[0, p].double()
    # the sums of exponentials are within 2^-19 as in a row of one piece, and ranks by at most as much
    assert ((mine - want).abs() <= 2.0 ** -18).all() and len({*zip(p.tolist(), t.tolist())}) == k
    assert ((best[0].double() - mine).abs() <= 2.0 ** -19 + 2.0 ** -24 * mine.abs()).all()


def spread(lo, hi, n, seed):
    rng = random.Random(seed)
    return [rng.randint(lo, hi) for _ in range(n)]


# lengths, nodes, KV heads: one unit a CTA (few and many sequences); small units, several a CTA; long ones among short
# ones; few long ones; units of one tile and of two
SLICES = [([1000, 1100, 900], [20, 60, 33], 2), (spread(800, 1300, 60, 1), spread(1, 40, 60, 2), 2),
          (spread(20, 1000, 100, 3), spread(1, 20, 100, 4), 2), (spread(60, 300, 100, 5) + [6000], spread(1, 30, 101, 6), 2),
          ([9000, 2000], [10, 64], 1), (spread(100, 1024, 41, 7), spread(33, 64, 41, 8), 4)]


@pytest.mark.gpu
@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("extra", [0, 70])
@pytest.mark.parametrize("case", range(len(SLICES)))
def test_units_that_are_cut_and_that_are_not(kv, extra, case):
    """The same trees with tables as wide as they need, and wider: what is cut depends on that, and on their lengths."""
    lens, nodes, n_kv = SLICES[case]
    with Cache(kv, n_kv, 64 if case % 2 else 128, lens, seed=case, table_extra=extra) as c:
        rng = random.Random(case)
        bits = [m for n in nodes for m in tree_bits(parents_of(n, rng))]
        ip = np.cumsum([0] + nodes)
        q = torch.randn(sum(nodes), 4 * n_kv, c.d, generator=torch.Generator().manual_seed(case)).to(torch.bfloat16).cuda()
        got = pkv.paged_tree_attention(c.pool, q, i32(ip), pack(bits, 1).cuda(), c.tables.cuda(), i32(lens), c.d ** -0.5)
        assert c.pool.get_error() == 0
        check(got, *plain(c, q, ip, bits, lens, c.d ** -0.5))


@pytest.mark.gpu
@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_a_graph_whose_lengths_change_what_is_cut(kv):
    lens, nodes = [4000, 500, 3900, 300], [20, 5, 40, 64]
    with Cache(kv, 2, 128, lens, seed=18, table_extra=0) as c:
        rng = random.Random(18)
        bits = [m for n in nodes for m in tree_bits(parents_of(n, rng))]
        ip = np.cumsum([0] + nodes)
        q = torch.randn(sum(nodes), 8, 128, generator=torch.Generator().manual_seed(18)).to(torch.bfloat16).cuda()
        args = [q, i32(ip), pack(bits, 1).cuda(), c.tables.cuda(), i32(lens), 128 ** -0.5]
        c.pool.reserve_tree_workspace(sum(nodes), 8)
        out = torch.zeros_like(q)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            pkv.paged_tree_attention(c.pool, *args, out=out)
        for now in ([4000, 500, 3900, 300], [400, 500, 390, 300], [20, 5, 40, 64], [4000, 5, 40, 64], [1000, 500, 900, 300]):
            args[4].copy_(i32(now))
            out.zero_()
            graph.replay()
            torch.cuda.synchronize()
            check(out, *plain(c, q, ip, bits, now, 128 ** -0.5))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,vocab", [(torch.float32, 50001), (torch.bfloat16, 100003)])
@pytest.mark.parametrize("kind", ["random", "rising", "late", "levels", "half"])
@pytest.mark.parametrize("k", [20, 64])
def test_selection_of_rows_in_one_piece(dtype, vocab, kind, k):
    """More rows than blocks run at once, each read by one block, in more parts than its first bar is good for."""
    S, beams = 115, 4
    g = torch.Generator().manual_seed(k)
    x = torch.randn(S, beams, vocab, generator=g)
    at = torch.arange(vocab) / vocab
    if kind == "rising":  # every part is above the one before
        x = x * 0.01 + 8 * at
    elif kind == "late":  # the best are at the end
        x = x + (at > 0.9) * 4.0
    elif kind == "levels":  # many equal ones
        x = (x * 2).round() / 2
    elif kind == "half":  # rising, behind where the second bar is from
        x = x * 0.1 + (at > 0.75) * (at - 0.75) * 20
    scores = -torch.rand(S, beams, generator=g).cuda()
    with pkv.kv_pool_create(2, 16, 1, 64, pkv.BF16) as pool:
        check_selection(pool, x.to(dtype).cuda(), scores, k)
