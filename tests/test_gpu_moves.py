"""Accepted paths and reordered beams: which bytes of the cache move, bit for bit, and which tables come out."""
import random

import numpy as np
import pytest
import torch

import gqa_decode_attention_paged_gb300 as pkv

KINDS = {"bf16": pkv.BF16, "fp8": pkv.FP8_E4M3, "int4": pkv.INT4}
BS = 16


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32).cuda()


class Bytes:
    """A pool of random bytes (NaN and infinities among them) and its mirror."""

    def __init__(self, kv, n_kv, d, blocks, seed=0):
        self.pool = pkv.kv_pool_create(blocks, BS, n_kv, d, KINDS[kv])
        g = torch.Generator().manual_seed(seed)
        self.views = [self.pool.k_view(), self.pool.v_view()]
        self.host = [torch.randint(0, 256, v.shape, generator=g, dtype=torch.uint8) for v in self.views]
        if kv == "int4":
            self.views.append(self.pool.v_params_view())
            self.host.append(torch.randn(self.views[2].shape, generator=g))
        for v, h in zip(self.views, self.host):
            v.copy_(h.cuda())
        torch.cuda.synchronize()

    def check(self):
        torch.cuda.synchronize()
        for v, h in zip(self.views, self.host):
            assert torch.equal(v.cpu(), h)

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.views = None
        self.pool.close()


def tables_for(lens, blocks, rng, extra=1):
    need = [(c + BS - 1) // BS for c in lens]
    W = max(need + [0]) + extra
    ids = list(range(blocks))
    rng.shuffle(ids)
    t = np.full((len(lens), W), -1, np.int32)
    at = 0
    for b, n in enumerate(need):
        t[b, :n] = ids[at:at + n]
        at += n
    return t, ids[at:]


def move(m, table, first, path):
    new = [[h[int(table[(first + j) // BS]), :, (first + j) % BS].clone() for h in m.host] for j in path]
    for i, rows in enumerate(new):
        for h, x in zip(m.host, rows):
            h[int(table[(first + i) // BS]), :, (first + i) % BS] = x


def paths(nodes, rng):
    """All nodes, none, the first, the last, a random ascending choice (places that others come from among them)."""
    out = []
    for b, t in enumerate(nodes):
        kind = b % 5
        out.append(list(range(t)) if kind == 0 else [] if kind == 1 else [t - 1][:t] if kind == 2 else
                   sorted(rng.sample(range(t), rng.randint(0, t))) if kind == 3 else sorted(rng.sample(range(t), min(t, 4))))
    return out


def padded(ps, most, fill=99):
    return np.array([p + [fill] * (most - len(p)) for p in ps], np.int32).reshape(len(ps), most)


@pytest.mark.gpu
@pytest.mark.parametrize("kv", ["bf16", "fp8", "int4"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n_kv", [1, 3, 8])
def test_commit_moves_the_path_and_nothing_else(kv, d, n_kv):
    rng = random.Random(d + n_kv)
    nodes = [5, 8, 1, 33, 64, 17, 1, 2, 200, 129, 0, 16, 31, 150]
    lens = [n + rng.randrange(60) for n in nodes]
    lens[3] = 33
    ps = paths(nodes, rng)
    table, _ = tables_for(lens, 250, rng)
    with Bytes(kv, n_kv, d, 250) as m:
        most = max(len(p) for p in ps) + 2
        got = pkv.paged_tree_commit(m.pool, i32(np.cumsum([0] + nodes)), i32(padded(ps, most)), i32([len(p) for p in ps]),
                                    i32(table), i32(lens))
        for b, p in enumerate(ps):
            move(m, table[b], lens[b] - nodes[b], p)
        m.check()
        assert got.tolist() == [c - t + len(p) for c, t, p in zip(lens, nodes, ps)]
        assert m.pool.get_error() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("kv", ["bf16", "int4"])
def test_commit_leaves_what_does_not_fit(kv):
    """Paths that are not ascending or leave the tree, counts and lengths that do not fit: the sequence keeps its rows."""
    nodes = [6, 6, 6, 6, 6, 6, 6, 6, 6]
    lens = [50, 50, 50, 50, 50, 4, 50, 50, 50]
    ps = [[0, 2, 5], [0, 3, 3], [2, 1], [0, 6], [-1, 2], [0, 2], [0, 1, 2, 3, 4, 5], [0, 2], [1, 4]]
    count = [3, 3, 2, 2, 2, 2, 7, -1, 2]
    rng = random.Random(1)
    table, _ = tables_for(lens, 60, rng)
    with Bytes(kv, 2, 64, 60) as m:
        got = pkv.paged_tree_commit(m.pool, i32(np.cumsum([0] + nodes)), i32(padded(ps, 6)), i32(count), i32(table), i32(lens))
        for b in (0, 8):
            move(m, table[b], 44, ps[b])
        m.check()
        assert got.tolist() == [47, 44, 44, 44, 44, 0, 44, 44, 46]
        assert m.pool.get_error(clear=True) == pkv.DEVERR_CTX_RANGE
        # a length past the table is clamped to it; rows that run backwards are no nodes
        got = pkv.paged_tree_commit(m.pool, i32([0, 6, 3]), i32([[0, 2], [0, 1]]), i32([2, 2]), i32(table[:2]),
                                    i32([table.shape[1] * BS + 1, 50]))
        m.check()
        assert got.tolist() == [table.shape[1] * BS - 6, 50]
        assert m.pool.get_error(clear=True) == pkv.DEVERR_CTX_RANGE


@pytest.mark.gpu
def test_commit_skips_rows_of_blocks_outside_the_pool():
    lens, nodes, ps = [64, 64], [40, 40], [[3, 20, 30], [3, 20, 30]]
    rng = random.Random(2)
    table, _ = tables_for(lens, 20, rng)
    with Bytes("bf16", 2, 64, 20) as m:
        bad = table.copy()
        bad[0, (24 + 20) // BS] = -1  # the second row's source
        bad[1, (24 + 1) // BS] = 20   # all places
        got = pkv.paged_tree_commit(m.pool, i32([0, 40, 80]), i32(ps), i32([3, 3]), i32(bad), i32(lens))
        for i, j in ((0, 3), (2, 30)):
            for h in m.host:
                h[table[0, (24 + i) // BS], :, (24 + i) % BS] = h[table[0, (24 + j) // BS], :, (24 + j) % BS]
        m.check()
        assert got.tolist() == [27, 27]
        assert m.pool.get_error(clear=True) == pkv.DEVERR_BLOCK_RANGE


@pytest.mark.gpu
def test_commit_captured_on_another_stream_and_refused():
    lens, nodes, ps = [30, 50], [10, 12], [[0, 4, 9], [1, 2, 3, 11]]
    rng = random.Random(3)
    table, _ = tables_for(lens, 20, rng)
    with Bytes("fp8", 2, 128, 20) as m:
        args = [i32(np.cumsum([0] + nodes)), i32(padded(ps, 5)), i32([3, 4]), i32(table), i32(lens)]
        out = torch.zeros(2, dtype=torch.int32, device="cuda")
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            pkv.paged_tree_commit(m.pool, *args, new_lens=out)
        for _ in range(2):  # every replay moves what is there then
            graph.replay()
            for b, p in enumerate(ps):
                move(m, table[b], lens[b] - nodes[b], p)
            m.check()
        assert out.tolist() == [23, 42]
        s = torch.cuda.Stream()
        torch.cuda.synchronize()
        got = pkv.paged_tree_commit(m.pool, *args, stream=s)
        s.synchronize()
        for b, p in enumerate(ps):
            move(m, table[b], lens[b] - nodes[b], p)
        m.check()
        assert got.tolist() == [23, 42]
        with pytest.raises(pkv.PagedKVError):
            pkv.paged_tree_commit(m.pool, *args, new_lens=args[4])
        with pytest.raises(pkv.PagedKVError):
            pkv.paged_tree_commit(m.pool, *args, new_lens=args[1].view(-1)[3:5])
        with pytest.raises(ValueError):
            pkv.paged_tree_commit(m.pool, args[0], args[1].long(), *args[2:])
        with pytest.raises(ValueError):
            pkv.paged_tree_commit(m.pool, args[0][:2], *args[1:])
        with pytest.raises(ValueError):
            pkv.paged_tree_commit(m.pool, *args[:4], args[4].cpu())
        none = pkv.paged_tree_commit(m.pool, i32([0]), i32(np.zeros((0, 3))), i32([]), i32(np.zeros((0, 4))), i32([]))
        assert none.shape == (0,)
        m.check()


# ------------------------------------------------------------------ beams

def reorder(m, parents, table, lens, spare, beams):
    """The tables, lengths and bytes that come out, one beam after the other."""
    W = table.shape[1]
    out, after, n = [], [], 0
    before = [h.clone() for h in m.host]
    for b, row in enumerate(parents):
        seen = set()
        for p in row:
            if p < 0:
                out.append([-1] * W)
                after.append(0)
                n += 1
                continue
            r = b * beams + p
            c = int(lens[r])
            here = c // BS
            entry = [int(x) if e <= here else -1 for e, x in enumerate(table[r])]
            if p in seen and here < W:
                for h, old in zip(m.host, before):
                    h[int(spare[n]), :, :c % BS] = old[entry[here], :, :c % BS] if c % BS else h[int(spare[n]), :, :0]
                entry[here] = int(spare[n])
            seen.add(p)
            out.append(entry)
            after.append(c)
            n += 1
    return out, after


def beam_case(batch, beams, k, hi, seed, extra):
    rng = random.Random(seed)
    lens = [rng.choice([0, 1, 15, 16, 17, 32, hi, rng.randrange(hi + 1)]) for _ in range(batch * beams)]
    need = [c + 1 for c in lens] if extra else lens
    blocks = sum((c + BS) // BS for c in need) + batch * k + 2
    table, free = tables_for(need, blocks, rng, 0)
    if not table.shape[1]:
        table = np.full((batch * beams, 1), -1, np.int32)
    parents = [[rng.choice([-1] + [rng.randrange(beams)] * 6) for _ in range(k)] for _ in range(batch)]
    return lens, table, parents, free[:batch * k], blocks


@pytest.mark.gpu
@pytest.mark.parametrize("kv", ["bf16", "fp8", "int4"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("batch,beams,k,n_kv,extra", [(1, 1, 1, 1, True), (3, 4, 4, 2, True), (5, 2, 7, 8, True), (2, 9, 3, 3, False),
                                                     (7, 64, 64, 1, True), (2, 3, 130, 2, True)])
def test_reorder_gives_each_beam_its_cache(kv, d, batch, beams, k, n_kv, extra):
    """Without `extra`, tables end with the last filled block: full tables have no block to write."""
    lens, table, parents, spare, blocks = beam_case(batch, beams, k, 200, batch * 7 + k, extra)
    with Bytes(kv, n_kv, d, blocks) as m:
        got, after = pkv.paged_beam_reorder(m.pool, i32(parents), i32(table), i32(lens), i32(spare))
        want, wlens = reorder(m, parents, table, lens, spare, beams)
        m.check()
        assert got.tolist() == want and after.tolist() == wlens
        assert m.pool.get_error() == 0


@pytest.mark.gpu
def test_reorder_reports_what_is_out_of_range():
    table = np.array([[0, 1, 2], [3, 4, -1]], np.int32)
    with Bytes("bf16", 2, 64, 12) as m:
        call = lambda parents, lens, spare=(8, 9, 10), t=table: pkv.paged_beam_reorder(m.pool, i32([parents]), i32(t), i32(lens), i32(spare))  # noqa: E731
        tab, ln = call([2, 0, -5], [20, 20])
        assert tab.tolist() == [[-1] * 3, [0, 1, -1], [-1] * 3] and ln.tolist() == [0, 20, 0]
        assert m.pool.get_error(clear=True) == pkv.DEVERR_BLOCK_RANGE
        tab, ln = call([0, 1, 1], [49, -3])
        assert ln.tolist() == [48, 0, 0] and tab.tolist() == [[0, 1, 2], [3, -1, -1], [9 + 1, -1, -1]]
        assert m.pool.get_error(clear=True) == pkv.DEVERR_CTX_RANGE
        tab, ln = call([0, 0, 0], [20, 20], spare=(8, 12, -1))  # spare blocks outside the pool: nothing copied
        assert tab.tolist() == [[0, 1, -1], [0, 12, -1], [0, -1, -1]]
        assert m.pool.get_error(clear=True) == pkv.DEVERR_BLOCK_RANGE
        t = table.copy()
        t[0, 1] = 77
        call([0, 0, 1], [20, 20], t=t)  # a source outside the pool
        assert m.pool.get_error(clear=True) == pkv.DEVERR_BLOCK_RANGE
        m.check()


@pytest.mark.gpu
def test_reorder_captured_on_another_stream_and_refused():
    lens, table, parents, spare, blocks = beam_case(4, 3, 3, 90, 5, True)
    with Bytes("int4", 2, 64, blocks) as m:
        args = [i32(parents), i32(table), i32(lens), i32(spare)]
        tab, ln = torch.zeros(12, table.shape[1], dtype=torch.int32, device="cuda"), torch.zeros(12, dtype=torch.int32, device="cuda")
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            pkv.paged_beam_reorder(m.pool, *args, tables_out=tab, lens_out=ln)
        want, wlens = reorder(m, parents, table, lens, spare, 3)
        for _ in range(2):
            graph.replay()
            m.check()
            assert tab.tolist() == want and ln.tolist() == wlens
        s = torch.cuda.Stream()
        got = pkv.paged_beam_reorder(m.pool, *args, stream=s)
        s.synchronize()
        assert got[0].tolist() == want and got[1].tolist() == wlens
        for bad in (dict(tables_out=args[1]), dict(lens_out=args[2]), dict(lens_out=tab.view(-1)[:12], tables_out=tab)):
            with pytest.raises(pkv.PagedKVError):
                pkv.paged_beam_reorder(m.pool, *args, **bad)
        with pytest.raises(ValueError):
            pkv.paged_beam_reorder(m.pool, args[0], args[1], args[2], args[3][:5])
        with pytest.raises(ValueError):
            pkv.paged_beam_reorder(m.pool, args[0], args[1][:11], args[2][:11], args[3])
        with pytest.raises(TypeError):
            pkv.paged_beam_reorder(m.pool, args[0].view(-1), *args[1:])
        m.check()
