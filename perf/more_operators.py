"""Cases of decoding with several candidates per sequence over a paged key/value cache.

A tree of drafted tokens: attention of the tree's nodes over the cache
(``tree``), and the move of an accepted path's rows to the front of the nodes
(``commit``).  Beam search: the selection over beams and vocabulary
(``select``), and the reordering of block tables with copies of the blocks
that are written next (``reorder``).  The cache has 16-token blocks, block
tables in random order, bf16, E4M3 (fp32 scale per KV head) or 4-bit storage
(codes of two channels a byte, a scale and zero point per value row), of which
``commit`` and ``reorder`` move rows as they are stored.

``own`` chooses what ``run`` computes with: the plain torch form (false) or
this package's calls (true).
"""
import math
import random

import torch

own = False

BLOCK = 16
WORD = 64  # nodes that a word of a node's mask stands for


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one short conversation, a few drafted tokens, small heads (latency)
        {"name": "tree_one_short", "op": "tree", "kv": "bf16", "batch": 1, "lo": 300, "hi": 300, "nodes_lo": 8,
         "nodes_hi": 8, "wide": 3, "n_q": 8, "n_kv": 2, "d": 64},
        # a step of 16 sequences, trees of 17..32 nodes
        {"name": "tree_b16", "op": "tree", "kv": "bf16", "batch": 16, "lo": 1024, "hi": 2048, "nodes_lo": 17,
         "nodes_hi": 32, "wide": 5, "n_q": 32, "n_kv": 8, "d": 128},
        # long contexts, 8 query heads on each KV head, trees of 64 nodes
        {"name": "tree_long_b16", "op": "tree", "kv": "bf16", "batch": 16, "lo": 32768, "hi": 32768, "nodes_lo": 64,
         "nodes_hi": 64, "wide": 8, "n_q": 64, "n_kv": 8, "d": 128},
        # one long context whose few rows have to keep the whole card busy
        {"name": "tree_one_long", "op": "tree", "kv": "bf16", "batch": 1, "lo": 32768, "hi": 32768, "nodes_lo": 26,
         "nodes_hi": 26, "wide": 4, "n_q": 32, "n_kv": 8, "d": 128},
        # many sequences of very unequal lengths and trees on an E4M3 cache
        {"name": "tree_b64_fp8", "op": "tree", "kv": "fp8", "batch": 64, "lo": 60, "hi": 4096, "nodes_lo": 1,
         "nodes_hi": 60, "wide": 6, "n_q": 32, "n_kv": 8, "d": 128},
        # 64 sequences' accepted paths moved to the front of their trees
        {"name": "commit_b64", "op": "commit", "kv": "bf16", "batch": 64, "lo": 40, "hi": 300, "nodes_lo": 32,
         "nodes_hi": 32, "wide": 9, "n_kv": 8, "d": 128},
        # the same on a 4-bit cache: ragged trees, many sequences
        {"name": "commit_b200_int4", "op": "commit", "kv": "int4", "batch": 200, "lo": 64, "hi": 200, "nodes_lo": 3,
         "nodes_hi": 63, "wide": 20, "n_kv": 4, "d": 128},
        # the first step of one search: all but one beam are dead, some tokens are forbidden (latency)
        {"name": "select_one_first", "op": "select", "type": "bf16", "batch": 1, "beams": 4, "vocab": 32000, "k": 8,
         "first": True, "banned": 3},
        # a step of 64 searches over a large vocabulary
        {"name": "select_b64", "op": "select", "type": "bf16", "batch": 64, "beams": 4, "vocab": 128256, "k": 8,
         "first": False, "banned": 0},
        # wide beams, fp32 logits of an odd vocabulary
        {"name": "select_b32_f32", "op": "select", "type": "f32", "batch": 32, "beams": 10, "vocab": 100277, "k": 20,
         "first": False, "banned": 17},
        # four small searches (latency)
        {"name": "reorder_b4", "op": "reorder", "kv": "bf16", "batch": 4, "beams": 4, "k": 4, "lo": 20, "hi": 500,
         "n_kv": 2, "d": 64},
        # 64 searches of 8 beams with long tables
        {"name": "reorder_b64", "op": "reorder", "kv": "bf16", "batch": 64, "beams": 8, "k": 8, "lo": 1000,
         "hi": 4096, "n_kv": 8, "d": 128},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["tree", "tree", "commit", "select", "reorder"])
    n_kv = rng.choice([1, 2, 4, 8])
    d = rng.choice([64, 128])
    if op == "tree":
        g = rng.choice([1, 2, 4, 8])
        nodes = _log(rng, 1, 200)
        hi = max(nodes, _log(rng, 16, 32768))
        most = min(16 * 32768 // hi, 2 ** 31 // (n_kv * g * nodes * hi))
        return {"op": op, "kv": rng.choice(["bf16", "fp8"]), "batch": _log(rng, 1, max(1, min(128, most))),
                "lo": max(nodes, hi // rng.choice([1, 2, 9])), "hi": hi, "nodes_lo": max(1, nodes // rng.choice([1, 3])),
                "nodes_hi": nodes, "wide": rng.randint(1, 9), "n_q": n_kv * g, "n_kv": n_kv, "d": d}
    if op == "commit":
        nodes = _log(rng, 1, 200)
        hi = nodes + _log(rng, 1, 300)
        return {"op": op, "kv": rng.choice(["bf16", "fp8", "int4"]), "batch": _log(rng, 1, 256),
                "lo": max(nodes, hi // 2), "hi": hi, "nodes_lo": max(1, nodes // rng.choice([1, 4])),
                "nodes_hi": nodes, "wide": _log(rng, 1, 40), "n_kv": n_kv, "d": d}
    if op == "select":
        kind = rng.choice(["bf16", "f32"])
        vocab = _log(rng, 300, 160000)
        beams = rng.randint(1, 16)
        k = min(64, beams * rng.choice([1, 2]) + rng.choice([0, 0, 1]))
        batch = _log(rng, 1, max(1, min(128, 2 ** 25 // (vocab * beams))))
        return {"op": op, "type": kind, "batch": batch, "beams": beams, "vocab": vocab, "k": k,
                "first": rng.random() < 0.25, "banned": rng.choice([0, 5, vocab // 3])}
    beams = rng.randint(1, 16)
    hi = _log(rng, 1, 4096)
    return {"op": op, "kv": rng.choice(["bf16", "fp8", "int4"]), "batch": _log(rng, 1, max(1, min(64, 2 ** 20 // (beams * hi)))),
            "beams": beams, "k": rng.choice([beams, beams, 2 * beams]), "lo": max(1, hi // rng.choice([1, 2, 8])),
            "hi": hi, "n_kv": n_kv, "d": d}


def _between(case, n, lo, hi, salt):
    """Lengths of the case: part of it, the same for every seed."""
    r = random.Random("%s %s %s %s" % (n, lo, hi, salt))
    return [r.randint(lo, hi) for _ in range(n)]


def _shape(case):
    """(cache lengths, nodes) of the case's sequences; the nodes are the last entries of the cache."""
    lens = _between(case, case["batch"], case["lo"], case["hi"], "context")
    nodes = _between(case, case["batch"], case["nodes_lo"], case["nodes_hi"], "nodes")
    return lens, [min(a, b) for a, b in zip(nodes, lens)]


def _trees(case):
    """Per sequence each node's parent (-1: the context) and an accepted path from the root: part of the case.
    No path's rows move to where others of its rows come from, so that a pass can be repeated."""
    _, nodes = _shape(case)
    r = random.Random("%s %s trees" % (case["batch"], case["wide"]))
    trees = []
    for t in nodes:
        parent = [-1] + [max(0, i - r.randint(1, case["wide"])) for i in range(1, t)]
        at, path = r.randrange(t), []
        while at >= 0:
            path.append(at)
            at = parent[at]
        path.reverse()
        while _moved(path) & {i for i, j in enumerate(path) if i != j}:
            path.pop()
        trees.append((parent, path))
    return trees


def _moved(path):
    """The nodes of an accepted path whose rows move."""
    return {j for i, j in enumerate(path) if i != j}


def _masks(parent):
    """The nodes that each node sees, as the bits of a number: its ancestors and itself."""
    bits = []
    for i, p in enumerate(parent):
        bits.append((bits[p] if p >= 0 else 0) | 1 << i)
    return bits


def _parents(case):
    """Reordering: the beams that the new ones go on from.  Good beams have several children, others none."""
    r = random.Random("%s %s %s parents" % (case["batch"], case["beams"], case["k"]))
    return [[min(r.randrange(case["beams"]), r.randrange(case["beams"])) for _ in range(case["k"])]
            for _ in range(case["batch"])]


def _stored(case):
    """Bytes of one token's key and value of one KV head in the cache."""
    d = case["d"]
    return {"bf16": 4 * d, "fp8": 2 * d, "int4": d + 8}[case["kv"]]


def work(case):
    if case["op"] == "select":
        rows = case["batch"] * case["beams"]
        size = {"bf16": 2, "f32": 4}[case["type"]]
        return {"bytes": rows * (case["vocab"] * size + 4) + case["batch"] * case["k"] * 12,
                "flops": 4 * rows * case["vocab"]}
    row = case["n_kv"] * _stored(case)
    if case["op"] == "reorder":
        beams, lens = case["beams"], _between(case, case["batch"] * case["beams"], case["lo"], case["hi"], "context")
        moved = 0
        for b, parents in enumerate(_parents(case)):
            for i, p in enumerate(parents):
                n = lens[b * beams + p]
                moved += 8 * (n // BLOCK + 1) + 16
                if p in parents[:i]:
                    moved += 2 * (n % BLOCK) * row
        return {"bytes": moved, "flops": 0}
    lens, nodes = _shape(case)
    rows = sum(nodes)
    if case["op"] == "commit":
        trees = _trees(case)
        return {"bytes": sum(2 * row * len(_moved(path)) + 4 * len(path) for _, path in trees) + 16 * len(trees),
                "flops": 0}
    n_q, d = case["n_q"], case["d"]
    seen = sum(t * (c - t) for c, t in zip(lens, nodes))  # (node, visible position) pairs
    seen += sum(bin(m).count("1") for parent, _ in _trees(case) for m in _masks(parent))
    words = (max(nodes) + WORD - 1) // WORD
    return {"bytes": sum(lens) * row + rows * (4 * n_q * d + 8 * words), "flops": seen * n_q * 4 * d}


# ------------------------------------------------------------------ inputs

def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    host = torch.Generator().manual_seed(seed)
    if case["op"] == "select":
        return _prepare_select(case, gen)
    batch, n_kv, d, kv = case["batch"], case["n_kv"], case["d"], case["kv"]
    s = {"op": case["op"], "kv": kv, "d": d, "n_kv": n_kv}
    if case["op"] == "reorder":
        rows = batch * case["beams"]
        lens = _between(case, rows, case["lo"], case["hi"], "context")
        need = [c // BLOCK + 1 for c in lens]  # the block that the next token is written to among them
        spare = batch * case["k"]
        nodes = None
    else:
        rows = batch
        lens, nodes = _shape(case)
        need = [(c + BLOCK - 1) // BLOCK for c in lens]
        spare = 0
    width = max(need)
    blocks = sum(need) + spare + 3
    order = torch.randperm(blocks, generator=host).to(torch.int32)
    tables = torch.full((rows, width), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        tables[b, :n] = order[at:at + n]
        at += n
    s["tables"], s["lens"] = tables.cuda(), torch.tensor(lens, dtype=torch.int32).cuda()
    _fill(s, gen, blocks)
    if case["op"] == "reorder":
        s["spare"] = order[at:at + spare].cuda()
        s["parents"] = torch.tensor(_parents(case), dtype=torch.int32).cuda()
    else:
        total = sum(nodes)
        indptr = torch.tensor([0] + nodes).cumsum(0)
        s["rows"], s["longest"] = total, max(nodes)
        s["indptr"] = indptr.to(torch.int32).cuda()
        trees = _trees(case)
        if case["op"] == "tree":
            words = (max(nodes) + WORD - 1) // WORD
            bits = [m for parent, _ in trees for m in _masks(parent)]
            cut = [[(m >> (WORD * w)) & (2 ** WORD - 1) for w in range(words)] for m in bits]
            signed = [[w - 2 ** WORD if w >= 2 ** (WORD - 1) else w for w in row] for row in cut]
            s["mask"] = torch.tensor(signed, dtype=torch.int64).cuda()
            s["q"] = torch.randn(total, case["n_q"], d, generator=gen, device="cuda", dtype=torch.bfloat16)
            s["scale"] = 1.0 / math.sqrt(d)
        else:
            most = max(len(path) for _, path in trees)
            s["accepted"] = torch.tensor([path + [-1] * (most - len(path)) for _, path in trees],
                                         dtype=torch.int32).cuda()
            s["count"] = torch.tensor([len(path) for _, path in trees], dtype=torch.int32).cuda()
    if own:
        _prepare_own(s, blocks)
    return s


def _fill(s, gen, blocks):
    """The cache's parameters and what is stored in it."""
    n_kv, d, kv = s["n_kv"], s["d"], s["kv"]
    shape = (blocks, n_kv, BLOCK, d)

    def normal(*size):
        return torch.randn(*size, generator=gen, device="cuda", dtype=torch.float32)

    if kv == "fp8":
        s["k_scale"], s["v_scale"] = ((5.5 + 0.5 * torch.rand(n_kv, generator=gen, device="cuda")) / 448 for _ in range(2))
        s["k"], s["v"] = ((normal(*shape) / s[n].view(1, n_kv, 1, 1)).clamp(-448, 448).to(torch.float8_e4m3fn)
                          for n in ("k_scale", "v_scale"))
    elif kv == "int4":
        s["k_scale"] = (normal(n_kv, d).abs() + 5.0) / 15
        s["k_zero"] = -7.5 * s["k_scale"] + 0.1 * normal(n_kv, d)
        s["k"], s["v"] = (torch.randint(0, 256, (*shape[:3], d // 2), generator=gen, device="cuda", dtype=torch.uint8)
                          for _ in range(2))
        s["v_params"] = torch.stack(((normal(*shape[:3]).abs() + 4.0) / 15, normal(*shape[:3]) - 2.5), dim=-1)
    else:
        s["k"], s["v"] = (torch.randn(*shape, generator=gen, device="cuda", dtype=torch.bfloat16) for _ in range(2))


def _prepare_own(s, blocks):
    """The pool with the same contents, as a serving program keeps it."""
    import gqa_decode_attention_paged_gb300 as pkv

    kinds = {"bf16": pkv.BF16, "fp8": pkv.FP8_E4M3, "int4": pkv.INT4}
    pool = pkv.kv_pool_create(blocks, BLOCK, s["n_kv"], s["d"], kinds[s["kv"]])
    if s["kv"] == "fp8":
        pool.set_fp8_scales(s["k_scale"].cpu().numpy(), s["v_scale"].cpu().numpy())
    if s["kv"] == "int4":
        pool.set_int4_key_params(s["k_scale"].cpu().numpy(), s["k_zero"].cpu().numpy())
        pool.v_params_view().copy_(s["v_params"])
        s["v_params"] = pool.v_params_view()
    pool.k_view().copy_(s["k"].view(torch.uint8))
    pool.v_view().copy_(s["v"].view(torch.uint8))
    s["pool"] = pool
    s["k"], s["v"] = pool.k_view().view(s["k"].dtype), pool.v_view().view(s["v"].dtype)


def _prepare_select(case, gen):
    batch, beams, vocab = case["batch"], case["beams"], case["vocab"]
    x = torch.randn(batch, beams, vocab, generator=gen, device="cuda")
    x = 2.5 * x  # a language model's logits: a few tokens stand out
    likely = torch.randint(0, vocab, (batch, beams, 12), generator=gen, device="cuda")
    x.scatter_add_(2, likely, 6.0 * torch.rand(batch, beams, 12, generator=gen, device="cuda"))
    if case["banned"]:
        banned = torch.randperm(vocab, generator=gen, device="cuda")[:case["banned"]]
        x[..., banned] = -math.inf
    if case["type"] == "bf16":
        x = x.to(torch.bfloat16)
    scores = -20.0 * torch.rand(batch, beams, generator=gen, device="cuda")
    scores = scores.sort(dim=-1, descending=True).values.contiguous()
    if case["first"]:
        scores[:, 0] = 0.0
        scores[:, 1:] = -math.inf
    s = {"op": "select", "logits": x, "scores": scores, "k": case["k"]}
    if own:
        import gqa_decode_attention_paged_gb300 as pkv

        s["pool"] = pkv.kv_pool_create(1, BLOCK, 1, 64, pkv.BF16)  # the cache whose beams are selected
    return s


# ------------------------------------------------------------------ one pass

def run(s):
    if own:
        return _run_own(s)
    return {"tree": _plain_tree, "commit": _plain_commit, "select": _plain_select, "reorder": _plain_reorder}[s["op"]](s)


def _run_own(s):
    import gqa_decode_attention_paged_gb300 as pkv

    pool = s["pool"]
    if s["op"] == "tree":
        return pkv.paged_tree_attention(pool, s["q"], s["indptr"], s["mask"], s["tables"], s["lens"], s["scale"])
    if s["op"] == "select":
        return pkv.paged_beam_select(pool, s["logits"], s["scores"], s["k"])
    if s["op"] == "commit":
        lens = pkv.paged_tree_commit(pool, s["indptr"], s["accepted"], s["count"], s["tables"], s["lens"])
        return (lens, *_contents(s))
    tables, lens = pkv.paged_beam_reorder(pool, s["parents"], s["tables"], s["lens"], s["spare"])
    return (tables, lens, *_contents(s))


def _contents(s):
    return (s["k"], s["v"], s["v_params"]) if s["kv"] == "int4" else (s["k"], s["v"])


def _raw(s):
    """The cache's arrays in types that can be indexed and written."""
    return [x.view(torch.uint8) if x.dtype == torch.float8_e4m3fn else x for x in _contents(s)]


def _plain_tree(s):
    d, n_kv = s["d"], s["n_kv"]
    batch, width = s["tables"].shape
    n_q = s["q"].shape[1]
    group, length, most = n_q // n_kv, width * BLOCK, s["longest"]
    tables = s["tables"].clamp(min=0).long()
    k, v = _raw(s)
    if s["kv"] == "fp8":
        k, v = (x[tables].view(torch.float8_e4m3fn).float() * s[n].view(-1, 1, 1) for x, n in ((k, "k_scale"), (v, "v_scale")))
    else:
        k, v = k[tables].float(), v[tables].float()
    k, v = (x.transpose(1, 2).reshape(batch, n_kv, length, d) for x in (k, v))
    # the sequences' rows side by side: [batch, n_kv, group * most, d]
    count = s["indptr"][1:] - s["indptr"][:-1]
    i = torch.arange(most, device="cuda", dtype=torch.int32)
    at = (s["indptr"][:-1, None] + i).clamp(max=s["rows"] - 1).long()
    q = s["q"][at].float().view(batch, most, n_kv, group, d).permute(0, 2, 3, 1, 4).reshape(batch, n_kv, group * most, d)
    score = (q @ k.transpose(-1, -2)).mul_(s["scale"])
    pos = torch.arange(length, device="cuda", dtype=torch.int32)
    node = pos - (s["lens"] - count)[:, None]  # [batch, length]: negative in the context
    bit = node.clamp(0, WORD * s["mask"].shape[1] - 1).long()
    word = s["mask"][at].gather(2, (bit // WORD)[:, None].expand(-1, most, -1))
    see = (word >> (bit % WORD)[:, None]) & 1 == 1
    see = (see | (node < 0)[:, None]) & (node < count[:, None])[:, None]
    score.view(batch, n_kv, group, most, length).masked_fill_(~see.view(batch, 1, 1, most, length), -math.inf)
    del see, word
    p = score.sub_(score.amax(-1, keepdim=True)).exp_()
    o = (p @ v) / p.sum(-1, keepdim=True)
    o = o.view(batch, n_kv, group, most, d).permute(0, 3, 1, 2, 4).reshape(batch, most, n_q, d)
    row = torch.arange(s["rows"], device="cuda", dtype=torch.int32)
    owner = torch.searchsorted(s["indptr"], row, right=True) - 1
    return o[owner, (row - s["indptr"][owner]).long()].to(torch.bfloat16)


def _plain_commit(s):
    count = s["indptr"][1:] - s["indptr"][:-1]
    first = (s["lens"] - count).long()
    batch, most = s["accepted"].shape
    i = torch.arange(most, device="cuda").expand(batch, most)
    live = i < s["count"][:, None]
    owner = torch.arange(batch, device="cuda")[:, None].expand(batch, most)[live]
    src, dst = (first[owner] + x[live] for x in (s["accepted"].long(), i))
    sb, db = s["tables"][owner, src // BLOCK].long(), s["tables"][owner, dst // BLOCK].long()
    for x in _raw(s):
        x[db, :, dst % BLOCK] = x[sb, :, src % BLOCK]
    return ((s["lens"] - count) + s["count"], *_contents(s))


def _plain_select(s):
    batch, beams, vocab = s["logits"].shape
    x = s["logits"].double()  # candidates of different beams meet within the last places of 32 bits
    top = x.amax(-1, keepdim=True)
    x -= (x - top).exp().sum(-1, keepdim=True).log() + top
    x += s["scores"].double()[..., None]
    best, at = x.view(batch, beams * vocab).sort(dim=-1, descending=True, stable=True)
    best, at = best[:, :s["k"]], at[:, :s["k"]]
    none = best == -math.inf
    token = torch.where(none, -1, at % vocab).to(torch.int32)
    parent = torch.where(none, -1, at // vocab).to(torch.int32)
    return token, parent, best.float()


def _plain_reorder(s):
    batch, k = s["parents"].shape
    rows, width = s["tables"].shape
    parent = s["parents"].long()
    earlier = torch.ones(k, k, device="cuda", dtype=torch.bool).tril(-1)
    other = ((parent[:, :, None] == parent[:, None]) & earlier).any(-1).view(-1)  # not its parent's first child
    src = (torch.arange(batch, device="cuda")[:, None] * (rows // batch) + parent).view(-1)
    lens = s["lens"][src]
    here = (lens // BLOCK).long()  # the entry that is written next
    entry = torch.arange(width, device="cuda")
    tables = torch.where(entry <= here[:, None], s["tables"][src], -1)
    fits = here < width
    old = tables.gather(1, here.clamp(max=width - 1)[:, None])
    tables = torch.where((entry == here[:, None]) & other[:, None], s["spare"].view(-1, 1), tables)
    off = torch.arange(BLOCK, device="cuda")
    copied = (off < (lens % BLOCK)[:, None]) & (other & fits)[:, None]
    n, o = copied.nonzero(as_tuple=True)
    for x in _raw(s):
        x[s["spare"][n].long(), :, o] = x[old[n, 0].long(), :, o]
    return (tables, lens, *_contents(s))


# ------------------------------------------------------------------ 64 bits

def exact(case, seed):
    global own
    kept, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = kept
    return {"tree": _exact_tree, "commit": _exact_commit, "select": _exact_select, "reorder": _exact_reorder}[s["op"]](s, case)


def _exact_tree(s, case):
    lens, nodes = _shape(case)
    d, n_q, n_kv = s["d"], case["n_q"], s["n_kv"]
    group = n_q // n_kv
    out = torch.empty(s["rows"], n_q, d, dtype=torch.float64, device="cuda")
    lo = 0
    for b, (c, t, (parent, _)) in enumerate(zip(lens, nodes, _trees(case))):
        ids = s["tables"][b, : (c + BLOCK - 1) // BLOCK].long()
        got = []
        for n in ("k", "v"):
            x = s[n].view(torch.uint8)[ids].view(s[n].dtype).transpose(0, 1).flatten(1, 2)[:, :c]
            x = x.float().double() if s["kv"] == "fp8" else x.double()
            got.append(x * s[n + "_scale"].double()[:, None, None] if s["kv"] == "fp8" else x)
        k, v = got
        family = torch.zeros(t, t, dtype=torch.bool)
        for i, p in enumerate(parent):
            if p >= 0:
                family[i] = family[p]
            family[i, i] = True
        see = torch.ones(t, c, dtype=torch.bool, device="cuda")
        see[:, c - t:] = family.cuda()
        for h in range(n_q):
            z = s["q"][lo:lo + t, h].double() @ k[h // group].t() * s["scale"]
            out[lo:lo + t, h] = torch.softmax(z.masked_fill(~see, -math.inf), dim=-1) @ v[h // group]
        lo += t
    return out


def _exact_commit(s, case):
    rows = [x.clone() for x in _contents(s)]
    flat = [x.view(torch.uint8) if x.dtype == torch.float8_e4m3fn else x for x in rows]
    tables = s["tables"].tolist()
    lens, nodes = _shape(case)
    after, at = [], []
    for b, (c, t, (_, path)) in enumerate(zip(lens, nodes, _trees(case))):
        for i, j in enumerate(path):
            src, dst = c - t + j, c - t + i
            at.append((tables[b][dst // BLOCK], dst % BLOCK, tables[b][src // BLOCK], src % BLOCK))
        after.append(c - t + len(path))
    db, do, sb, so = torch.tensor(at, dtype=torch.int64, device="cuda").t()
    for x in flat:
        x[db, :, do] = x[sb, :, so]  # (all are read before any is written)
    return (torch.tensor(after, dtype=torch.int32, device="cuda"), *rows)


def _exact_select(s, case):
    batch, beams, vocab = s["logits"].shape
    tokens, parents, best = (torch.full((batch, s["k"]), -1, dtype=t, device="cuda")
                             for t in (torch.int32, torch.int32, torch.float64))
    for b in range(batch):
        v = torch.log_softmax(s["logits"][b].double(), dim=-1) + s["scores"][b].double()[:, None]
        v = v.view(-1)
        for i in range(s["k"]):
            top = v.max()
            best[b, i] = top
            if float(top) == -math.inf:
                best[b, i:] = -math.inf
                break
            at = int((v == top).nonzero()[0])
            tokens[b, i], parents[b, i] = at % vocab, at // vocab
            v[at] = -math.inf
    return tokens, parents, best


def _exact_reorder(s, case):
    rows = [x.clone() for x in _contents(s)]
    flat = [x.view(torch.uint8) if x.dtype == torch.float8_e4m3fn else x for x in rows]
    old, lens, spare = s["tables"].tolist(), s["lens"].tolist(), s["spare"].tolist()
    tables, after, n = [], [], 0
    src, dst, off = [], [], []
    for b, parents in enumerate(_parents(case)):
        seen = set()
        for p in parents:
            row = b * case["beams"] + p
            c = lens[row]
            entry = list(old[row][:c // BLOCK + 1]) + [-1] * (len(old[row]) - c // BLOCK - 1)
            if p in seen:
                src += [entry[c // BLOCK]] * (c % BLOCK)
                dst += [spare[n]] * (c % BLOCK)
                off += list(range(c % BLOCK))
                entry[c // BLOCK] = spare[n]
            seen.add(p)
            tables.append(entry)
            after.append(c)
            n += 1
    src, dst, off = (torch.tensor(x, dtype=torch.int64, device="cuda") for x in (src, dst, off))
    for x in flat:
        x[dst, :, off] = x[src, :, off]
    return (torch.tensor(tables, dtype=torch.int32, device="cuda"), torch.tensor(after, dtype=torch.int32, device="cuda"),
            *rows)
