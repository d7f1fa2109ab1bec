"""Cases of the rotary cache write, the cache read-back and differential attention.

Each case is one call (or, where the name says so, a write followed by the
read of what it wrote) on a paged key/value cache: 16-token blocks, block
tables in random order, bf16, E4M3 (fp32 scale per KV head) or 4-bit storage
(keys: scale and zero point per KV head and channel; values: per row).

``own`` chooses what ``run`` computes with: the plain torch form (false) or
this package's calls (true).
"""
import math
import random

import torch

own = False

BLOCK = 16
LAMBDA_INIT = 0.6
EPS = 1e-5


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one decode step of 64 sequences: every sequence's new token is rotated and written (latency)
        {"name": "write_step_bf16", "op": "write", "kv": "bf16", "batch": 64, "lo": 1, "hi": 1, "start": 1500,
         "n_q": 32, "n_kv": 8, "d": 128, "rot": 128, "axes": 1, "inter": False},
        # prompts with images: time, height and width positions, an E4M3 cache, ragged prompt lengths
        {"name": "write_prompt_image_fp8", "op": "write", "kv": "fp8", "batch": 12, "lo": 700, "hi": 2731,
         "start": 0, "n_q": 32, "n_kv": 8, "d": 128, "rot": 128, "axes": 3, "inter": False},
        # prompt chunks quantised to 4 bits as they are written, then read back as the model will see them;
        # half of each head rotated, adjacent pairs
        {"name": "write_read_int4", "op": "write_read", "kv": "int4", "batch": 9, "lo": 301, "hi": 1999,
         "start": 37, "n_q": 16, "n_kv": 4, "d": 128, "rot": 64, "axes": 1, "inter": True},
        # a few short sequences read back from a bf16 cache (latency)
        {"name": "read_small_bf16", "op": "read", "kv": "bf16", "batch": 4, "lo": 1, "hi": 257, "start": 0,
         "n_kv": 2, "d": 64},
        # a batch's whole E4M3 cache read back to bf16, lengths 1024..4096
        {"name": "read_batch_fp8", "op": "read", "kv": "fp8", "batch": 64, "lo": 1024, "hi": 4096, "start": 0,
         "n_kv": 8, "d": 128},
        # one short conversation, small heads (latency)
        {"name": "decode_one_short", "op": "diff", "kv": "bf16", "batch": 1, "lo": 300, "hi": 300, "chunk_lo": 1,
         "chunk_hi": 1, "n_q": 8, "n_kv": 2, "d": 64},
        # a decode step of 64 sequences of 1024..2048 tokens
        {"name": "decode_b64", "op": "diff", "kv": "bf16", "batch": 64, "lo": 1024, "hi": 2048, "chunk_lo": 1,
         "chunk_hi": 1, "n_q": 32, "n_kv": 8, "d": 128},
        # long contexts, 8 query heads on each KV head: 2 GiB of cache read in a step
        {"name": "decode_long_b16", "op": "diff", "kv": "bf16", "batch": 16, "lo": 32768, "hi": 32768,
         "chunk_lo": 1, "chunk_hi": 1, "n_q": 64, "n_kv": 8, "d": 128},
        # many sequences of very unequal lengths on an E4M3 cache
        {"name": "decode_b256_fp8", "op": "diff", "kv": "fp8", "batch": 256, "lo": 16, "hi": 4096, "chunk_lo": 1,
         "chunk_hi": 1, "n_q": 32, "n_kv": 8, "d": 128},
        # short chunks (drafted tokens under check) on top of cached contexts
        {"name": "chunk_draft_b16", "op": "diff", "kv": "bf16", "batch": 16, "lo": 900, "hi": 2000, "chunk_lo": 1,
         "chunk_hi": 9, "n_q": 32, "n_kv": 8, "d": 128},
        # prompt chunks of 16 sequences, up to 1024 tokens each over contexts of up to 2048
        {"name": "chunk_prompt_b16", "op": "diff", "kv": "bf16", "batch": 16, "lo": 1100, "hi": 2048,
         "chunk_lo": 700, "chunk_hi": 1024, "n_q": 32, "n_kv": 8, "d": 128},
        # whole prompts of odd lengths, small heads, an E4M3 cache
        {"name": "chunk_prompt_d64_fp8", "op": "diff", "kv": "fp8", "batch": 24, "lo": 129, "hi": 1023,
         "chunk_lo": 129, "chunk_hi": 1023, "n_q": 16, "n_kv": 8, "d": 64},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["write", "write_read", "read", "decode", "chunk"])
    kv = rng.choice(["bf16", "fp8"])
    n_kv = rng.choice([2, 4, 8])
    d = rng.choice([64, 128])
    g = rng.choice([1, 2, 4, 8])
    if op in ("write", "write_read"):
        hi = _log(rng, 1, 2731)
        batch = _log(rng, 1, max(1, min(64, 24000 // hi)))
        return {"op": op, "kv": rng.choice(["bf16", "fp8", "int4"]) if op == "write_read" else kv, "batch": batch,
                "lo": max(1, hi // rng.choice([1, 2, 5])), "hi": hi, "start": rng.choice([0, 1, 15, 16, 100, 1500]),
                "n_q": n_kv * g, "n_kv": n_kv, "d": d, "rot": rng.choice([16, d // 2, d]), "axes": rng.choice([1, 3]),
                "inter": rng.random() < 0.5}
    if op == "read":
        hi = _log(rng, 1, 8192)
        batch = _log(rng, 1, max(1, min(128, 64 * 2560 // hi)))
        return {"op": op, "kv": rng.choice(["bf16", "fp8", "int4"]), "batch": batch, "lo": max(1, hi // 3), "hi": hi,
                "start": rng.choice([0, 1, 16, 33]), "n_kv": n_kv, "d": d}
    if op == "decode":
        hi = _log(rng, 1, 32768)
        batch = _log(rng, 1, max(1, min(256, 16 * 32768 // hi)))
        return {"op": "diff", "kv": kv, "batch": batch, "lo": max(1, hi // rng.choice([1, 2, 7, 100])), "hi": hi,
                "chunk_lo": 1, "chunk_hi": 1, "n_q": n_kv * g, "n_kv": n_kv, "d": d}
    hi = _log(rng, 2, 2048)
    chunk = _log(rng, 2, min(hi, 1024))
    batch = _log(rng, 1, max(1, min(32, 16 * 1024 * 2048 // (chunk * hi))))
    g = min(g, 4)
    return {"op": "diff", "kv": kv, "batch": batch, "lo": max(chunk, hi // 2), "hi": hi,
            "chunk_lo": max(1, chunk // rng.choice([1, 3])), "chunk_hi": chunk, "n_q": n_kv * g, "n_kv": n_kv, "d": d}


def _between(case, lo, hi, salt):
    """Lengths of the case's sequences: part of the case, the same for every seed."""
    r = random.Random("%s %s %s %s" % (case["batch"], lo, hi, salt))
    return [r.randint(lo, hi) for _ in range(case["batch"])]


def _shape(case):
    """(cache lengths, chunk lengths) of the case's sequences."""
    if case["op"] == "diff":
        lens = _between(case, case["lo"], case["hi"], "context")
        chunk = _between(case, case["chunk_lo"], case["chunk_hi"], "chunk")
        if (case["chunk_lo"], case["chunk_hi"]) == (case["lo"], case["hi"]):
            chunk = lens  # whole prompts
        return lens, [min(a, b) for a, b in zip(chunk, lens)]
    chunk = _between(case, case["lo"], case["hi"], "chunk")
    return [case["start"] + c for c in chunk], chunk


def _stored(case):
    """Bytes of one token's key and value of one KV head in the cache."""
    d = case["d"]
    return {"bf16": 4 * d, "fp8": 2 * d, "int4": d + 8}[case["kv"]]


def work(case):
    lens, chunk = _shape(case)
    rows, d, n_kv = sum(chunk), case["d"], case["n_kv"]
    stored = n_kv * _stored(case)
    if case["op"] == "read":
        return {"bytes": rows * (stored + n_kv * 4 * d), "flops": 2 * rows * n_kv * 2 * d if case["kv"] != "bf16" else 0}
    n_q = case["n_q"]
    if case["op"] in ("write", "write_read"):
        moved = rows * (4 * n_q * d + 4 * n_kv * d + stored + 4 * case["axes"] + 8)
        if case["op"] == "write_read":
            moved += rows * (stored + n_kv * 4 * d)
        return {"bytes": moved, "flops": 3 * rows * (n_q + n_kv) * case["rot"]}
    seen = sum(t * (c - t) + t * (t + 1) // 2 for c, t in zip(lens, chunk))  # (token, visible position) pairs
    return {"bytes": sum(lens) * stored + rows * 4 * n_q * d, "flops": seen * n_q * (2 * d + 4 * d)}


# ------------------------------------------------------------------ inputs

def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    host = torch.Generator().manual_seed(seed)
    lens, chunk = _shape(case)
    batch, n_kv, d, kv = case["batch"], case["n_kv"], case["d"], case["kv"]
    width = (max(lens) + BLOCK - 1) // BLOCK
    need = [(c + BLOCK - 1) // BLOCK for c in lens]
    blocks = sum(need) + 3
    order = torch.randperm(blocks, generator=host)
    tables = torch.full((batch, width), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        tables[b, :n] = order[at:at + n].to(torch.int32)
        at += n
    indptr = torch.tensor([0] + chunk).cumsum(0)
    s = {"op": case["op"], "kv": kv, "d": d, "n_kv": n_kv, "rows": int(indptr[-1]), "longest": max(chunk),
         "tables": tables.to(dev), "lens": torch.tensor(lens, dtype=torch.int32).to(dev),
         "indptr": indptr.to(torch.int32).to(dev), "decode": max(chunk) == 1 and case["op"] == "diff"}
    rows = s["rows"]
    shape = (blocks, n_kv, BLOCK, d)

    def normal(*size):
        return torch.randn(*size, generator=gen, device=dev, dtype=torch.float32)

    # the cache's parameters and what is stored in it
    if kv == "fp8":
        s["k_scale"], s["v_scale"] = ((5.5 + 0.5 * torch.rand(n_kv, generator=gen, device=dev)) / 448 for _ in range(2))
    if kv == "int4":
        s["k_scale"] = (normal(n_kv, d).abs() + 5.0) / 15
        s["k_zero"] = -7.5 * s["k_scale"] + 0.1 * normal(n_kv, d)
    if case["op"] in ("write", "write_read"):
        dt = {"bf16": torch.bfloat16, "fp8": torch.float8_e4m3fn, "int4": torch.uint8}[kv]
        s["k"], s["v"] = (torch.zeros(*shape[:3], d // 2 if kv == "int4" else d, dtype=dt, device=dev) for _ in range(2))
        if kv == "int4":
            s["v_params"] = torch.zeros(*shape[:3], 2, device=dev)
    elif kv == "bf16":
        s["k"], s["v"] = (torch.randn(*shape, generator=gen, device=dev, dtype=torch.bfloat16) for _ in range(2))
    elif kv == "fp8":
        s["k"], s["v"] = ((normal(*shape) / s[n].view(1, n_kv, 1, 1)).clamp(-448, 448).to(torch.float8_e4m3fn)
                          for n in ("k_scale", "v_scale"))
    else:
        s["k"], s["v"] = (torch.randint(0, 256, (*shape[:3], d // 2), generator=gen, device=dev, dtype=torch.uint8)
                          for _ in range(2))
        s["v_params"] = torch.stack(((normal(*shape[:3]).abs() + 4.0) / 15, normal(*shape[:3]) - 2.5), dim=-1)

    starts = torch.tensor([c - t for c, t in zip(lens, chunk)], dtype=torch.int32)
    s["starts"] = starts.to(dev)
    if case["op"] in ("write", "write_read"):
        owner = torch.repeat_interleave(torch.arange(batch), torch.tensor(chunk))
        pos = starts[owner] + torch.arange(rows) - indptr[owner]
        s["slots"] = (tables[owner, pos // BLOCK].to(torch.int64) * BLOCK + pos % BLOCK).to(dev)
        if case["axes"] == 1:
            positions = pos.view(1, rows)
        else:  # text in front, then an image's rows and columns
            side = 1 + torch.randint(8, 64, (1,), generator=host)
            positions = torch.stack((pos // 64, pos // side, pos % side))
        s["positions"] = positions.to(torch.int32).contiguous().to(dev)
        pairs = case["rot"] // 2
        s["inv_freq"] = 500000.0 ** (-torch.arange(pairs, dtype=torch.float64) / pairs)
        cut = [0] * pairs if case["axes"] == 1 else [0] * (pairs // 4) + [1] * ((pairs - pairs // 4) // 2)
        s["axis"] = torch.tensor(cut + [2] * (pairs - len(cut)))
        s["inter"] = case["inter"]
        s["q"] = torch.randn(rows, case["n_q"], d, generator=gen, device=dev, dtype=torch.bfloat16)
        s["k_new"], s["v_new"] = (torch.randn(rows, n_kv, d, generator=gen, device=dev, dtype=torch.bfloat16)
                                  for _ in range(2))
    elif case["op"] == "diff":
        s["q"] = torch.randn(rows, case["n_q"], d, generator=gen, device=dev, dtype=torch.bfloat16)
        s["scale"] = 1.0 / math.sqrt(d)
        s["lambdas"] = 0.1 * normal(4, d)
        s["weight"] = 1.0 + 0.1 * normal(2 * d)
    if own:
        _prepare_own(s, blocks)
    else:
        for n in ("inv_freq", "axis"):
            if n in s:
                s[n] = s[n].to(dev)
    return s


def _prepare_own(s, blocks):
    """The pool with the same contents, and the handles that a serving program keeps."""
    import gqa_decode_attention_paged_gb300 as pkv

    pool = pkv.kv_pool_create(blocks, BLOCK, s["n_kv"], s["d"], {"bf16": pkv.BF16, "fp8": pkv.FP8_E4M3, "int4": pkv.INT4}[s["kv"]])
    if s["kv"] == "fp8":
        pool.set_fp8_scales(s["k_scale"].cpu().numpy(), s["v_scale"].cpu().numpy())
    if s["kv"] == "int4":
        pool.set_int4_key_params(s["k_scale"].cpu().numpy(), s["k_zero"].cpu().numpy())
        if s["op"] == "read":
            pool.v_params_view().copy_(s["v_params"])
    if s["op"] not in ("write", "write_read"):
        pool.k_view().copy_(s["k"].view(torch.uint8))
        pool.v_view().copy_(s["v"].view(torch.uint8))
    s["pool"] = pool
    if s["op"] == "write":
        s["k"], s["v"] = pool.k_view().view(s["k"].dtype), pool.v_view().view(s["v"].dtype)
    else:
        del s["k"], s["v"]
    if "inv_freq" in s:
        s["rope"] = pkv.Rope(s["inv_freq"], pair_axis=s["axis"], interleaved=s["inter"])
    if "lambdas" in s:
        s["params"] = pkv.DiffParams(s["lambdas"], LAMBDA_INIT, norm_weight=s["weight"], eps=EPS)


# ------------------------------------------------------------------ one pass

def run(s):
    if own:
        return _run_own(s)
    if s["op"] == "read":
        return _plain_read(s)
    if s["op"] == "diff":
        return _plain_diff(s)
    q = _plain_write(s)
    if s["op"] == "write":
        return q, s["k"], s["v"]
    return (q, *_plain_read(s))


def _run_own(s):
    import gqa_decode_attention_paged_gb300 as pkv

    pool = s["pool"]
    if s["op"] == "diff":
        if s["decode"]:
            return pkv.paged_diff_decode_attention(pool, s["q"], s["tables"], s["lens"], s["scale"], s["params"])
        return pkv.paged_diff_prefill_attention(pool, s["q"], s["indptr"], s["tables"], s["lens"], s["scale"],
                                                s["params"])
    if s["op"] == "read":
        return pkv.paged_kv_gather(pool, s["indptr"], s["tables"], s["starts"], n_rows=s["rows"])
    q = pkv.paged_rope_append(pool, s["rope"], s["q"], s["k_new"], s["v_new"], s["positions"], s["slots"])
    if s["op"] == "write":
        return q, s["k"], s["v"]
    return (q, *pkv.paged_kv_gather(pool, s["indptr"], s["tables"], s["starts"], n_rows=s["rows"]))


def _rotate(x, cos, sin, inter):
    """x [rows, heads, d] in 32 bits; the first 2 * pairs values of each head are rotated."""
    r = 2 * cos.shape[-1]
    part, rest = x[..., :r], x[..., r:]
    a, b = (part[..., 0::2], part[..., 1::2]) if inter else (part[..., : r // 2], part[..., r // 2:])
    cos, sin = cos.unsqueeze(1), sin.unsqueeze(1)
    c, e = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack((c, e), dim=-1).flatten(-2) if inter else torch.cat((c, e), dim=-1)
    return torch.cat((turned, rest), dim=-1)


def _plain_write(s):
    angle = s["positions"].double()[s["axis"]].t() * s["inv_freq"]  # far positions: 64 bits
    cos, sin = angle.cos().float(), angle.sin().float()
    q = _rotate(s["q"].float(), cos, sin, s["inter"]).to(torch.bfloat16)
    k, v = _rotate(s["k_new"].float(), cos, sin, s["inter"]), s["v_new"].float()
    block, off = s["slots"] // BLOCK, s["slots"] % BLOCK
    if s["kv"] == "bf16":
        k, v = k.to(torch.bfloat16), v.to(torch.bfloat16)
    elif s["kv"] == "fp8":
        k, v = ((x / s[n].view(1, -1, 1)).clamp(-448, 448).to(torch.float8_e4m3fn)
                for x, n in ((k, "k_scale"), (v, "v_scale")))
    else:
        code = ((k - s["k_zero"]) / s["k_scale"]).round().clamp(0, 15).to(torch.uint8)
        k = code[..., 0::2] | (code[..., 1::2] << 4)
        zero = v.amin(-1, keepdim=True)
        step = (v.amax(-1, keepdim=True) - zero) / 15
        step = torch.where(step == 0, torch.ones_like(step), step)
        code = ((v - zero) / step).round().clamp(0, 15).to(torch.uint8)
        v = code[..., 0::2] | (code[..., 1::2] << 4)
        s["v_params"][block, :, off] = torch.cat((step, zero), dim=-1)
    if s["kv"] == "fp8":  # written as bytes: no indexed store of this type
        s["k"].view(torch.uint8)[block, :, off] = k.view(torch.uint8)
        s["v"].view(torch.uint8)[block, :, off] = v.view(torch.uint8)
    else:
        s["k"][block, :, off] = k
        s["v"][block, :, off] = v
    return q


def _widen(s, which, raw, at=None):
    """Stored rows [..., n_kv, 16 or none, d] of the keys or values as 32-bit numbers; 4-bit: `at` are the value rows' parameters."""
    if s["kv"] == "bf16":
        return raw.float()
    heads = (-1,) + (1,) * (raw.dim() - 1 - s["heads_dim"])
    if s["kv"] == "fp8":
        return raw.view(torch.float8_e4m3fn).float() * s[which + "_scale"].view(heads)
    code = torch.stack((raw & 15, raw >> 4), dim=-1).flatten(-2).float()
    if which == "v":
        return code * at[..., :1] + at[..., 1:]
    return code * s["k_scale"] + s["k_zero"]


def _plain_read(s):
    row = torch.arange(s["rows"], device=s["indptr"].device, dtype=torch.int32)
    owner = torch.searchsorted(s["indptr"], row, right=True) - 1
    pos = s["starts"][owner] + row - s["indptr"][owner]
    block, off = s["tables"][owner, pos // BLOCK].long(), (pos % BLOCK).long()
    t = {**s, "heads_dim": 1}
    raw = lambda x: (x.view(torch.uint8) if s["kv"] == "fp8" else x)[block, :, off]  # noqa: E731
    k = _widen(t, "k", raw(s["k"]))
    v = _widen(t, "v", raw(s["v"]), s["v_params"][block, :, off] if s["kv"] == "int4" else None)
    return k.to(torch.bfloat16), v.to(torch.bfloat16)


def _plain_diff(s):
    d, n_kv = s["d"], s["n_kv"]
    batch, width = s["tables"].shape
    n_q = s["q"].shape[1]
    pairs, group, length, most = n_kv // 2, n_q // n_kv, width * BLOCK, s["longest"]
    tables = s["tables"].clamp(min=0).long()
    t = {**s, "heads_dim": 2}
    raw = lambda x: (x.view(torch.uint8) if s["kv"] == "fp8" else x)[tables]  # noqa: E731
    k, v = (_widen(t, n, raw(s[n])).permute(0, 2, 1, 3, 4).reshape(batch, pairs, 2, length, d) for n in ("k", "v"))
    v = v.transpose(2, 3).reshape(batch, pairs, length, 2 * d)
    # the sequences' rows side by side: [batch, most, ...]
    count = s["indptr"][1:] - s["indptr"][:-1]
    i = torch.arange(most, device=count.device, dtype=torch.int32)
    at = (s["indptr"][:-1, None] + i).clamp(max=s["rows"] - 1).long()
    q = s["q"][at].float().view(batch, most, pairs, group, 2, d).permute(0, 2, 4, 3, 1, 5)
    q = q.reshape(batch, pairs, 2, group * most, d)
    score = (q @ k.transpose(-1, -2)).mul_(s["scale"])
    last = (s["lens"] - count)[:, None] + i  # the last position that a row sees
    hidden = torch.arange(length, device=count.device) > last[..., None]
    score.view(batch, pairs, 2, group, most, length).masked_fill_(hidden.view(batch, 1, 1, 1, most, length), -math.inf)
    p = score.sub_(score.amax(-1, keepdim=True)).exp_()
    total = p.sum(-1, keepdim=True)
    o = (p.view(batch, pairs, 2 * group * most, length) @ v).view(batch, pairs, 2, group, most, 2 * d)
    o = o / total.view(batch, pairs, 2, group, most, 1)
    dots = (s["lambdas"][0] * s["lambdas"][1]).sum().exp() - (s["lambdas"][2] * s["lambdas"][3]).sum().exp()
    x = o[:, :, 0] - (dots + LAMBDA_INIT) * o[:, :, 1]
    x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * s["weight"] * (1.0 - LAMBDA_INIT)
    x = x.permute(0, 3, 1, 2, 4).reshape(batch, most, pairs * group, 2 * d)
    row = torch.arange(s["rows"], device=count.device, dtype=torch.int32)
    owner = torch.searchsorted(s["indptr"], row, right=True) - 1
    return x[owner, (row - s["indptr"][owner]).long()].to(torch.bfloat16)


# ------------------------------------------------------------------ 64 bits

def exact(case, seed):
    global own
    kept, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = kept
    if case["op"] == "diff":
        return _exact_diff(s)
    if case["op"] == "read":
        return _exact_rows(s)
    rows = s["rows"]
    turn = torch.empty(rows, len(s["axis"]), dtype=torch.float64, device="cuda")
    for i, (f, a) in enumerate(zip(s["inv_freq"].tolist(), s["axis"].tolist())):
        turn[:, i] = s["positions"][a].double() * f
    whirl = torch.polar(torch.ones_like(turn), turn).unsqueeze(1)
    n = turn.shape[1]

    def turned(x):
        x = x.double()
        out = x.clone()
        first = slice(0, 2 * n, 2) if s["inter"] else slice(0, n)
        second = slice(1, 2 * n, 2) if s["inter"] else slice(n, 2 * n)
        z = torch.complex(x[..., first].contiguous(), x[..., second].contiguous()) * whirl
        out[..., first], out[..., second] = z.real, z.imag
        return out

    q, k, v = turned(s["q"]), turned(s["k_new"]), s["v_new"].double()
    if case["kv"] == "fp8":
        k, v = (x / s[m].double().view(1, -1, 1) for x, m in ((k, "k_scale"), (v, "v_scale")))
        if case["op"] == "write":
            k, v = (x.clamp(-448, 448).float().to(torch.float8_e4m3fn).double() for x in (k, v))
        else:
            k, v = (x.clamp(-448, 448).float().to(torch.float8_e4m3fn).double() * s[m].double().view(1, -1, 1)
                    for x, m in ((k, "k_scale"), (v, "v_scale")))
    if case["kv"] == "int4":
        step, zero = s["k_scale"].double(), s["k_zero"].double()
        k = ((k - zero) / step).round().clamp(0, 15) * step + zero
        # a value row's step is stored in 32 bits and its codes are by definition 32-bit divisions by it (values
        # of 16 bits meet the border between two codes exactly); from there on 64 bits
        v = v.float()
        low, high = v.aminmax(dim=-1, keepdim=True)
        step = (high - low) / 15
        step[step == 0] = 1
        v = ((v - low) / step).round().clamp(0, 15).double() * step.double() + low.double()
    if case["op"] == "write_read":
        return q, k, v
    out = [q]
    for x in (k, v):
        pool = torch.zeros(s["k"].shape[0] * BLOCK, s["n_kv"], s["d"], dtype=torch.float64, device="cuda")
        pool[s["slots"]] = x
        out.append(pool.view(-1, BLOCK, s["n_kv"], s["d"]).transpose(1, 2).contiguous())
    return tuple(out)


def _exact_cache(s, b, first, last):
    """Keys and values [n_kv, positions, d] in 64 bits of sequence b's positions first .. last - 1."""
    blocks = s["tables"][b, : (last + BLOCK - 1) // BLOCK].long()
    got = []
    for n in ("k", "v"):
        x = s[n].view(torch.uint8)[blocks].view(s[n].dtype).transpose(0, 1).flatten(1, 2)[:, first:last]
        if s["kv"] == "int4":
            x = torch.stack((x % 16, x // 16), dim=-1).flatten(-2).double()
            if n == "k":
                x = x * s["k_scale"].double()[:, None] + s["k_zero"].double()[:, None]
            else:
                par = s["v_params"][blocks].transpose(0, 1).flatten(1, 2)[:, first:last].double()
                x = x * par[..., :1] + par[..., 1:]
        elif s["kv"] == "fp8":
            x = x.float().double() * s[n + "_scale"].double()[:, None, None]
        got.append(x.double())
    return got


def _exact_rows(s):
    k_rows, v_rows = [], []
    count = s["indptr"].diff().tolist()
    for b, (first, n) in enumerate(zip(s["starts"].tolist(), count)):
        k, v = _exact_cache(s, b, first, first + n)
        k_rows.append(k.transpose(0, 1))
        v_rows.append(v.transpose(0, 1))
    return torch.cat(k_rows), torch.cat(v_rows)


def _exact_diff(s):
    d, n_q, n_kv = s["d"], s["q"].shape[1], s["n_kv"]
    group = n_q // n_kv
    a = s["lambdas"].double()
    lam = math.exp(float(a[0] @ a[1])) - math.exp(float(a[2] @ a[3])) + LAMBDA_INIT
    out = torch.empty(s["rows"], n_q // 2, 2 * d, dtype=torch.float64, device="cuda")
    ends = s["indptr"].tolist()
    for b, c in enumerate(s["lens"].tolist()):
        lo, hi = ends[b], ends[b + 1]
        t = hi - lo
        k, v = _exact_cache(s, b, 0, c)
        see = torch.ones(t, c, dtype=torch.bool, device="cuda").tril(c - t)
        for h in range(n_q // 2):
            p = h // group
            values = torch.cat((v[2 * p], v[2 * p + 1]), dim=-1)
            maps = []
            for m in (0, 1):
                z = s["q"][lo:hi, 2 * h + m].double() @ k[2 * p + m].t() * s["scale"]
                maps.append(torch.softmax(z.masked_fill(~see, -math.inf), dim=-1))
            x = (maps[0] - lam * maps[1]) @ values
            x = x / (x.square().mean(-1, keepdim=True) + EPS).sqrt()
            out[lo:hi, h] = x * s["weight"].double() * (1 - LAMBDA_INIT)
    return out
