"""The operators between a block's projections: cases, plain forms, exact values.

A LittleBit block's query, key and value projections give one row a token; its output projection takes the
attention's.  Between the two a user needs

* ``rope``    the norm of each head of the queries and keys with the position rotation, in one pass, with its
              backward pass;
* ``append``  the same on the way into a paged cache of keys and values, which takes the values too;
* ``attend``  the attention over that cache, of single tokens, of prompts and of trees of drafted tokens (the
              projections take 2 to 16 tokens in one pass over the weights, which is what drafts are for);
* ``accept``  after a tree is verified, its accepted path moved together in the cache.

A cache holds pages of keys and of values, heads x slots x dim each; a sequence's keys lie in the pages that its
row of the table names.  The tokens of a call are the last of their sequences' keys.

``run`` computes them in plain torch operations, or with the package's kernels where ``own`` is true.
"""

import math
import random

import torch

own = False

_TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}
_EPS = 1e-5
_BASE = 10000.0


# --------------------------------------------------------------------------------------------------------- cases

def listed():
    return [
        # a short text of a training step: queries and keys of forty heads, normed by head and rotated, and back
        {"name": "rope_train_37x40x40x128_fp16", "op": "rope", "tokens": 37, "heads": 40, "kv_heads": 40, "dim": 128, "rot": 128,
         "norm": True, "interleaved": False, "type": "fp16"},
        # a long one with shared key heads
        {"name": "rope_train_4000x64x8x128_bf16", "op": "rope", "tokens": 4000, "heads": 64, "kv_heads": 8, "dim": 128, "rot": 128,
         "norm": True, "interleaved": False, "type": "bf16"},
        # one token of a decode step joins a cache
        {"name": "append_1x40x40x128_fp16", "op": "append", "seqs": 1, "tokens": 1, "cached": 2000, "heads": 40, "kv_heads": 40, "dim": 128,
         "rot": 128, "norm": False, "interleaved": False, "page": 64, "tree": False, "type": "fp16"},
        # a prompt joins it, behind a text that is there already
        {"name": "append_2039x64x8x128_bf16", "op": "append", "seqs": 1, "tokens": 2039, "cached": 301, "heads": 64, "kv_heads": 8, "dim": 128,
         "rot": 128, "norm": True, "interleaved": True, "page": 16, "tree": False, "type": "bf16"},
        # one token's attention over its own long text: the cache's bytes
        {"name": "attend_1x1_40x40x128_4000_fp16", "op": "attend", "seqs": 1, "tokens": 1, "cached": 4000, "heads": 40, "kv_heads": 40, "dim": 128,
         "page": 64, "tree": False, "type": "fp16"},
        # a served batch, one token of each of many texts of all lengths, shared key heads
        {"name": "attend_32x1_64x8x128_8000_bf16", "op": "attend", "seqs": 32, "tokens": 1, "cached": 8000, "heads": 64, "kv_heads": 8, "dim": 128,
         "page": 32, "tree": False, "type": "bf16"},
        # a tree of as many drafted tokens as the packed layers take in one pass
        {"name": "attend_tree_1x16_40x40x128_2000_fp16", "op": "attend", "seqs": 1, "tokens": 16, "cached": 2000, "heads": 40, "kv_heads": 40,
         "dim": 128, "page": 64, "tree": True, "type": "fp16"},
        # larger trees over long texts
        {"name": "attend_tree_4x61_64x8x128_30000_bf16", "op": "attend", "seqs": 4, "tokens": 61, "cached": 30000, "heads": 64, "kv_heads": 8,
         "dim": 128, "page": 64, "tree": True, "type": "bf16"},
        # prompts of different lengths from their first token on
        {"name": "attend_3x1500_32x32x128_0_fp16", "op": "attend", "seqs": 3, "tokens": 1500, "cached": 0, "heads": 32, "kv_heads": 32, "dim": 128,
         "page": 16, "tree": False, "type": "fp16"},
        # a long prompt's second half
        {"name": "attend_1x4000_64x8x128_4100_bf16", "op": "attend", "seqs": 1, "tokens": 4000, "cached": 4100, "heads": 64, "kv_heads": 8, "dim": 128,
         "page": 64, "tree": False, "type": "bf16"},
        # the accepted tokens of one tree
        {"name": "accept_1x16_40x128_fp16", "op": "accept", "seqs": 1, "tokens": 16, "cached": 2000, "kv_heads": 40, "dim": 128, "page": 64,
         "tree": True, "type": "fp16"},
        # of a served batch of trees
        {"name": "accept_48x61_40x128_bf16", "op": "accept", "seqs": 48, "tokens": 61, "cached": 500, "kv_heads": 40, "dim": 128, "page": 16,
         "tree": True, "type": "bf16"},
    ]


def _spread(rng, low, high):
    """A whole number between the two, spread over its logarithm."""
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(["rope", "append", "attend", "attend", "attend", "accept"])
    kv_heads = rng.choice([1, 2, 4, 5, 8, 16, 32, 40])
    group = rng.choice([1, 1, 2, 4, 5, 7, 8])
    while kv_heads * group > 64:
        group = rng.choice([1, 2, 4])
    dim = rng.choice([64, 80, 96, 128, 128, 128, 192, 256])
    c = {"op": op, "heads": kv_heads * group, "kv_heads": kv_heads, "dim": dim, "type": rng.choice(["fp16", "bf16"])}
    width = (c["heads"] + 2 * kv_heads) * dim
    if op in ("rope", "append"):
        c |= {"rot": rng.choice([dim, dim, dim // 2]), "norm": rng.random() < 0.5, "interleaved": rng.random() < 0.3}
    if op == "rope":
        return c | {"tokens": _spread(rng, 1, min(8000, 4000 * 80 * 128 // width))}
    c |= {"seqs": _spread(rng, 1, 64), "page": rng.choice([8, 16, 32, 64, 128]), "tree": False}
    if op == "append":
        c["tokens"] = rng.choice([1, rng.randint(2, 16), _spread(rng, 17, max(18, 2039 * 80 * 128 // (width * c["seqs"])))])
        return c | {"cached": _spread(rng, 1, 2000)}
    if op == "accept":
        del c["heads"]
        return c | {"tokens": rng.randint(2, 64), "cached": _spread(rng, 1, 1000), "tree": True, "seqs": min(48, c["seqs"])}
    kind = rng.choice(["one", "tree", "prompt"])
    if kind == "prompt":
        c["tokens"] = _spread(rng, 2, 4000)
        c["cached"] = rng.choice([0, _spread(rng, 1, 4000)])
        most = 64 * 4000 * 8100 // (c["heads"] * c["tokens"] * (c["tokens"] + c["cached"]) * max(1, dim // 128))
        return c | {"seqs": max(1, min(c["seqs"], most, 8))}
    c |= {"tokens": 1 if kind == "one" else rng.randint(2, 64), "tree": kind == "tree", "cached": _spread(rng, 1, 30000)}
    most = 4 * 30000 * 8 * 128 * (2 if kind == "one" else 1) // (c["cached"] * kv_heads * dim)
    return c | {"seqs": max(1, min(c["seqs"], most))}


def _counts(case):
    """(tokens, keys cached before them) of each sequence: the largest first, the others spread below it."""
    out = []
    for i in range(case["seqs"]):
        share = 1.0 if i == 0 else 1.0 - 0.9 * ((0.6180339887 * i) % 1.0)
        tokens = case["tokens"] if case["tokens"] == 1 else max(1, int(case["tokens"] * (0.5 + 0.5 * share)))
        out.append((tokens, int(case["cached"] * share)))
    return out


# -------------------------------------------------------------------------------------------------------- inputs

def _inv_freq(rot):
    return (_BASE ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)).float().cuda()


def _projected(g, tokens, heads, dim, t):
    """A projection's output seen as heads: channels of different size, a few tokens far larger than the others."""
    x = torch.randn(tokens, heads, dim, device="cuda", generator=g)
    x *= torch.exp(0.4 * torch.randn(heads, dim, device="cuda", generator=g))
    x *= torch.where(torch.rand(tokens, 1, 1, device="cuda", generator=g) < 0.02, 6.0, 1.0)
    return x.to(t)


def _trees(case, seed):
    """For each sequence of the batch: the parents of its drafted tokens (level by level, the likeliest child first) and
    an accepted path, from the root on."""
    rng = random.Random(seed)
    trees = []
    for tokens, _ in _counts(case):
        parents, level, width = [-1], [0], 1
        while len(parents) < tokens:
            width = rng.randint(max(2, width), 2 * width + 6)
            new = []
            for i in range(min(width, tokens - len(parents))):
                new.append(len(parents))
                parents.append(level[0] if i == 0 else rng.choice(level))
            level = new
        path = [tokens - 1] if rng.random() < 0.7 else [rng.randrange(tokens)]
        while parents[path[0]] >= 0:
            path.insert(0, parents[path[0]])
        # what is moved twice has to stay: a path is cut where it would read a place that it fills
        while any(p != j and p < len(path) for j, p in enumerate(path)):
            path.pop()
        trees.append((parents, path))
    return trees


def _batch(case, seed):
    """Where each sequence's rows begin, its keys with them, and its pages."""
    rng = random.Random(seed)
    counts = _counts(case)
    order = list(range(len(counts)))
    rng.shuffle(order)
    trees = _trees(case, seed) if case["tree"] else [None] * len(counts)
    counts, trees = [counts[i] for i in order], [trees[i] for i in order]
    starts = [0]
    for tokens, _ in counts:
        starts.append(starts[-1] + tokens)
    lens = [tokens + cached for tokens, cached in counts]
    columns = -(-max(lens) // case["page"])
    free = list(range(sum(-(-n // case["page"]) for n in lens) + 3))
    rng.shuffle(free)
    table = [[free.pop() if i * case["page"] < n else 0 for i in range(columns)] for n in lens]
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    s = {"starts": ints(starts), "lens": ints(lens), "table": ints(table), "rows": starts[-1], "longest": max(lens),
         "most": max(t for t, _ in counts), "pages": sum(-(-n // case["page"]) for n in lens) + 3, "trees": trees, "counts": counts}
    positions = []
    words = []
    for (tokens, cached), tree in zip(counts, trees):
        if tree is None:
            positions += [cached + i for i in range(tokens)]
            continue
        depth, seen = [0], [1]
        for i in range(1, tokens):
            depth.append(depth[tree[0][i]] + 1)
            seen.append(seen[tree[0][i]] | (1 << i))
        positions += [cached + d for d in depth]
        words += [w - (1 << 64) if w >> 63 else w for w in seen]
    s["positions"] = ints(positions)
    s["tree"] = torch.tensor(words, dtype=torch.int64, device="cuda") if case["tree"] else None
    return s


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    t, dim, s = _TYPES[case["type"]], case["dim"], dict(case)
    kv_heads = case["kv_heads"]
    weight = lambda: (0.5 + torch.rand(dim, device="cuda", generator=g)).to(t)  # noqa: E731
    if case["op"] in ("rope", "append"):
        s["inv_freq"] = _inv_freq(case["rot"])
        s["q_weight"] = weight() if case["norm"] else None
        s["k_weight"] = weight() if case["norm"] else None
    if case["op"] == "rope":
        tokens, heads = case["tokens"], case["heads"]
        first = random.Random(seed).randrange(1 << 16)  # a text of a packed batch, or one that goes on
        s["positions"] = torch.arange(first, first + tokens, dtype=torch.int32, device="cuda")
        s["q"], s["k"] = _projected(g, tokens, heads, dim, t), _projected(g, tokens, kv_heads, dim, t)
        s["dq"], s["dk"] = 0.1 * _projected(g, tokens, heads, dim, t), 0.1 * _projected(g, tokens, kv_heads, dim, t)
        return s
    s |= _batch(case, int(seed))
    # normal keys and values, which is what normed heads look like
    s["k_pages"] = torch.randn(s["pages"], kv_heads, case["page"], dim, device="cuda", generator=g).to(t)
    s["v_pages"] = torch.randn(s["pages"], kv_heads, case["page"], dim, device="cuda", generator=g).to(t)
    if case["op"] == "append":
        s["q"] = _projected(g, s["rows"], case["heads"], dim, t)
        s["k"] = _projected(g, s["rows"], kv_heads, dim, t)
        s["v"] = _projected(g, s["rows"], kv_heads, dim, t)
    elif case["op"] == "attend":
        s["q"] = (1.5 * torch.randn(s["rows"], case["heads"], dim, device="cuda", generator=g)).to(t)
    else:
        most = max(len(path) for _, path in s["trees"])
        s["path"] = torch.tensor([path + [-1] * (most - len(path)) for _, path in s["trees"]], dtype=torch.int32, device="cuda")
    return s


# --------------------------------------------------------------------------------------------------- plain forms

def _pairs(x, rot, interleaved):
    """The two halves of every rotated pair, and what is not rotated."""
    if interleaved:
        return x[..., 0:rot:2], x[..., 1:rot:2], x[..., rot:]
    return x[..., : rot // 2], x[..., rot // 2 : rot], x[..., rot:]


def _joined(a, b, rest, interleaved):
    both = torch.stack([a, b], -1).flatten(-2) if interleaved else torch.cat([a, b], -1)
    return torch.cat([both, rest], -1)


def _angles(s):
    angle = s["positions"].double()[:, None, None] * s["inv_freq"].double()  # far positions: 32 bits lose the turn
    return torch.cos(angle).float(), torch.sin(angle).float()


def _turned(x, s, cos, sin):
    a, b, rest = _pairs(x, s["rot"], s["interleaved"])
    return _joined(a * cos - b * sin, b * cos + a * sin, rest, s["interleaved"])


def _plain_rope(x, weight, s, cos, sin):
    y = x.float()
    if weight is not None:
        y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + _EPS) * weight.float()
    return _turned(y, s, cos, sin).to(x.dtype)


def _plain_rope_bwd(dy, x, weight, s, cos, sin):
    dz = _turned(dy.float(), s, cos, -sin)
    if weight is None:
        return dz.to(x.dtype), None
    h = x.float()
    rstd = torch.rsqrt((h * h).mean(-1, keepdim=True) + _EPS)
    xhat, du = h * rstd, dz * weight.float()
    dx = rstd * (du - xhat * (du * xhat).mean(-1, keepdim=True))
    return dx.to(x.dtype), (dz * xhat).sum((0, 1))


def _plain_train(s):
    cos, sin = _angles(s)
    out = {"q_out": _plain_rope(s["q"], s["q_weight"], s, cos, sin), "k_out": _plain_rope(s["k"], s["k_weight"], s, cos, sin)}
    out["dq_in"], out["dq_weight"] = _plain_rope_bwd(s["dq"], s["q"], s["q_weight"], s, cos, sin)
    out["dk_in"], out["dk_weight"] = _plain_rope_bwd(s["dk"], s["k"], s["k_weight"], s, cos, sin)
    return out


def _rows_of(s):
    """For each row of the call: its sequence, and which of that one's tokens it is."""
    row = torch.arange(s["rows"], device="cuda")
    seq = torch.searchsorted(s["starts"][1:].long(), row, right=True)
    return seq, row - s["starts"].long()[seq]


def _plain_append(s):
    cos, sin = _angles(s)
    seq, nth = _rows_of(s)
    at = s["lens"].long()[seq] - (s["starts"][1:] - s["starts"][:-1]).long()[seq] + nth
    page, slot = s["table"].long()[seq, at // s["page"]], at % s["page"]
    s["k_pages"][page, :, slot] = _plain_rope(s["k"], s["k_weight"], s, cos, sin)
    s["v_pages"][page, :, slot] = s["v"]
    return {"q_out": _plain_rope(s["q"], s["q_weight"], s, cos, sin), "k_pages": s["k_pages"], "v_pages": s["v_pages"]}


def _plain_attend(s):
    heads, kv_heads, dim, most = s["heads"], s["kv_heads"], s["dim"], s["most"]
    starts, lens = s["starts"].long(), s["lens"].long()
    key = torch.arange(s["longest"], device="cuda")
    page = s["table"].long()[:, key // s["page"]]
    slot = (key % s["page"]).expand_as(page)
    k = s["k_pages"][page, :, slot].float().permute(0, 2, 3, 1).contiguous()  # sequence, head, dim, key
    v = s["v_pages"][page, :, slot].float().permute(0, 2, 1, 3).contiguous()
    nth = torch.arange(most, device="cuda")
    count = starts[1:] - starts[:-1]
    row = (starts[:-1, None] + nth).clamp(max=s["rows"] - 1)
    q = s["q"][row].float().view(s["seqs"], most, kv_heads, heads // kv_heads, dim).permute(0, 2, 3, 1, 4)
    score = torch.matmul(q.reshape(s["seqs"], kv_heads, -1, dim), k).view(s["seqs"], kv_heads, -1, most, s["longest"])
    score *= 1.0 / math.sqrt(dim)
    drafted = key - (lens - count)[:, None]  # which of the call's tokens a key is: negative before them
    if s["tree"] is None:
        seen = drafted[:, None] <= nth[:, None]
    else:
        seen = (s["tree"][row][:, :, None] >> drafted.clamp(0, 63)[:, None]) & 1 == 1
        seen = seen | (drafted < 0)[:, None]
    seen = seen & (key < lens[:, None])[:, None]
    score.masked_fill_(~seen[:, None, None], -math.inf)
    score -= score.amax(-1, keepdim=True).clamp(min=-1e30)
    p = score.exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(s["seqs"], kv_heads, -1, s["longest"]), v).view(*p.shape[:-1], dim) / torch.where(total > 0, total, 1.0)
    seq, of = _rows_of(s)
    return o.permute(0, 3, 1, 2, 4).reshape(s["seqs"], most, heads, dim)[seq, of].to(s["q"].dtype)


def _plain_accept(s):
    base = (s["lens"] - (s["starts"][1:] - s["starts"][:-1])).long()[:, None]
    path = s["path"].long()
    seq, nth = torch.nonzero(path >= 0, as_tuple=True)
    to, source = (base + torch.arange(path.shape[1], device="cuda"))[seq, nth], (base + path)[seq, nth]
    table = s["table"].long()
    for pages in (s["k_pages"], s["v_pages"]):
        pages[table[seq, to // s["page"]], :, to % s["page"]] = pages[table[seq, source // s["page"]], :, source % s["page"]]
    return {"k_pages": s["k_pages"], "v_pages": s["v_pages"]}


# ----------------------------------------------------------------------------------------------------- one pass

def run(s):
    if own:
        return _run_own(s)
    return {"rope": _plain_train, "append": _plain_append, "attend": _plain_attend, "accept": _plain_accept}[s["op"]](s)


def _run_own(s):
    from binary_rank_gemv_amd import attn
    if s["op"] == "rope":
        turn = {"eps": _EPS, "interleaved": s["interleaved"]}
        q, k = attn.littlebit_rope_fwd(s["q"], s["k"], s["positions"], s["inv_freq"], s["q_weight"], s["k_weight"], **turn)
        dq, dk, dqw, dkw = attn.littlebit_rope_bwd(s["dq"], s["dk"], s["positions"], s["inv_freq"], s["q"], s["k"], s["q_weight"],
                                                   s["k_weight"], **turn)
        return {"q_out": q, "k_out": k, "dq_in": dq, "dq_weight": dqw, "dk_in": dk, "dk_weight": dkw}
    cache = attn.LittleBitCache(s["k_pages"], s["v_pages"])
    batch = attn.CacheBatch(s["starts"], s["lens"], s["table"])
    if s["op"] == "append":
        q = attn.littlebit_cache_append(cache, batch, s["k"], s["v"], s["q"], s["positions"], s["inv_freq"], s["q_weight"], s["k_weight"],
                                        eps=_EPS, interleaved=s["interleaved"])
        return {"q_out": q, "k_pages": cache.k, "v_pages": cache.v}
    if s["op"] == "attend":
        return attn.littlebit_cache_attention_fwd(s["q"], cache, batch, tree=s["tree"])
    attn.littlebit_cache_accept(cache, batch, s["path"])
    return {"k_pages": cache.k, "v_pages": cache.v}


# --------------------------------------------------------------------------------------------- work, exact values

def work(case):
    heads, kv_heads, dim = case.get("heads", 0), case["kv_heads"], case["dim"]
    if case["op"] == "rope":  # q, k in and out; their gradients in and out, with q, k again where a norm's needs them
        values = case["tokens"] * (heads + kv_heads) * dim
        return {"bytes": 2 * values * (5 if case["norm"] else 4) + 4 * case["tokens"] + 2 * case["rot"],
                "flops": values * (20 if case["norm"] else 6)}
    counts = _counts(case)
    rows = sum(t for t, _ in counts)
    if case["op"] == "append":  # q, k, v in; q out, k and v into their pages
        values = rows * (heads + 2 * kv_heads) * dim
        return {"bytes": 4 * values + 8 * rows + 2 * case["rot"], "flops": rows * (heads + kv_heads) * dim * (8 if case["norm"] else 3)}
    if case["op"] == "accept":  # of each sequence, a path of two tokens moves one row of each head
        return {"bytes": 8 * kv_heads * dim * len(counts), "flops": 0}
    keys = sum(t + c for t, c in counts)
    pairs = sum(t * (c + 1) if case["tree"] else t * c + t * (t + 1) // 2 for t, c in counts)
    return {"bytes": 4 * rows * heads * dim + 4 * keys * kv_heads * dim + 4 * -(-keys // case["page"]), "flops": 4 * dim * heads * pairs}


def _turn_exact(x, s, sign):
    """Every pair as a complex number, times exp(i angle)."""
    rot = s["rot"]
    if s["interleaved"]:
        z = torch.view_as_complex(x[..., :rot].reshape(*x.shape[:-1], rot // 2, 2).contiguous())
    else:
        z = torch.complex(x[..., : rot // 2].contiguous(), x[..., rot // 2 : rot].contiguous())
    angle = s["positions"].double()[:, None, None] * s["inv_freq"].double() * sign
    z = z * torch.polar(torch.ones_like(angle), angle)
    turned = torch.view_as_real(z).flatten(-2) if s["interleaved"] else torch.cat([z.real, z.imag], -1)
    return torch.cat([turned, x[..., rot:]], -1)


def _rope_exact(x, weight, s):
    h = x.double()
    if weight is not None:
        h = h / torch.sqrt(h.pow(2).sum(-1, keepdim=True) / s["dim"] + _EPS) * weight.double()
    return _turn_exact(h, s, 1.0)


def _rope_bwd_exact(dy, x, weight, s):
    d = _turn_exact(dy.double(), s, -1.0)
    if weight is None:
        return d, None
    h, w = x.double(), weight.double()
    size = torch.sqrt(h.pow(2).sum(-1, keepdim=True) / s["dim"] + _EPS)
    along = (d * w * h).sum(-1, keepdim=True)
    return d * w / size - h * along / (s["dim"] * size.pow(3)), torch.einsum("thd,thd,th->d", d, h, 1 / size[..., 0])


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        out = {"q_out": _rope_exact(s["q"], s["q_weight"], s), "k_out": _rope_exact(s["k"], s["k_weight"], s)}
        out["dq_in"], out["dq_weight"] = _rope_bwd_exact(s["dq"], s["q"], s["q_weight"], s)
        out["dk_in"], out["dk_weight"] = _rope_bwd_exact(s["dk"], s["k"], s["k_weight"], s)
        return out
    group, size = case.get("heads", 0) // case["kv_heads"], case["page"]
    if case["op"] == "append":
        k, v = s["k_pages"].double(), s["v_pages"].double()
        turned, row = _rope_exact(s["k"], s["k_weight"], s), 0
        for i, (tokens, cached) in enumerate(s["counts"]):
            at = torch.arange(cached, cached + tokens, device="cuda")
            page = s["table"][i].long()[at // size]
            k[page, :, at % size], v[page, :, at % size] = turned[row : row + tokens], s["v"][row : row + tokens].double()
            row += tokens
        return {"q_out": _rope_exact(s["q"], s["q_weight"], s), "k_pages": k, "v_pages": v}
    if case["op"] == "accept":
        k, v = s["k_pages"].double(), s["v_pages"].double()
        for i, ((_, cached), (_, path)) in enumerate(zip(s["counts"], s["trees"])):
            place = lambda at: (s["table"][i].long()[at // size], slice(None), at % size)  # noqa: E731,B023
            source, to = torch.tensor(path, device="cuda") + cached, torch.arange(len(path), device="cuda") + cached
            k[place(to)], v[place(to)] = k[place(source)], v[place(source)]
        return {"k_pages": k, "v_pages": v}
    out, row = [], 0
    for i, (tokens, cached) in enumerate(s["counts"]):
        n = tokens + cached
        page = s["table"][i].long()[: -(-n // size)]
        seen = torch.ones(tokens, n, dtype=torch.bool, device="cuda")
        if s["tree"] is None:
            seen = seen.tril(cached)
        else:
            parents = s["trees"][i][0]
            own_part = torch.zeros(tokens, tokens, dtype=torch.bool)
            for j in range(tokens):
                if j:
                    own_part[j] = own_part[parents[j]]
                own_part[j, j] = True
            seen[:, cached:] = own_part.cuda()
        heads = []
        for h in range(case["heads"]):
            k = s["k_pages"][page, h // group].reshape(-1, case["dim"])[:n].double()
            v = s["v_pages"][page, h // group].reshape(-1, case["dim"])[:n].double()
            score = s["q"][row : row + tokens, h].double() @ k.T / math.sqrt(case["dim"])
            heads.append(torch.softmax(score.masked_fill(~seen, -math.inf), -1) @ v)
        out.append(torch.stack(heads, 1))
        row += tokens
    return torch.cat(out)
