"""The operators at the end of a model whose blocks are LittleBit layers: cases, plain forms, exact values.

A LittleBit model keeps its norms and its output head dense.  Around the packed layers a user needs

* ``norm``    the root-mean-square norm that adds the residual stream first, as an int8 output with one scale a
              token (what an 8-bit product reads) or as a dense output with its backward pass (what a LittleBit
              layer reads, and what training goes back through);
* ``linear``  the product of 8-bit integers with a scale for each token and each output channel (the head);
* ``logprobs`` from the head's logits, the log probability of given tokens, the entropy and the top alternatives,
              with the gradient of the logits.

``run`` computes them in plain torch operations, or with the package's kernels where ``own`` is true.
"""

import math

import torch

own = False

_TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}
_EPS = 1e-5


# --------------------------------------------------------------------------------------------------------- cases

def listed():
    return [
        # one token of a decode step: the last block's output joins the residual stream in front of the head
        {"name": "norm_q8_1x5120_fp16", "op": "norm_q8", "tokens": 1, "n": 5120, "type": "fp16", "pad": 0},
        # a prompt's tokens in front of an 8-bit projection; an odd number of them, the widest model here
        {"name": "norm_q8_2047x8192_bf16", "op": "norm_q8", "tokens": 2047, "n": 8192, "type": "bf16", "pad": 0},
        # a training step's norm in front of a block's projections, forward and backward
        {"name": "norm_train_2048x4096_bf16", "op": "norm_train", "tokens": 2048, "n": 4096, "type": "bf16", "pad": 0},
        # the head for one token, logits in 32 bits: the weights are read once, and that is all the time
        {"name": "linear_1x5120_32000_fp32", "op": "linear", "tokens": 1, "n": 5120, "m": 32000, "type": "fp32", "pad": 0},
        # an up-projection kept in 8 bits, for a small ragged batch of decoded tokens
        {"name": "linear_13x4096_11008_fp16", "op": "linear", "tokens": 13, "n": 4096, "m": 11008, "type": "fp16", "pad": 0},
        # a short prompt: neither the weights' bytes nor the products alone decide
        {"name": "linear_201x5120_13824_bf16", "op": "linear", "tokens": 201, "n": 5120, "m": 13824, "type": "bf16", "pad": 0},
        # the head over a whole text that is scored
        {"name": "linear_2000x4096_32000_fp16", "op": "linear", "tokens": 2000, "n": 4096, "m": 32000, "type": "fp16", "pad": 0},
        # one sampled token and its alternatives
        {"name": "logprobs_1x32000_fp32_top5", "op": "logprobs", "tokens": 1, "vocab": 32000, "top": 5, "type": "fp32", "pad": 0},
        # a batch of decoded tokens over a large vocabulary of an odd size, rows that start at any element
        {"name": "logprobs_61x100003_bf16_top20", "op": "logprobs", "tokens": 61, "vocab": 100003, "top": 20, "type": "bf16", "pad": 0},
        # a text that is scored: the log probabilities behind a perplexity
        {"name": "logprobs_2048x32000_fp16_top1", "op": "logprobs", "tokens": 2048, "vocab": 32000, "top": 1, "type": "fp16", "pad": 0},
        # a small batch's gradient, through the alternatives' log probabilities too
        {"name": "logprobs_train_17x50257_fp32_top4", "op": "logprobs_train", "tokens": 17, "vocab": 50257, "top": 4, "type": "fp32", "pad": 3},
        # a training step's loss and entropy term, forward and backward
        {"name": "logprobs_train_1021x32000_bf16", "op": "logprobs_train", "tokens": 1021, "vocab": 32000, "top": 0, "type": "bf16", "pad": 0},
    ]


def _spread(rng, low, high):
    """A whole number between the two, spread over its logarithm."""
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(["norm_q8", "norm_train", "linear", "linear", "logprobs", "logprobs", "logprobs_train"])
    pad = rng.choice([0, 0, 0, 1, 8, 40])
    if op in ("norm_q8", "norm_train"):
        n = _spread(rng, 64, 16384)
        if rng.random() < 0.5:
            n = -(-n // 64) * 64
        most = (2047 * 8192 if op == "norm_q8" else 2048 * 4096) // n
        return {"op": op, "tokens": _spread(rng, 1, min(4096, most)), "n": n, "type": rng.choice(["fp16", "bf16"]), "pad": pad}
    if op == "linear":
        n, m = _spread(rng, 64, 13824), _spread(rng, 64, 32000)
        if rng.random() < 0.7:
            n = -(-n // 64) * 64
        most = min(2000, 2000 * 4096 * 32000 // (n * m))
        return {"op": op, "tokens": _spread(rng, 1, most), "n": n, "m": m, "type": rng.choice(["fp16", "bf16", "fp32"]), "pad": pad}
    vocab = _spread(rng, 1000, 131072)
    kind = rng.choice(["fp16", "bf16", "fp32"])
    most = (2048 * 32000 if op == "logprobs" else 1021 * 32000) // vocab // (2 if kind == "fp32" else 1)
    return {"op": op, "tokens": _spread(rng, 1, min(2048, most)), "vocab": vocab, "top": rng.choice([0, 1, 4, 20]), "type": kind, "pad": pad}


# -------------------------------------------------------------------------------------------------------- inputs

def _rows(g, tokens, n, pad, make):
    """A tokens x n tensor whose rows lie n + pad elements apart."""
    whole = make(g, tokens, n + pad)
    return whole[:, :n]


def _hidden(t):
    """Hidden states: a few channels far larger than the others, tokens of different size."""
    def make(g, tokens, n):
        x = torch.randn(tokens, n, device="cuda", generator=g)
        loud = torch.rand(n, device="cuda", generator=g) < 0.004
        x *= torch.where(loud, 12.0, 1.0)
        x *= torch.exp(0.5 * torch.randn(tokens, 1, device="cuda", generator=g))
        return x.to(t)
    return make


def _codes(g, rows, n):
    """What an 8-bit quantisation of roughly normal values looks like: one code of a row or so at the border."""
    return torch.randn(rows, n, device="cuda", generator=g).mul_(31.0).round_().clamp_(-127, 127).to(torch.int8)


def _logits(t):
    def make(g, tokens, n):
        x = torch.randn(tokens, n, device="cuda", generator=g)
        x *= 1.5 + torch.rand(tokens, 1, device="cuda", generator=g)
        x += 4.0 * (torch.rand(tokens, n, device="cuda", generator=g) < 3e-4)
        return x.to(t)
    return make


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    t = _TYPES[case["type"]]
    tokens, pad, s = case["tokens"], case["pad"], dict(case)
    if case["op"] in ("norm_q8", "norm_train"):
        n = case["n"]
        s["x"] = _rows(g, tokens, n, pad, _hidden(t))
        s["residual"] = _rows(g, tokens, n, pad, _hidden(t))
        s["weight"] = (0.5 + torch.rand(n, device="cuda", generator=g)).to(t)
        if case["op"] == "norm_train":
            small = lambda g, a, b: (0.1 * torch.randn(a, b, device="cuda", generator=g)).to(t)  # noqa: E731
            s["dy"] = _rows(g, tokens, n, pad, small)
            s["dhidden"] = _rows(g, tokens, n, pad, small)
        else:
            s["values"] = torch.empty(tokens, n, device="cuda", dtype=t)
    elif case["op"] == "linear":
        n, m = case["n"], case["m"]
        s["xq"] = _rows(g, tokens, n, pad, _codes)
        s["xscale"] = 0.02 + 0.03 * torch.rand(tokens, device="cuda", generator=g)
        s["wq"] = _rows(g, m, n, pad, _codes)
        s["wscale"] = (0.5 + torch.rand(m, device="cuda", generator=g)) / (60.0 * math.sqrt(n))
    else:
        vocab, top = case["vocab"], case["top"]
        s["logits"] = _rows(g, tokens, vocab, pad, _logits(t))
        targets = torch.randint(0, vocab, (tokens,), device="cuda", generator=g)
        # padding of a batch: no token is given there
        s["targets"] = torch.where(torch.rand(tokens, device="cuda", generator=g) < 0.05, -100, targets)
        if case["op"] == "logprobs_train":
            s["dlogprob"] = -torch.rand(tokens, device="cuda", generator=g)
            s["dentropy"] = -0.01 * torch.rand(tokens, device="cuda", generator=g)
            s["dtop"] = 0.1 * torch.randn(tokens, top, device="cuda", generator=g) if top else None
    return s


# --------------------------------------------------------------------------------------------------- plain forms

def _plain_norm(s):
    hidden = (s["x"].float() + s["residual"].float()).to(s["x"].dtype)
    h = hidden.float()
    rstd = torch.rsqrt((h * h).mean(1, keepdim=True) + _EPS)
    return hidden, h, rstd, h * rstd * s["weight"].float()


def _plain_norm_q8(s):
    hidden, _, _, y = _plain_norm(s)
    scale = y.abs().amax(1, keepdim=True) / 127.0
    q = torch.round(y / torch.where(scale > 0, scale, 1.0))
    return hidden, (q * scale).to(hidden.dtype), scale[:, 0]


def _plain_norm_train(s):
    hidden, h, rstd, y = _plain_norm(s)
    dy = s["dy"].float()
    xhat = h * rstd
    dxhat = dy * s["weight"].float()
    dx = s["dhidden"].float() + rstd * (dxhat - xhat * (dxhat * xhat).mean(1, keepdim=True))
    return y.to(hidden.dtype), hidden, dx.to(hidden.dtype), (dy * xhat).sum(0)


def _plain_linear(s):
    y = torch.matmul(s["xq"].float(), s["wq"].float().t())
    return (y * s["xscale"][:, None] * s["wscale"]).to(_TYPES[s["type"]])


def _ordered(x):
    """The order of 32-bit floats as whole numbers."""
    b = x.view(torch.int32).to(torch.int64)
    return torch.where(b < 0, -(b & 0x7FFFFFFF), b)


def _plain_top(x, top):
    """The `top` largest of each row and where they are, the lowest place first among equals."""
    place = torch.arange(x.shape[1], device=x.device)
    keys = _ordered(x) * (1 << 24) + ((1 << 24) - 1 - place)
    where = (1 << 24) - 1 - (torch.topk(keys, top, dim=1).values & ((1 << 24) - 1))
    return x.gather(1, where), where


def _plain_logprobs(s):
    x = s["logits"].float().contiguous()
    given = s["targets"] >= 0
    place = s["targets"].clamp(min=0)[:, None]
    most = x.amax(1, keepdim=True)
    d = x - most
    e = torch.exp(d)
    total = e.sum(1, keepdim=True)
    lse = most + torch.log(total)
    logprob = torch.where(given, (x.gather(1, place) - lse)[:, 0], 0.0)
    entropy = (torch.log(total) - torch.where(e > 0, e * d, 0.0).sum(1, keepdim=True) / total)[:, 0]
    if not s["top"]:
        return x, lse, logprob, entropy, None, None
    values, where = _plain_top(x, s["top"])
    return x, lse, logprob, entropy, values - lse, where


def _plain_logprobs_train(s):
    x, lse, logprob, entropy, values, where = _plain_logprobs(s)
    p = torch.exp(x - lse)
    given = s["targets"] >= 0
    dlogprob = torch.where(given, s["dlogprob"], 0.0)[:, None]
    all_given = dlogprob if where is None else dlogprob + s["dtop"].sum(1, keepdim=True)
    dlogits = -p * all_given - torch.where(p > 0, p * (x - lse + entropy[:, None]), 0.0) * s["dentropy"][:, None]
    dlogits.scatter_add_(1, s["targets"].clamp(min=0)[:, None], dlogprob)
    if where is not None:
        dlogits.scatter_add_(1, where, s["dtop"])
    return logprob, entropy, values, where, dlogits.to(s["logits"].dtype)


# ----------------------------------------------------------------------------------------------------- one pass

def run(s):
    if own:
        return _run_own(s)
    if s["op"] == "norm_q8":
        return dict(zip(("hidden", "values", "scale"), _plain_norm_q8(s)))
    if s["op"] == "norm_train":
        return dict(zip(("y", "hidden", "dx", "dweight"), _plain_norm_train(s)))
    if s["op"] == "linear":
        return _plain_linear(s)
    if s["op"] == "logprobs":
        return dict(zip(("logprob", "entropy", "top", "index"), _plain_logprobs(s)[2:]))
    return dict(zip(("logprob", "entropy", "top", "index", "dlogits"), _plain_logprobs_train(s)))


def _run_own(s):
    from binary_rank_gemv_amd import head
    if s["op"] == "norm_q8":
        q, scale, hidden = head.littlebit_rmsnorm_q8(s["x"], s["weight"], s["residual"], eps=_EPS)
        torch.mul(q, scale[:, None], out=s["values"])  # the values that the codes stand for
        return {"hidden": hidden, "values": s["values"], "scale": scale}
    if s["op"] == "norm_train":
        y, hidden = head.littlebit_rmsnorm_fwd(s["x"], s["weight"], s["residual"], eps=_EPS)
        dx, dweight = head.littlebit_rmsnorm_bwd(s["dy"], hidden, s["weight"], dhidden=s["dhidden"], eps=_EPS)
        return {"y": y, "hidden": hidden, "dx": dx, "dweight": dweight}
    if s["op"] == "linear":
        return head.littlebit_q8_linear_fwd(s["xq"], s["xscale"], s["wq"], s["wscale"], dtype=_TYPES[s["type"]])
    logprob, entropy, lse, values, where = head.littlebit_logprobs_fwd(s["logits"], s["targets"], top=s["top"])
    if s["op"] == "logprobs":
        return {"logprob": logprob, "entropy": entropy, "top": values, "index": where}
    dlogits = head.littlebit_logprobs_bwd(s["logits"], s["targets"], lse, entropy, s["dlogprob"], s["dentropy"],
                                          top_index=where, dtop=s["dtop"])
    return {"logprob": logprob, "entropy": entropy, "top": values, "index": where, "dlogits": dlogits}


# --------------------------------------------------------------------------------------------- work, exact values

def work(case):
    b = 4 if case["type"] == "fp32" else 2
    tokens = case["tokens"]
    if case["op"] == "norm_q8":
        n = case["n"]
        return {"bytes": tokens * n * (3 * b + 1) + n * b + 4 * tokens, "flops": 6 * tokens * n}
    if case["op"] == "norm_train":
        n = case["n"]  # read x, residual, dy, dhidden; write hidden, y, dx, dweight
        return {"bytes": 7 * tokens * n * b + n * b + 4 * n, "flops": 14 * tokens * n}
    if case["op"] == "linear":
        n, m = case["n"], case["m"]
        return {"bytes": tokens * n + m * n + 4 * (tokens + m) + tokens * m * b, "flops": 2 * tokens * m * n}
    vocab, top = case["vocab"], case["top"]
    small = tokens * (8 + 4 + 4 + 12 * top)
    if case["op"] == "logprobs":
        return {"bytes": tokens * vocab * b + small, "flops": 6 * tokens * vocab}
    # the logits once, their gradient once
    return {"bytes": 2 * tokens * vocab * b + small + tokens * (8 + 4 * top), "flops": 11 * tokens * vocab}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("norm_q8", "norm_train"):
        hidden = (s["x"].double() + s["residual"].double()).to(s["x"].dtype)  # what is kept, rounded once
        h, w = hidden.double(), s["weight"].double()
        size = torch.sqrt(h.pow(2).sum(1) / case["n"] + _EPS)
        y = h / size[:, None] * w
        if case["op"] == "norm_q8":
            step = y.abs().max(1).values / 127
            codes = torch.div(y, step[:, None]).nan_to_num().round()
            return {"hidden": h, "values": codes * step[:, None], "scale": step}
        dy = s["dy"].double()
        # d y_j / d h_i = w_j (1[i = j] / size - h_i h_j / (n size^3))
        along = torch.linalg.vecdot(dy * w, h)
        dx = s["dhidden"].double() + dy * w / size[:, None] - h * (along / (case["n"] * size.pow(3)))[:, None]
        return {"y": y, "hidden": h, "dx": dx, "dweight": torch.einsum("tn,tn,t->n", dy, h, 1 / size)}
    if case["op"] == "linear":
        w = s["wq"].double() * s["wscale"].double()[:, None]
        return (s["xq"].double() * s["xscale"].double()[:, None]) @ w.T
    x = s["logits"].double()
    logp = torch.log_softmax(x, 1)
    p = logp.exp()
    entropy = torch.special.entr(p).sum(1)
    rows = torch.arange(case["tokens"], device=x.device)
    given = (s["targets"] >= 0).double()
    place = torch.where(s["targets"] >= 0, s["targets"], 0)
    out = {"logprob": logp[rows, place] * given, "entropy": entropy, "top": None, "index": None}
    if case["top"]:
        where = torch.sort(x, dim=1, descending=True, stable=True).indices[:, : case["top"]]
        out["top"] = logp[rows[:, None], where]
    if case["op"] == "logprobs_train":
        d = torch.zeros_like(x)  # the gradient with respect to all log probabilities
        d[rows, place] += s["dlogprob"].double() * given
        if case["top"]:
            d.index_put_((rows[:, None].expand_as(where), where), s["dtop"].double(), accumulate=True)
        d -= s["dentropy"].double()[:, None] * p * (logp.clamp(min=-800.0) + 1)  # H = - sum exp(logp) logp
        out["dlogits"] = d - p * d.sum(1, keepdim=True)
    return out
