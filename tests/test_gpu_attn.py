"""GPU parity of what lies between the projections against the float64 reference
(oracle/attn.py).

Bounds are counted in roundings.  u = 2^-24 is half a step of fp32, e = half a
step of the heads' type (eps / 2); sub is half its smallest subnormal.
* Turns: position * inv_freq / 2 pi in 64 bits is off by 2^-52 of itself, its
  fraction rounded to fp32 by u / 2 of a turn at most; sine and cosine by 2 u more: 2 pi
  (u / 2 + 2^-52 |t|) + 2 u, below 6 u for |t| up to 2^25 turns.
* The norm: a sum of dim squares, 16 in a lane and 4 moves, root, quotient,
  products: 40 u.  The two products and the sum of a turn: 2 u.
* Scores: dim products, exact, added in fp32: dim u sum |q k|, and 4 u |s| of the
  scaling.  exp(d): (|d| + 2) 2 u.  A probability is rounded to the type (e, for fp16
  at least 2^-25 of the largest), the sums of n keys are off by (n + 64) u of their terms.
"""

import itertools

import numpy as np
import pytest
import torch

from oracle import attn as oa

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}
SUB = {torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134}


@pytest.fixture(scope="module")
def attn():
    from binary_rank_gemv_amd import attn
    return attn


def half_step(t):
    return torch.finfo(t).eps / 2


def f64(t):
    return t.detach().cpu().double().numpy()


def randn(seed, *shape, scale=1.0):
    return torch.from_numpy(np.random.default_rng(seed).standard_normal(shape) * scale)


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def case(*what):
    print("[case]", *what, flush=True)


def heads_of(t, how):
    """The same heads as a tensor of their own, as a slice of wider rows at any element, or heads before tokens."""
    n, h, d = t.shape
    if how == "own":
        return t.cuda()
    if how == "fused":
        buf = torch.full((n, 3 + (h + 2) * (d + 1)), 77.0, dtype=t.dtype, device="cuda")
        v = buf[:, 3:3 + h * (d + 1)].unflatten(1, (h, d + 1))[:, :, :d]
    else:
        v = torch.full((h, n, d), 77.0, dtype=t.dtype, device="cuda").transpose(0, 1)
    v.copy_(t)
    return v


# ------------------------------------------------------------------------------------------ head norm and rotation

def turned_bound(a_err, y, positions, inv, interleaved):
    """Bound of a turn's result: the inputs' error, and 8 u of both channels of the pair."""
    big = np.abs(y)
    rot = 0 if inv is None else 2 * len(inv)
    both = big.copy()
    if rot:
        a, b = oa._pairs(y.shape[2], rot, interleaved)
        both[:, :, a] = both[:, :, b] = big[:, :, a] + big[:, :, b]
    far = 0.0 if inv is None else 2 * np.pi * 2.0 ** -51 * np.max(np.abs(positions)) * np.max(np.abs(inv))
    return (a_err + 8 * U + far) * both


def check_rope(got, x, w, positions, inv, interleaved, t):
    y = oa.head_norm(x, w, 1e-5)
    want = oa.turn(y, positions, inv, interleaved)
    err = turned_bound(40 * U if w is not None else 0.0, y, positions, inv, interleaved)
    e = half_step(t)
    bad = np.abs(f64(got) - want) - (e * np.abs(want) + err * (1 + e) + SUB[t])
    assert (bad <= 0).all(), bad.max()


ROPE = [(1, 1, 1, 2, 2), (3, 2, 1, 8, 4), (2, 5, 3, 34, 10), (5, 3, 2, 64, 64), (7, 8, 2, 80, 80), (4, 5, 5, 96, 48), (9, 40, 40, 128, 128),
        (3, 9, 1, 128, 32), (2, 7, 1, 130, 66), (2, 4, 4, 192, 192), (3, 3, 3, 256, 128), (300, 6, 2, 128, 128), (2000, 2, 1, 64, 32)]


def inv_freq(rot):
    return torch.from_numpy(10000.0 ** (-np.arange(0, rot, 2) / rot)).float()


@pytest.mark.parametrize("dt", list(TYPES))
@pytest.mark.parametrize("tokens,heads,kv,dim,rot", ROPE)
def test_rope_forward(attn, tokens, heads, kv, dim, rot, dt):
    t = TYPES[dt]
    rng = np.random.default_rng(dim + tokens)
    for inter, norm, how in ((False, True, "own"), (True, False, "fused"), (False, False, "heads"), (True, True, "fused")):
        case("rope", tokens, heads, kv, dim, rot, dt, inter, norm, how)
        q, k = randn(dim, tokens, heads, dim, scale=3).to(t), randn(dim + 1, tokens, kv, dim).to(t)
        qw, kw = (1 + 0.3 * randn(2, dim)).to(t), (1 + 0.3 * randn(3, dim)).to(t)
        pos = torch.from_numpy(rng.integers(-100, 1 << 17, tokens)).int()
        inv = inv_freq(rot)
        qo, ko = attn.littlebit_rope_fwd(heads_of(q, how), heads_of(k, how), pos.cuda(), inv.cuda(), qw.cuda() if norm else None,
                                         kw.cuda() if norm else None, interleaved=inter)
        check_rope(qo, f64(q), f64(qw) if norm else None, pos.numpy(), f64(inv), inter, t)
        check_rope(ko, f64(k), f64(kw) if norm else None, pos.numpy(), f64(inv), inter, t)


def check_rope_backward(got, dw, dy, x, w, positions, inv, interleaved, t):
    want, wantw = oa.rope_backward(dy, x, w, positions, inv, 1e-5, interleaved)
    dz = oa.turn(dy, positions, inv, interleaved, -1.0)
    err = turned_bound(0.0, dy, positions, inv, interleaved)
    if w is not None:
        r = 1 / np.sqrt(np.mean(x * x, 2, keepdims=True) + 1e-5)
        xr = np.abs(x) * r
        along = lambda v: xr * np.mean(np.abs(w) * v * xr, 2, keepdims=True)  # noqa: E731
        terms = int(np.prod(dy.shape[:2]))
        chain = 16 + terms // 256 + 100
        bound = np.sum(err * xr + (40 + chain) * U * np.abs(dz) * xr, axis=(0, 1))
        assert (np.abs(f64(dw) - wantw) <= bound).all()
        err = r * (np.abs(w) * err + along(err)) + 100 * U * r * (np.abs(w * dz) + along(np.abs(dz)))
    e = half_step(t)
    bad = np.abs(f64(got) - want) - (e * np.abs(want) + err * (1 + e) + SUB[t])
    assert (bad <= 0).all(), bad.max()


@pytest.mark.parametrize("dt", list(TYPES))
@pytest.mark.parametrize("tokens,heads,kv,dim,rot", ROPE)
def test_rope_backward(attn, tokens, heads, kv, dim, rot, dt):
    t = TYPES[dt]
    rng = np.random.default_rng(dim + tokens)
    for inter, norm, how in ((False, True, "own"), (True, False, "fused"), (True, True, "heads"), (False, True, "fused")):
        case("rope backward", tokens, heads, kv, dim, rot, dt, inter, norm, how)
        x = [randn(dim, tokens, heads, dim, scale=3).to(t), randn(dim + 1, tokens, kv, dim).to(t)]
        dy = [randn(dim + 2, tokens, heads, dim).to(t), randn(dim + 3, tokens, kv, dim).to(t)]
        w = [(1 + 0.3 * randn(2, dim)).to(t), (1 + 0.3 * randn(3, dim)).to(t)]
        pos = torch.from_numpy(rng.integers(-100, 1 << 17, tokens)).int()
        inv = inv_freq(rot)
        xs = [heads_of(v, how) for v in x] if norm else [None, None]
        ws = [v.cuda() for v in w] if norm else [None, None]
        got = attn.littlebit_rope_bwd(heads_of(dy[0], how), heads_of(dy[1], how), pos.cuda(), inv.cuda(), *xs, *ws, interleaved=inter)
        for i in range(2):
            assert (got[2 + i] is None) == (not norm)
            check_rope_backward(got[i], got[2 + i], f64(dy[i]), f64(x[i]), f64(w[i]) if norm else None, pos.numpy(), f64(inv), inter, t)


def test_rope_of_one_of_the_two_and_norm_alone(attn):
    q, w = randn(1, 5, 3, 64).half(), (1 + 0.3 * randn(2, 64)).half()
    qo, ko = attn.littlebit_rope_fwd(q.cuda(), None, q_weight=w.cuda())
    assert ko is None
    check_rope(qo, f64(q), f64(w), None, None, False, torch.float16)
    qo, ko = attn.littlebit_rope_fwd(None, q.cuda(), torch.arange(5).int().cuda(), inv_freq(64).cuda(), k_weight=w.cuda())
    assert qo is None
    check_rope(ko, f64(q), f64(w), np.arange(5), f64(inv_freq(64)), False, torch.float16)
    dq, dk, dqw, dkw = attn.littlebit_rope_bwd(None, q.cuda(), k=(2 * q).cuda(), k_weight=w.cuda())
    assert dq is None and dqw is None
    check_rope_backward(dk, dkw, f64(q), f64(2 * q), f64(w), None, None, False, torch.float16)


def test_rope_in_place_and_surroundings(attn):
    t = torch.bfloat16
    x, w, pos, inv = randn(1, 9, 4, 128).to(t), (1 + 0.3 * randn(2, 128)).to(t), torch.arange(9).int().cuda(), inv_freq(128).cuda()
    for how in ("own", "fused", "heads"):
        want, _ = attn.littlebit_rope_fwd(x.cuda(), None, pos, inv, w.cuda())
        v = heads_of(x, how)
        out, _ = attn.littlebit_rope_fwd(v, None, pos, inv, w.cuda(), q_out=v)
        assert out is v and torch.equal(v, want)
        back, _, dw, _ = attn.littlebit_rope_bwd(x.cuda(), None, pos, inv, q=x.cuda(), q_weight=w.cuda())
        v = heads_of(x, how)
        got, _, dw2, _ = attn.littlebit_rope_bwd(v, None, pos, inv, q=x.cuda(), q_weight=w.cuda(), dq_in=v)
        assert got is v and torch.equal(v, back) and torch.equal(dw, dw2)   # the same bits
        base = v._base if v._base is not None else v
        if how == "fused":
            inside = torch.zeros_like(base, dtype=torch.bool)
            inside[:, 3:3 + 4 * 129].unflatten(1, (4, 129))[:, :, :128] = True
            assert (base[~inside] == 77).all()


def test_rope_of_values_whose_squares_leave_fp32(attn):
    """bf16 heads around 1e30 and 1e-25 (with eps 0), beside ordinary ones in one call."""
    t = torch.bfloat16
    for size, eps in ((1e30, 1e-5), (1e-25, 0.0)):
        case("rope of", size)
        x = randn(3, 4, 10, 128)
        x[1, 3] *= size
        x[2] *= size
        x, w, dy = x.to(t), (1 + 0.2 * randn(4, 128)).to(t), randn(5, 4, 10, 128).to(t)
        got, _ = attn.littlebit_rope_fwd(x.cuda(), None, q_weight=w.cuda(), eps=eps)
        want = oa.head_norm(f64(x), f64(w), eps)
        assert (np.abs(f64(got) - want) <= (half_step(t) + 60 * U) * np.abs(want)).all()
        dx, _, dw, _ = attn.littlebit_rope_bwd(dy.cuda(), None, q=x.cuda(), q_weight=w.cuda(), eps=eps)
        wantx, wantw = oa.rope_backward(f64(dy), f64(x), f64(w), None, None, eps)
        # of each head's largest: 100 u and a rounding
        most = np.abs(wantx).max(2, keepdims=True)
        # below bf16's smallest normal value the steps are 2^-133
        assert (np.abs(f64(dx) - wantx) <= (half_step(t) + 200 * U) * most + 2.0 ** -133).all()
        terms = np.sum(np.abs(f64(dy) * want / f64(w)), axis=(0, 1))
        assert (np.abs(f64(dw) - wantw) <= 200 * U * terms).all()


def test_far_positions_keep_their_turn(attn):
    pos = torch.tensor([2 ** 31 - 1, -2 ** 31, 2 ** 30 + 1, 12345678], dtype=torch.int32)
    x, inv = randn(1, 4, 1, 64).half(), torch.tensor([1.0] * 16 + [0.3] * 16)
    got, _ = attn.littlebit_rope_fwd(x.cuda(), None, pos.cuda(), inv.cuda())
    check_rope(got, f64(x), None, pos.numpy().astype(np.float64), f64(inv), False, torch.float16)


def test_rotated_and_plain_channels_do_not_mix_infinities(attn):
    x = randn(1, 1, 1, 64).half()
    x[0, 0, 40] = float("inf")
    for inter in (False, True):
        got, _ = attn.littlebit_rope_fwd(x.cuda(), None, ints([3]), inv_freq(32).cuda(), interleaved=inter)
        assert torch.equal(got[0, 0, 32:].cpu(), x[0, 0, 32:]) and torch.isfinite(got[0, 0, :32]).all()


def test_rope_of_no_tokens(attn):
    x, w = torch.empty(0, 3, 64, dtype=torch.float16, device="cuda"), torch.ones(64, dtype=torch.float16, device="cuda")
    q, k = attn.littlebit_rope_fwd(x, x, ints([]), inv_freq(64).cuda(), w, w)
    assert q.shape == k.shape == x.shape
    out = attn.littlebit_rope_bwd(x, x, ints([]), inv_freq(64).cuda(), x, x, w, w)
    assert (out[2] == 0).all() and (out[3] == 0).all()


# ---------------------------------------------------------------------------------------------- caches and batches

class Paged:
    """A cache of random values with room for the sequences, in any layout, and its batch."""

    def __init__(self, attn, seed, counts, kv, dim, page, t, layout="heads", before=0, behind=0, spare=1):
        self.counts, self.page, self.t = counts, page, t
        rng = np.random.default_rng(seed)
        self.starts = np.concatenate([[0], np.cumsum([n for n, _ in counts])]).astype(int) + before
        self.lens = np.array([n + c for n, c in counts])
        self.tokens = int(self.starts[-1]) + behind
        columns = max(1, -(-int(self.lens.max()) // page)) + spare
        pages = len(counts) * columns + 2
        self.table = rng.permutation(pages)[:len(counts) * columns].reshape(len(counts), columns)
        shape = (pages, kv, page, dim)
        if layout == "heads":
            k, v = (torch.empty(shape, dtype=t, device="cuda") for _ in range(2))
        elif layout == "slots":
            k, v = (torch.empty(pages, page, kv, dim, dtype=t, device="cuda").transpose(1, 2) for _ in range(2))
        else:  # keys and values of a page in one tensor, with room between the slots
            both = torch.empty(pages, 2, kv, page, dim + 8, dtype=t, device="cuda")
            k, v = both[:, 0, :, :, :dim], both[:, 1, :, :, :dim]
        k.copy_(torch.from_numpy(rng.standard_normal(shape)))
        v.copy_(torch.from_numpy(rng.standard_normal(shape)))
        self.cache = attn.LittleBitCache(k, v)
        self.batch = attn.CacheBatch(ints(self.starts.tolist()), ints(self.lens.tolist()), ints(self.table.tolist()))

    def say(self):
        self.batch.lens.copy_(torch.from_numpy(self.lens))
        self.batch.table.copy_(torch.from_numpy(self.table))


def check_attention(got, lse, q, p, scale, tree=None):
    k, v = f64(p.cache.k), f64(p.cache.v)
    args = (p.starts, p.lens, p.table, scale, tree)
    want, want_lse = oa.attention(f64(q), k, v, *args)
    size, _ = oa.attention(f64(q), k, np.abs(v), *args)
    mine = ~np.isnan(want_lse)
    e, n, dim = half_step(p.t), max(1, int(p.lens.max())), q.shape[2]
    norm = np.sqrt(np.sum(f64(q) ** 2, 2)) * np.sqrt(np.max(np.sum(k ** 2, 3)))   # of any |q| |k|
    score = abs(scale) * (dim + 8) * U * norm
    ds = 2 * (score + 2 * U * (min(30.0, 2 * float(np.max(abs(scale) * norm))) + 2) + (n + 80) * U)
    err = (e + ds)[:, :, None] * size
    if p.t == torch.float16:
        err = err + n * 2.0 ** -25 * np.abs(v).max()
    bad = np.abs(f64(got) - want) - (e * np.abs(want) + err * (1 + e) + SUB[p.t])
    assert mine.any() and (bad[mine] <= 0).all(), np.nanmax(bad)
    if lse is not None:
        g = f64(lse)
        assert (np.isneginf(g[mine]) == np.isneginf(want_lse[mine])).all()
        fine = mine & np.isfinite(want_lse)
        assert (np.abs(g[fine] - want_lse[fine]) <= (ds + 4 * U * (1 + np.abs(want_lse)))[fine]).all()


def run_attention(attn, p, q, scale=None, tree=None, how="own"):
    out = torch.full(q.shape, 55.0, dtype=q.dtype, device="cuda")
    lse = torch.full(q.shape[:2], 55.0, device="cuda")
    t = None if tree is None else torch.from_numpy(np.array(tree, dtype=np.int64)).cuda()
    got = attn.littlebit_cache_attention_fwd(heads_of(q, how), p.cache, p.batch, t, scale, out=out, lse=lse)
    assert got is out
    outside = np.ones(q.shape[0], bool)
    outside[[t for t in oa.rows(p.starts, q.shape[0])]] = False
    assert (out[outside] == 55).all() and (lse[outside] == 55).all()   # left as they were
    return out, lse


# (rows, keys before them) of each sequence, heads, kv heads, dim, page
ATTEND = [
    ([(1, 0)], 1, 1, 8, 8), ([(1, 1)], 2, 1, 64, 8), ([(1, 30)], 3, 3, 128, 16), ([(1, 31), (1, 32), (1, 33)], 8, 1, 128, 32),
    ([(1, 511), (0, 77), (1, 0), (1, 1023)], 4, 2, 80, 16), ([(2, 100)], 5, 5, 96, 8), ([(16, 250)], 8, 8, 128, 64),
    ([(7, 900), (16, 3), (1, 2000)], 16, 2, 128, 128), ([(5, 0), (33, 7)], 6, 2, 64, 16), ([(70, 200)], 7, 1, 128, 64),
    ([(150, 0), (0, 0), (3, 50)], 4, 4, 192, 8), ([(40, 333)], 4, 2, 256, 32), ([(1, 5000)], 2, 1, 128, 64),
    ([(9, 4000), (1, 1)], 4, 1, 256, 64), ([(3, 2500)], 2, 2, 64, 8), ([(300, 40)], 3, 1, 64, 16), ([(1, 3000)], 40, 1, 24, 16),
    ([(130, 1111), (257, 0)], 4, 2, 128, 16), ([(1, 700), (2, 90)], 64, 1, 128, 1024), ([(100, 6000)], 4, 1, 128, 64),
    ([(40, 2500), (41, 2400)], 16, 4, 64, 32), ([(200, 1500)], 1, 1, 256, 128), ([(90, 40), (300, 7), (513, 0), (1, 9)], 2, 2, 96, 8),
    ([(300, 4200), (300, 10), (0, 3)], 4, 2, 112, 32), ([(600, 100)], 8, 1, 128, 64), ([(140, 4500), (31, 225)], 4, 1, 128, 16),
]


@pytest.mark.parametrize("dt", list(TYPES))
@pytest.mark.parametrize("counts,heads,kv,dim,page", ATTEND)
def test_attention_of_causal_rows(attn, counts, heads, kv, dim, page, dt):
    for layout, how, pad in (("heads", "own", 0), ("slots", "fused", 3), ("both", "heads", 1)):
        case("attention", counts, heads, kv, dim, page, dt, layout)
        p = Paged(attn, dim, counts, kv, dim, page, TYPES[dt], layout, before=pad, behind=2 * pad)
        q = randn(dim + 1, p.tokens, heads, dim, scale=1.5).to(p.t)
        out, lse = run_attention(attn, p, q, how=how)
        check_attention(out, lse, q, p, dim ** -0.5)


def tree_words(rng, rows):
    words = [1]
    for i in range(1, rows):
        words.append(words[rng.integers(0, i)] | 1 << i)
    return [w - (1 << 64) if w >> 63 else w for w in words]


TREES = [([(1, 0)], 1, 1, 64, 8), ([(2, 0), (16, 31)], 4, 4, 128, 16), ([(64, 0)], 2, 1, 128, 8), ([(64, 1000), (13, 64), (0, 4), (27, 1)], 8, 2, 128, 64),
         ([(33, 4099)], 4, 1, 64, 32), ([(61, 77), (5, 3)], 3, 1, 256, 16), ([(16, 2000)], 2, 2, 80, 64), ([(64, 31), (64, 32), (64, 33)], 8, 8, 96, 8), ([(64, 5000)], 4, 1, 128, 64), ([(50, 3000), (64, 9)], 8, 2, 256, 16),
         ([(64, 4300), (5, 70), (33, 0)], 8, 1, 72, 16)]


@pytest.mark.parametrize("dt", list(TYPES))
@pytest.mark.parametrize("counts,heads,kv,dim,page", TREES)
def test_attention_of_trees(attn, counts, heads, kv, dim, page, dt):
    rng = np.random.default_rng(len(counts))
    for layout, pad in (("heads", 0), ("slots", 2)):
        case("tree", counts, heads, kv, dim, page, dt, layout)
        p = Paged(attn, dim, counts, kv, dim, page, TYPES[dt], layout, before=pad, behind=pad)
        tree = [7] * pad + [w for n, _ in counts for w in (tree_words(rng, n) if n else [])] + [-1] * pad
        q = randn(dim + 1, p.tokens, heads, dim, scale=1.5).to(p.t)
        out, lse = run_attention(attn, p, q, tree=tree)
        check_attention(out, lse, q, p, dim ** -0.5, tree)


def test_rows_that_see_nothing(attn):
    """Words of zeros, bits of rows that are not there, sequences with fewer keys than rows."""
    p = Paged(attn, 1, [(5, 0), (6, 40), (4, 0)], 2, 128, 8, torch.float16)
    tree = [0, 1 << 1, 1 << 9, -1 << 60, 3] + [0, -1, 1 << 5, -(1 << 63), 0, 1] + [0, 0, 0, 0]
    q = randn(2, p.tokens, 4, 128).half()
    out, lse = run_attention(attn, p, q, tree=tree)
    check_attention(out, lse, q, p, 128 ** -0.5, tree)
    assert (out[0] == 0).all() and torch.isneginf(lse[0]).all() and (out[11:15] == 0).all()
    p.lens[:] = [2, 46, 0]   # rows whose keys were never counted
    p.say()
    out, lse = run_attention(attn, p, q)
    check_attention(out, lse, q, p, 128 ** -0.5)
    assert (out[:3] == 0).all() and (out[11:15] == 0).all()


def test_many_sequences(attn):
    """More than a wave has lanes, of all lengths, empty ones among them."""
    rng = np.random.default_rng(3)
    for seqs in (63, 64, 65, 130, 300):
        case("sequences", seqs)
        counts = [(int(rng.integers(0, 4)), int(rng.integers(0, 90))) for _ in range(seqs)]
        counts[0], counts[-1] = (0, 5), (2, 700)
        p = Paged(attn, seqs, counts, 1, 64, 16, torch.bfloat16)
        q = randn(seqs, p.tokens, 2, 64).bfloat16()
        out, lse = run_attention(attn, p, q)
        check_attention(out, lse, q, p, 0.125)


@pytest.mark.parametrize("seqs,rows,heads,dim", [(129, 3, 2, 64), (2000, 3, 2, 128), (4200, 1, 1, 64), (200, 70, 4, 128), (150, 90, 2, 256)])
def test_thousands_of_sequences(attn, seqs, rows, heads, dim):
    """More than are added up by every workgroup, some long enough for several parts, some empty."""
    case("thousands", seqs, rows)
    rng = np.random.default_rng(seqs)
    counts = [(int(rng.integers(0, rows + 1)), int(rng.integers(0, 40))) for _ in range(seqs)]
    counts[0], counts[64], counts[65], counts[seqs - 1] = (rows, 1500), (0, 70), (rows, 0), (rows, 3000)
    p = Paged(attn, seqs, counts, 1, dim, 16, torch.float16)
    q = randn(seqs, p.tokens, heads, dim).half()
    out, lse = run_attention(attn, p, q)
    check_attention(out, lse, q, p, dim ** -0.5)


@pytest.mark.parametrize("scale", [0.0, -0.2, 3.0])
def test_scales(attn, scale):
    p = Paged(attn, 4, [(3, 100)], 1, 64, 16, torch.float16)
    q = randn(5, 3, 2, 64).half()
    out, lse = run_attention(attn, p, q, scale=scale)
    check_attention(out, lse, q, p, scale)


def test_scores_that_rise_and_fall(attn):
    """The maximum grows step by step, by less and by more than the sums are let stand; and the first key is the largest."""
    for keys, G in ((700, 1), (700, 8), (3000, 20)):
        for step in (0.02, 0.9, -0.5):
            case("rising", keys, G, step)
            p = Paged(attn, 4, [(2, keys)], 1, 64, 16, torch.float16)
            p.cache.k.zero_()
            for j in range(keys + 2):
                a = oa.place(0, j, p.table, 16, p.cache.k.shape[0])
                p.cache.k[a[0], 0, a[1], 0] = step * (j // 32)
            q = torch.zeros(2, G, 64, dtype=torch.float16)
            q[:, :, 0] = 8.0
            out, lse = run_attention(attn, p, q)
            check_attention(out, lse, q, p, 0.125)


def spoil(p, seq, key, value, which):
    a = oa.place(seq, key, p.table, p.page, p.cache.k.shape[0])
    for c in which:
        c[a[0], :, a[1], 1::3] = value


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("rows", [1, 5, 40, 200])
@pytest.mark.parametrize("dt", list(TYPES))
def test_what_is_not_seen_has_no_part(attn, rows, value, dt):
    """NaN and infinities in later rows' keys and values, in rows of other branches, and behind the sequences."""
    case("unseen", rows, value, dt)
    for dim, G in ((128, 2), (256, 1), (64, 8)):
        p = Paged(attn, 6, [(rows, 60), (2, 9)], 1, dim, 16, TYPES[dt], spare=2)
        q = randn(7, p.tokens, G, dim).to(p.t)
        clean, _ = run_attention(attn, p, q)
        for key in range(p.lens[0], p.lens[0] + 16):
            spoil(p, 0, key, value, (p.cache.k, p.cache.v))
        hit = max(0, rows - 3)   # the keys and values of this row
        if rows > 1:
            spoil(p, 0, 60 + hit, value, (p.cache.k, p.cache.v))
        out, _ = run_attention(attn, p, q)
        assert torch.equal(out[:hit], clean[:hit]) and torch.equal(out[rows:], clean[rows:])
        if rows > 1:
            assert not torch.isfinite(out[hit:rows]).all(2).any()
        if 1 < rows <= 64:
            tree = [1 | 1 << i for i in range(rows)] + [1, 3]
            tree = [w - (1 << 64) if w >> 63 else w for w in tree]
            out, _ = run_attention(attn, p, q, tree=tree)
            others = [i for i in range(rows) if i != hit]
            if hit > 0:
                assert torch.isfinite(out[others]).all() and not torch.isfinite(out[hit]).all(1).any()


@pytest.mark.parametrize("dt", list(TYPES))
@pytest.mark.parametrize("rows,cached,heads,dim", [(6, 40, 2, 128), (300, 40, 1, 128), (300, 4200, 2, 128), (200, 2000, 2, 64), (150, 1030, 1, 256), (40, 900, 2, 256)])
def test_values_that_are_seen_keep_their_infinities(attn, rows, cached, heads, dim, dt):
    """Infinite values of one sign in a channel give that infinity to the rows that see them, of both signs NaN; among
    the keys before the rows they reach every row."""
    p = Paged(attn, 8, [(rows, cached)], 1, dim, 8, TYPES[dt])
    at = lambda key: oa.place(0, key, p.table, 8, p.cache.k.shape[0])  # noqa: E731
    inf, mid = float("inf"), rows // 2
    for row, channel, value in ((1, 3, inf), (3, 3, -inf), (4, dim - 28, -inf), (mid, 30, float("nan")), (2 - cached, 9, inf)):
        p.cache.v[at(cached + row)[0], :, at(cached + row)[1], channel] = value
    out, _ = run_attention(attn, p, randn(9, rows, heads, dim).to(p.t))
    o = out.float()
    assert (o[:, :, 9] == inf).all() and torch.isfinite(o[0, :, [3, 30]]).all()
    assert (o[1:3, :, 3] == inf).all() and torch.isnan(o[3:, :, 3]).all()
    assert (o[4:, :, dim - 28] == -inf).all() and torch.isfinite(o[:4, :, dim - 28]).all()
    assert torch.isnan(o[mid:, :, 30]).all() and torch.isfinite(o[:mid, :, 30]).all()
    rest = [d for d in range(dim) if d not in (3, 9, 30, dim - 28)]
    assert torch.isfinite(o[:, :, rest]).all()


def test_entries_that_name_no_page(attn):
    """Their keys are not attended and not written, and nothing else is touched."""
    for rows, cached in ((1, 300), (100, 300), (100, 4300)):
        dim = 128 if cached > 4096 else 64
        case("bad entries", rows, cached)
        p = Paged(attn, 10, [(rows, cached), (1, 50)], 2, dim, 16, torch.bfloat16)
        pages = p.cache.k.shape[0]
        p.table[0, 2], p.table[0, 5], p.table[0, -2], p.table[1, 1] = -1, pages, 2 ** 31 - 1, -2 ** 31
        p.say()
        q = randn(11, p.tokens, 4, dim).bfloat16()
        out, lse = run_attention(attn, p, q)
        check_attention(out, lse, q, p, dim ** -0.5)
        k, v = randn(12, p.tokens, 2, dim).bfloat16(), randn(13, p.tokens, 2, dim).bfloat16()
        want = oa.append(f64(p.cache.k), f64(p.cache.v), f64(k), f64(v), p.starts, p.lens, p.table)
        attn.littlebit_cache_append(p.cache, p.batch, k.cuda(), v.cuda())
        assert np.array_equal(f64(p.cache.k), want[0]) and np.array_equal(f64(p.cache.v), want[1])
    p.lens[:] = [1 << 30, 2 ** 31 - 1]   # more keys than columns hold
    p.say()
    p.lens[:] = [p.table.shape[1] * 16 + 10 ** 6] * 2
    out, _ = run_attention(attn, p, q)
    assert torch.isfinite(out).all()


def test_starts_that_leave_the_rows(attn):
    """Sequences that begin or end outside of the call's rows have only those inside, or none."""
    p = Paged(attn, 14, [(2, 30), (2, 30), (2, 30)], 1, 64, 16, torch.float16)
    q = randn(15, 6, 1, 64).half()
    p.starts = np.array([0, 2, 4, 900])
    p.lens[2] = 30 + 896
    p.batch.starts.copy_(torch.from_numpy(p.starts))
    p.say()
    out, lse = run_attention(attn, p, q)
    check_attention(out, lse, q, p, 0.125)
    p.batch.starts.copy_(torch.tensor([-5, 2, 1, 6]))   # no sequence has rows 0 to 1 by its own start
    out = attn.littlebit_cache_attention_fwd(q.cuda(), p.cache, p.batch, out=torch.zeros_like(q, device="cuda"))
    assert torch.isfinite(out).all()


@pytest.mark.parametrize("dt", list(TYPES))
def test_a_cache_of_more_than_32_bits(attn, dt):
    t = TYPES[dt]
    pages, page, kv, dim = 9000, 256, 8, 128   # 2.4e9 elements, 4.7 GB each of keys and values
    k = torch.empty(pages, kv, page, dim, dtype=t, device="cuda")
    v = torch.empty_like(k)
    cache = attn.LittleBitCache(k, v)
    table = np.array([[pages - 1, 0, pages - 2]])
    new = [randn(i, 600, kv, dim).to(t) for i in range(3)]
    batch = attn.CacheBatch(ints([0, 600]), ints([600]), ints(table.tolist()))
    q = attn.littlebit_cache_append(cache, batch, new[0].cuda(), new[1].cuda(), new[2].cuda())
    out = attn.littlebit_cache_attention_fwd(q, cache, batch)
    p = Paged(attn, 1, [(600, 0)], kv, dim, page, t, spare=0)
    p.cache = attn.LittleBitCache(k[[pages - 1, 0, pages - 2]], v[[pages - 1, 0, pages - 2]])
    p.table = np.array([[0, 1, 2]])
    rows = slice(0, 600, 37)
    want, _ = oa.attention(f64(new[2]), f64(p.cache.k), f64(p.cache.v), [0, 600], [600], p.table, dim ** -0.5)
    # e of the output and e of the probabilities, which add to values of size 1
    assert (np.abs(f64(out) - want)[rows] <= 2.1 * half_step(t) * (1 + np.abs(want)[rows]) * 4).all()
    attn.littlebit_cache_accept(cache, batch, ints([[550, 551]]))
    assert torch.equal(k[pages - 1, :, 0].cpu(), new[0][550]) and torch.equal(v[pages - 1, :, 1].cpu(), new[1][551])


# -------------------------------------------------------------------------------------------- append, accept, chains

@pytest.mark.parametrize("dt", list(TYPES))
@pytest.mark.parametrize("counts,heads,kv,dim,page", [
    ([(1, 0)], 1, 1, 8, 8), ([(1, 63), (1, 64)], 40, 40, 128, 64), ([(5, 3), (0, 9), (20, 100)], 8, 2, 128, 16),
    ([(3, 7)], 7, 1, 80, 8), ([(200, 11)], 4, 4, 64, 32), ([(9, 0)], 3, 3, 256, 16), ([(4, 4)], 5, 5, 24, 8)])
def test_append(attn, counts, heads, kv, dim, page, dt):
    t = TYPES[dt]
    for layout, how, norm, inter, rot in (("heads", "own", True, False, dim), ("slots", "fused", False, True, dim // 4 * 2), ("both", "heads", True, True, 0)):
        case("append", counts, heads, kv, dim, page, dt, layout)
        p = Paged(attn, dim, counts, kv, dim, page, t, layout, before=1, behind=3)
        q, k, v = (randn(i, p.tokens, h, dim).to(t) for i, h in ((1, heads), (2, kv), (3, kv)))
        qw, kw = ((1 + 0.3 * randn(i, dim)).to(t) for i in (4, 5))
        pos = torch.arange(100, 100 + p.tokens).int()
        inv = inv_freq(rot) if rot else None
        before = [c.clone() for c in (p.cache.k, p.cache.v)]
        out = torch.full((p.tokens, heads, dim), 55.0, dtype=t, device="cuda")
        turn = (pos.cuda(), inv.cuda()) if rot else (None, None)
        got = attn.littlebit_cache_append(p.cache, p.batch, heads_of(k, how), heads_of(v, how), heads_of(q, how), *turn, qw.cuda() if norm else None,
                                          kw.cuda() if norm else None, interleaved=inter, q_out=out)
        mine = sorted(oa.rows(p.starts, p.tokens))
        outside = [i for i in range(p.tokens) if i not in mine]
        assert got is out and (out[outside] == 55).all()
        dense = attn.littlebit_rope_fwd(q.cuda(), k.cuda(), *turn, qw.cuda() if norm else None, kw.cuda() if norm else None, interleaved=inter)
        check_rope(dense[1], f64(k), f64(kw) if norm else None, pos.numpy(), f64(inv) if rot else None, inter, t)
        assert torch.equal(out[mine], dense[0][mine])   # the same arithmetic
        want = oa.append(f64(before[0]), f64(before[1]), f64(dense[1]), f64(v), p.starts, p.lens, p.table)
        assert np.array_equal(f64(p.cache.k), want[0]) and np.array_equal(f64(p.cache.v), want[1])
        attn.littlebit_cache_append(p.cache, p.batch, k.cuda(), v.cuda())   # without queries, as they are
        want = oa.append(want[0], want[1], f64(k), f64(v), p.starts, p.lens, p.table)
        assert np.array_equal(f64(p.cache.k), want[0]) and np.array_equal(f64(p.cache.v), want[1])


@pytest.mark.parametrize("dt", list(TYPES))
@pytest.mark.parametrize("counts,kv,dim,page,columns", [
    ([(1, 5)], 1, 8, 8, 1), ([(16, 30)], 40, 128, 64, 5), ([(64, 3), (0, 5), (20, 100), (7, 0)], 3, 256, 8, 64), ([(33, 7)] * 70, 2, 80, 16, 9)])
def test_accept(attn, counts, kv, dim, page, columns, dt):
    rng = np.random.default_rng(columns)
    for layout in ("heads", "slots", "both"):
        case("accept", counts[:4], kv, dim, page, columns, dt, layout)
        p = Paged(attn, dim, counts, kv, dim, page, TYPES[dt], layout)
        # ancestors first, and any order, the same row twice and rows that are not there
        for path in ([sorted(rng.choice(64, columns, replace=False).tolist()) for _ in counts], rng.integers(-3, 70, (len(counts), columns)).tolist()):
            want = [oa.accept(f64(c), path, p.starts, p.lens, p.table) for c in (p.cache.k, p.cache.v)]
            attn.littlebit_cache_accept(p.cache, p.batch, ints(path))
            assert np.array_equal(f64(p.cache.k), want[0]) and np.array_equal(f64(p.cache.v), want[1])


def test_a_verified_tree_is_the_text_of_its_path(attn):
    """Append a tree, attend, accept a path: the cache and the path's outputs are those of the plain text."""
    t, dim, kv, heads = torch.bfloat16, 128, 2, 8
    p = Paged(attn, 20, [(11, 70)], kv, dim, 16, t)
    q, k, v = (randn(i, 11, h, dim).to(t).cuda() for i, h in ((1, heads), (2, kv), (3, kv)))
    parents = [-1, 0, 0, 1, 1, 2, 3, 5, 5, 6, 9]
    words, depth = [], []
    for i, a in enumerate(parents):
        words.append((words[a] if a >= 0 else 0) | 1 << i)
        depth.append(depth[a] + 1 if a >= 0 else 0)
    inv = inv_freq(dim).cuda()
    turned = attn.littlebit_cache_append(p.cache, p.batch, k, v, q, ints([70 + d for d in depth]), inv)
    out = attn.littlebit_cache_attention_fwd(turned, p.cache, p.batch, torch.tensor(words).cuda())
    path = [0, 1, 3, 6, 9, 10]
    attn.littlebit_cache_accept(p.cache, p.batch, ints([path]))
    text = Paged(attn, 20, [(6, 70)], kv, dim, 16, t, spare=1)
    text.cache, text.table = p.cache, p.table
    plain = attn.LittleBitCache(p.cache.k.clone(), p.cache.v.clone())
    batch = attn.CacheBatch(ints([0, 6]), ints([76]), p.batch.table)
    turned = attn.littlebit_cache_append(plain, batch, k[path].contiguous(), v[path].contiguous(), q[path].contiguous(), ints(range(70, 76)), inv)
    assert torch.equal(plain.k, p.cache.k) and torch.equal(plain.v, p.cache.v)
    again = attn.littlebit_cache_attention_fwd(turned, plain, batch)
    for rows in (out[path], again):
        check_attention(rows, None, turned.cpu(), text, dim ** -0.5)


def test_same_call_same_bits_on_any_stream(attn):
    p = Paged(attn, 21, [(1, 3000), (3, 900), (70, 20)], 2, 128, 16, torch.float16)
    q = randn(22, p.tokens, 8, 128).half().cuda()
    want = attn.littlebit_cache_attention_fwd(q, p.cache, p.batch)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(3):
        assert torch.equal(attn.littlebit_cache_attention_fwd(q, p.cache, p.batch), want)
        got = attn.littlebit_cache_attention_fwd(q, p.cache, p.batch, stream=side)
        side.synchronize()
        assert torch.equal(got, want)


def test_two_streams_at_once(attn):
    """Calls that overlap share nothing but what they read."""
    p = Paged(attn, 23, [(1, 3000), (3, 900)], 2, 128, 16, torch.float16)
    qs = [randn(i, 4, 8, 128).half().cuda() for i in range(2)]
    want = [attn.littlebit_cache_attention_fwd(q, p.cache, p.batch) for q in qs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in qs]
    got = [[], []]
    for _ in range(20):
        for i, s in enumerate(streams):
            got[i].append(attn.littlebit_cache_attention_fwd(qs[i], p.cache, p.batch, stream=s))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(g, want[i]) for g in got[i])


def test_one_captured_step_serves_any_lengths(attn):
    """Append and attention captured once for a padded batch; lengths, pages, rows and positions change between replays."""
    t, dim, kv, heads, page = torch.bfloat16, 128, 2, 8, 16
    p = Paged(attn, 24, [(1, 2000), (1, 2000), (1, 2000)], kv, dim, page, t, behind=1)
    other = Paged(attn, 24, [(1, 2000), (1, 2000), (1, 2000)], kv, dim, page, t, behind=1)
    q, k, v = (randn(i, 4, h, dim).to(t).cuda() for i, h in ((1, heads), (2, kv), (3, kv)))
    pos, inv = ints([0] * 4), inv_freq(dim).cuda()
    out, lse = torch.zeros(4, heads, dim, dtype=t, device="cuda"), torch.zeros(4, heads, device="cuda")

    def step(cache, batch, out, lse):
        turned = attn.littlebit_cache_append(cache, batch, k, v, q, pos, inv)
        attn.littlebit_cache_attention_fwd(turned, cache, batch, out=out, lse=lse)

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step(p.cache, p.batch, out, lse)
        step(other.cache, other.batch, out, lse)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(p.cache, p.batch, out, lse)
    rng = np.random.default_rng(5)
    for lens, starts in (([2001, 5, 900], [0, 1, 2, 3]), ([1, 1, 1], [0, 1, 2, 3]), ([2, 2001, 700], [1, 2, 2, 4]), ([300, 301, 1999], [0, 2, 3, 3])):
        case("replay", lens, starts)
        for x in (p, other):
            x.batch.lens.copy_(torch.tensor(lens))
            x.batch.starts.copy_(torch.tensor(starts))
        table = p.batch.table[torch.from_numpy(rng.permutation(3)).cuda()].clone()
        p.batch.table.copy_(table)
        other.batch.table.copy_(table)
        for x in (q, k, v):
            x.copy_(torch.from_numpy(rng.standard_normal(tuple(x.shape))))
        pos.copy_(torch.tensor([n - 1 for n in lens] + [3]))
        for c in (out, lse):
            c.fill_(9.0)
        want, want_lse = out.clone(), lse.clone()
        graph.replay()
        step(other.cache, other.batch, want, want_lse)
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(lse, want_lse)
        assert torch.equal(p.cache.k, other.cache.k) and torch.equal(p.cache.v, other.cache.v)


def test_a_captured_call_of_many_sequences(attn):
    """More than every workgroup adds up by itself, captured once; one with several parts, others shorter by the replay."""
    p = Paged(attn, 50, [(1, 20 + i % 60) for i in range(199)] + [(1, 2500)], 1, 64, 16, torch.float16)
    q = randn(51, p.tokens, 2, 64).half()
    q_gpu, out, lse = q.cuda(), torch.zeros(200, 2, 64, dtype=torch.float16, device="cuda"), torch.zeros(200, 2, device="cuda")
    call = lambda: attn.littlebit_cache_attention_fwd(q_gpu, p.cache, p.batch, out=out, lse=lse)  # noqa: E731
    with torch.cuda.stream(torch.cuda.Stream()):
        call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    full = p.lens.copy()
    for cut in (0, 1, 7, 1):
        case("replay", cut)
        p.lens[:] = np.maximum(full - cut * (np.arange(200) % 5) ** 2, 1)
        p.say()
        out.fill_(9.0)
        lse.fill_(9.0)
        graph.replay()
        check_attention(out, lse, q, p, 0.125)
        assert torch.equal(out, attn.littlebit_cache_attention_fwd(q_gpu, p.cache, p.batch))


def test_rope_captured_with_its_backward(attn):
    x, dy, w = (randn(i, 50, 4, 64).half().cuda() for i in (1, 2, 3))
    w = (1 + w[0, 0] / 4).contiguous()
    pos, inv = torch.arange(50).int().cuda(), inv_freq(64).cuda()

    def step():
        return attn.littlebit_rope_fwd(x, x, pos, inv, w, w) + attn.littlebit_rope_bwd(dy, dy, pos, inv, x, x, w, w)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for i in range(3):
        x.copy_(randn(10 + i, 50, 4, 64))
        graph.replay()
        want = step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_a_block_between_its_projections(attn):
    """LittleBitAttention: a prompt in two parts, then a tree, against the same steps on its projections' outputs."""
    from binary_rank_gemv_amd import littlebit as lb
    rng = np.random.default_rng(30)
    n, dim, heads, kv = 256, 64, 4, 2

    def layer(m, n):
        return lb.LittleBitLayer.from_latents([{"U": rng.standard_normal((m, 32)).astype(np.float32), "V": rng.standard_normal((n, 32)).astype(np.float32),
                                                "h": (rng.random(m) * 0.02).astype(np.float16), "l": rng.random(32).astype(np.float16),
                                                "g": rng.random(n).astype(np.float16)} for _ in range(2)])
    block = attn.LittleBitAttention(layer(heads * dim, n), layer(kv * dim, n), layer(kv * dim, n), layer(n, heads * dim), dim, inv_freq(dim).cuda(),
                                    q_norm=torch.ones(dim, dtype=torch.float16, device="cuda"))
    p = Paged(attn, 31, [(30, 0)], kv, dim, 16, torch.float16)
    x = randn(32, 37, n).half().cuda()
    words = [1, 3, 5, 0b1011, 0b10101, 0b100001, 0b1000101]
    depth = [0, 1, 1, 2, 2, 1, 2]
    for rows, before, tree, positions in ((20, 0, None, range(20)), (10, 20, None, range(20, 30)), (7, 30, words, [30 + d for d in depth])):
        case("block", rows, before)
        p.starts, p.lens = np.array([0, rows]), np.array([before + rows])
        p.batch = attn.CacheBatch(ints([0, rows]), ints([before + rows]), p.batch.table)
        xs = x[before:before + rows]
        y = block(xs, p.cache, p.batch, ints(list(positions)), None if tree is None else torch.tensor(tree).cuda())
        q = lb.littlebit_linear_fwd(block.q, xs).view(rows, heads, dim)
        k = lb.littlebit_linear_fwd(block.k, xs).view(rows, kv, dim)
        q, k = attn.littlebit_rope_fwd(q, k, ints(list(positions)), block.inv_freq, block.q_norm)
        a = oa.place(0, before, p.table, 16, p.cache.k.shape[0])
        assert torch.equal(p.cache.k[a[0], :, a[1]], k[0])
        out = attn.littlebit_cache_attention_fwd(q, p.cache, p.batch, None if tree is None else torch.tensor(tree).cuda())
        check_attention(out, None, q.cpu(), p, dim ** -0.5, tree)
        assert torch.equal(y, lb.littlebit_linear_fwd(block.o, out.view(rows, -1)))


def test_a_tensor_that_requires_a_gradient_is_refused(attn):
    p = Paged(attn, 40, [(1, 5)], 1, 64, 8, torch.float16)
    x = randn(1, 1, 1, 64).half().cuda().requires_grad_()
    y = x.detach()
    for call in (lambda: attn.littlebit_rope_fwd(x, None), lambda: attn.littlebit_rope_bwd(x, None), lambda: attn.littlebit_cache_append(p.cache, p.batch, x, y),
                 lambda: attn.littlebit_cache_append(p.cache, p.batch, y, x), lambda: attn.littlebit_cache_attention_fwd(x, p.cache, p.batch)):
        with pytest.raises(ValueError, match="requires a gradient"):
            call()
        with torch.no_grad():
            call()


def test_binding_refuses(attn):
    p = Paged(attn, 41, [(3, 5)], 2, 64, 8, torch.float16)
    x = randn(1, 3, 4, 64).half().cuda()
    kv = x[:, :2]
    w, pos, inv = torch.ones(64, dtype=torch.float16, device="cuda"), ints([0, 1, 2]), inv_freq(64).cuda()
    A, R, B = attn.littlebit_cache_attention_fwd, attn.littlebit_rope_fwd, attn.CacheBatch
    b = p.batch
    words = torch.ones(3, dtype=torch.int64, device="cuda")
    refused = [
        lambda: R(x.float(), None), lambda: R(x[0], None), lambda: R(x, x.bfloat16()), lambda: R(x, x[:2]), lambda: R(x, x[:, :, :32]), lambda: R(x, x.cpu()),
        lambda: R(x, None, pos.long(), inv), lambda: R(x, None, pos[:2], inv), lambda: R(x, None, pos, inv.double()), lambda: R(x, None, None, inv),
        lambda: R(x, None, q_weight=w[:32]), lambda: R(x, None, q_weight=w.float()), lambda: R(x, None, q_out=x[:, :2]), lambda: R(x, None, k_out=x),
        lambda: R(x[:, :, ::2], None), lambda: R(None, None),
        lambda: attn.littlebit_rope_bwd(x, None, q_weight=w), lambda: attn.littlebit_rope_bwd(x, None, q=kv, q_weight=w),
        lambda: attn.littlebit_cache_append(p.cache, b, x, x), lambda: attn.littlebit_cache_append(p.cache, b, kv, kv[:2]),
        lambda: attn.littlebit_cache_append(p.cache, b, kv, kv, q_out=x), lambda: attn.littlebit_cache_append(p.cache, b, kv.bfloat16(), kv),
        lambda: A(x.bfloat16(), p.cache, b), lambda: A(x[:, :3], p.cache, b), lambda: A(x, p.cache, b, tree=words.int()), lambda: A(x, p.cache, b, tree=words[:2]),
        lambda: A(x, p.cache, b, scale=float("inf")), lambda: A(x, p.cache, b, out=x), lambda: A(x, p.cache, b, lse=torch.empty(3, 3, device="cuda")),
        lambda: A(x, p.cache, B(b.starts[:1], b.lens, b.table)), lambda: A(x, p.cache, B(b.starts, b.lens.long(), b.table)),
        lambda: A(x, p.cache, B(b.starts, b.lens, b.table[0])), lambda: A(x, p.cache, B(b.starts, b.lens, b.table.cpu())),
        lambda: A(x, attn.LittleBitCache(p.cache.k, p.cache.v[:-1]), b), lambda: A(x, attn.LittleBitCache(p.cache.k[:, :, :7], p.cache.v[:, :, :7]), b),
        lambda: attn.littlebit_cache_accept(p.cache, b, ints([1])), lambda: attn.littlebit_cache_accept(p.cache, b, ints([[1], [2]])),
        lambda: attn.littlebit_cache_accept(p.cache, b, ints([[0] * 65])), lambda: attn.littlebit_cache_accept(p.cache, b, torch.ones(1, 2, device="cuda")),
    ]
    for i, call in enumerate(refused):
        with pytest.raises((ValueError, RuntimeError)):
            print("[refusal]", i, flush=True)
            call()


# ------------------------------------------------------------------------------------- long prompts among many others

class Packed(Paged):
    """The same with as many pages as the keys need; what the table names behind a sequence's keys is another's."""

    def __init__(self, attn, seed, counts, kv, dim, page, t):
        self.counts, self.page, self.t = counts, page, t
        rng = np.random.default_rng(seed)
        self.starts = np.concatenate([[0], np.cumsum([n for n, _ in counts])]).astype(int)
        self.lens = np.array([n + c for n, c in counts])
        self.tokens = int(self.starts[-1])
        used = -(-self.lens // page)
        pages = int(used.sum()) + 2
        order = rng.permutation(pages)
        self.table = rng.integers(0, pages, (len(counts), max(1, int(used.max()))))
        at = 0
        for i, n in enumerate(used):
            self.table[i, :n] = order[at:at + n]
            at += n
        shape = (pages, kv, page, dim)
        k, v = (torch.from_numpy(rng.standard_normal(shape, dtype=np.float32)).to(t).cuda() for _ in range(2))
        self.cache = attn.LittleBitCache(k, v)
        self.batch = attn.CacheBatch(ints(self.starts.tolist()), ints(self.lens.tolist()), ints(self.table.tolist()))


def check_sampled(out, lse, q, p, scale, picked):
    """check_attention of some rows: each, with the keys that it sees, as a sequence of its own."""
    place = oa.rows(p.starts, p.tokens)
    one = Packed.__new__(Packed)
    one.t, one.cache, one.page = p.t, p.cache, p.page
    one.starts = np.arange(len(picked) + 1)
    one.lens = np.array([p.lens[place[r][0]] - p.counts[place[r][0]][0] + place[r][1] + 1 for r in picked])
    one.table = p.table[[place[r][0] for r in picked]]
    check_attention(out[picked], lse[picked], q[picked], one, scale)


@pytest.mark.parametrize("counts,heads,kv,dim", [
    ([(5600, 3400)] + [(1, 999)] * 69, 4, 1, 64), ([(20000, 0)] + [(1, 0)] * 69, 1, 1, 64), ([(20000, 0)] + [(10, 0)] * 64, 1, 1, 64),
    ([(9000, 0)] + [(1, 69)] * 140, 2, 1, 64), ([(8192, 0)] + [(0, 0)] * 64, 4, 1, 128), ([(6000, 100)] + [(3, 37)] * 130, 4, 1, 256)])
def test_every_row_of_a_long_prompt_among_many_sequences(attn, counts, heads, kv, dim):
    for name, order in (("first", counts), ("last", counts[::-1])):
        case("long", name, counts[0], len(counts), heads, kv, dim)
        p = Packed(attn, dim, order, kv, dim, 64, torch.float16)
        q = randn(dim + 1, p.tokens, heads, dim, scale=1.5).to(p.t)
        out, lse = run_attention(attn, p, q)
        assert (lse != 55).all() and not (out == 55).all(2).any()   # no row was left out
        long = 0 if name == "first" else len(counts) - 1
        begin, end = p.starts[long], p.starts[long + 1]
        picked = sorted({0, 1, p.tokens - 1, begin, end - 1, *range(begin, end, 397), *range(0, p.tokens, p.tokens // 7)})
        check_sampled(out, lse, q, p, dim ** -0.5, picked)


def attend_in(attn, p, q, out, lse, ws):
    """The attention in a workspace of the caller's."""
    ref = attn._ref
    c, b = p.cache.c_struct(), p.batch.c_struct(0)
    h = [attn._Heads(t.data_ptr(), *t.stride()[:2], t.shape[1]) for t in (q, out)]
    attn._check(attn.LIB.littlebit_cache_attention_fwd(ref(c), ref(b), q.shape[0], ref(h[0]), None, q.shape[2] ** -0.5, ref(h[1]), lse.data_ptr(),
                                                       ws.data_ptr(), ws.numel(), attn._raw_stream(0)))


@pytest.mark.parametrize("rows,heads,dim", [(2, 4, 64), (60, 4, 128), (300, 2, 128)])
@pytest.mark.parametrize("seqs", [3, 70, 140])
def test_rows_of_no_sequence_are_not_joined_from_an_earlier_call(attn, rows, heads, dim, seqs):
    """A workspace that holds another call's parts for every row; sequences with a negative length, a negative start, or
    an end before their start have no rows then, and what they would name stays as it is."""
    counts = [(rows, 3000), (rows, 2900), (rows, 3100)] + [(1, 5)] * (seqs - 3)
    p = Packed(attn, 3, counts, 1, dim, 64, torch.bfloat16)
    q = randn(4, p.tokens, heads, dim).bfloat16().cuda()
    out, lse = torch.zeros_like(q), torch.zeros(p.tokens, heads, device="cuda")
    c, b = p.cache.c_struct(), p.batch.c_struct(0)
    ws = torch.zeros(attn.LIB.littlebit_cache_attention_workspace_bytes(attn._ref(c), attn._ref(b), p.tokens, heads), dtype=torch.uint8, device="cuda")
    attend_in(attn, p, q, out, lse, ws)
    full, full_lse = out.clone(), lse.clone()
    starts, lens = p.batch.starts.clone(), p.batch.lens.clone()
    for name, at, value, gone in (("length", 1, -1, range(rows, 2 * rows)), ("length", 0, -2 ** 31, range(rows)), ("start", 0, -3, range(rows)),
                                  ("start", 0, 2 ** 31 - 1, range(rows)), ("start", 2, rows - 1, range(rows - 1, 2 * rows))):
        case("no sequence", name, at, value)
        p.batch.starts.copy_(starts)
        p.batch.lens.copy_(lens)
        (p.batch.lens if name == "length" else p.batch.starts)[at] = value
        out.fill_(9.0)
        lse.fill_(9.0)
        attend_in(attn, p, q, out, lse, ws)
        left = torch.zeros(p.tokens, dtype=torch.bool, device="cuda")
        left[list(gone)] = True
        if value == rows - 1:   # the first sequence ends a row earlier, the third begins where the second did not
            assert (out[0:rows - 1] != 9).any(2).all() and torch.isfinite(out.float()).all()
            continue
        assert (out[left] == 9).all() and (lse[left] == 9).all()
        others = ~left
        # of other lengths of parts, perhaps: e of an output and of a probability on either side
        assert (out[others].float() - full[others].float()).abs().max() <= 4 * half_step(p.t) * p.cache.v.float().abs().max()
        assert (lse[others] - full_lse[others]).abs().max() <= 1e-3


@pytest.mark.parametrize("dt", list(TYPES))
@pytest.mark.parametrize("keys,size", [(30000, 1), (900, 512)])   # in many parts, with maxima of their own, and in one
@pytest.mark.parametrize("rows,heads,dim", [(1, 2, 64), (20, 1, 128), (3, 3, 256), (200, 1, 64), (150, 1, 256), (300, 1, 128)])
def test_a_key_that_outweighs_all_others(attn, rows, heads, dim, keys, size, dt):
    """The first key has nearly all of the softmax and a value of 0: the output is what the other keys add up to.  Half a step
    of the type each, e, beside that of the output; of fp16 at least half its smallest step, 2^-25, of probabilities whose
    largest is at least 2^14 (few rows) or 2^7 (many): 2^-39 or 2^-32 of it, for every key.  Sums of n terms: (n + 80) u."""
    t = TYPES[dt]
    for gap in (12.0, 20.0, 24.0, 25.2, 28.0):
        case("outweighed", rows, heads, dim, keys, dt, gap)
        p = Packed(attn, 60, [(rows, keys)], 1, dim, 64, t)
        p.cache.k.zero_()
        p.cache.v.abs_().mul_(size)
        at = oa.place(0, 0, p.table, 64, p.cache.k.shape[0])
        p.cache.k[at[0], 0, at[1], 0] = gap * np.log(2.0)
        p.cache.v[at[0], 0, at[1]] = 0
        q = torch.zeros(rows, heads, dim, dtype=t)
        q[:, :, 0] = 1.0
        out, lse = run_attention(attn, p, q, scale=1.0)
        sample = sorted({0, rows // 2, rows - 1})
        k, v = f64(p.cache.k), f64(p.cache.v)
        n = keys + rows
        lost = 0.0 if dt == "bf16" else 2.0 ** (-32 if rows * heads > 112 else -39)
        for r in sample:
            want, want_lse = oa.attention(f64(q[r:r + 1]), k, v, [0, 1], [keys + r + 1], p.table, 1.0)
            e, ds = half_step(t), (n + 80) * U
            assert want.min() > 2.0 ** -14   # no subnormal outputs
            bound = e * want + (1 + e) * ((e + 2 * ds) * want + n * lost * v.max())
            bad = np.abs(f64(out[r:r + 1]) - want) - bound
            assert (bad <= 0).all(), (gap, r, (np.abs(f64(out[r:r + 1]) - want) / want).max())
            assert np.abs(f64(lse[r:r + 1]) - want_lse).max() <= ds + 8 * U * np.abs(want_lse).max()


@pytest.mark.parametrize("rows", [1, 200])
@pytest.mark.parametrize("dt", list(TYPES))
def test_scores_of_many_millions(attn, rows, dt):
    """Neighbouring scores in fp32 are up to 16 apart here: one key has it all, and no probability leaves the type."""
    t, scale = TYPES[dt], 2.0 ** 10
    for big in (2.0 ** 5, 2.0 ** 7 + 2.0 ** 3, 2.0 ** 8, 2.0 ** 8 + 2.0 ** 7):
        case("millions", rows, dt, big)
        p = Packed(attn, 61, [(rows, 700)], 1, 64, 16, t)
        p.cache.k.zero_()
        q = torch.zeros(rows, 1, 64, dtype=t)
        q[:, :, 0] = 256.0
        for key, share in ((5, 0.5), (300, 0.75), (611, 1.0)):   # step by step to scores of `big` 2^18
            at = oa.place(0, key, p.table, 16, p.cache.k.shape[0])
            p.cache.k[at[0], 0, at[1], 0] = share * big
        out, lse = run_attention(attn, p, q, scale=scale)
        at = oa.place(0, 611, p.table, 16, p.cache.k.shape[0])
        # one probability of 1, in fp32: its product over its sum, rounded
        want = p.cache.v[at[0], 0, at[1]].double().cpu().numpy()
        assert (np.abs(f64(out) - want) <= (2 * half_step(t) + 4 * U) * np.abs(want)).all()
        score = scale * 256.0 * big
        assert (np.abs(f64(lse) - score) <= 16 * U * score).all()


@pytest.mark.parametrize("dt", list(TYPES))
@pytest.mark.parametrize("seqs,rows,heads,dim", [(40, 1, 4, 64), (12, 16, 1, 128), (6, 30, 1, 128), (10, 9, 2, 256), (8, 100, 1, 64), (6, 24, 2, 80)])
def test_few_rows_are_rounded_once(attn, seqs, rows, heads, dim, dt):
    """Of few rows nothing but the output is rounded to the type: beside that rounding what is computed in fp32 is small.  An
    output whose exact value lies within an error d of the middle between two neighbours a step s apart may fall to the other
    one: a share 2 d / s of them, a step off each, while roundings are s / sqrt(12) in the mean.  Here d is some 10 u of the
    values' mean size, which is up to 9 times the outputs' for 64 to 164 keys: 2 d / s below 180 u / 2^-11 = 0.022 for fp16,
    less for bf16.  (Probabilities of half a step e would be off by e / sqrt(3) each: d = e / 2, and a share of 1 / 4 and more.)"""
    t = TYPES[dt]
    case("rounded once", seqs, rows, heads, dim, dt)
    p = Paged(attn, 70, [(rows, 64)] * seqs, 1, dim, 16, t)
    q = randn(71, p.tokens, heads, dim, scale=0.3).to(t)
    out, _ = run_attention(attn, p, q)
    want, _ = oa.attention(f64(q), f64(p.cache.k), f64(p.cache.v), p.starts, p.lens, p.table, dim ** -0.5)
    nearest = f64(torch.from_numpy(want).to(t))
    rounding = np.sqrt(np.mean((nearest - want) ** 2))
    others = np.sqrt(np.mean((f64(out) - nearest) ** 2))
    print("others / rounding", others / rounding)
    assert others <= np.sqrt(0.022 * 12) * rounding


@pytest.mark.parametrize("dt", list(TYPES))
@pytest.mark.parametrize("rows,cached,heads,dim", [(1, 90, 1, 64), (1, 3000, 4, 128), (30, 700, 1, 128), (9, 400, 2, 256), (200, 1500, 1, 128)])
def test_an_infinite_value_that_all_rows_see_is_alone_in_its_channel(attn, rows, cached, heads, dim, dt):
    """That channel's outputs are that infinity, NaN for both signs; all others keep their bits."""
    case("alone", rows, cached, heads, dim, dt)
    p = Paged(attn, 72, [(rows, cached), (1, 40)], 1, dim, 16, TYPES[dt])
    q = randn(73, p.tokens, heads, dim, scale=0.3).to(p.t)
    clean, clean_lse = run_attention(attn, p, q)
    inf = float("inf")
    for key, channel, value in ((3, 9, inf), (cached // 2, 9, inf), (cached // 2, 30, -inf), (cached - 1, 41, inf), (0, 41, -inf), (64, 55, float("nan"))):
        a = oa.place(0, key, p.table, 16, p.cache.k.shape[0])
        p.cache.v[a[0], :, a[1], channel] = value
    out, lse = run_attention(attn, p, q)
    assert (out[:rows, :, 9] == inf).all() and (out[:rows, :, 30] == -inf).all() and torch.isnan(out[:rows, :, [41, 55]]).all()
    rest = [d for d in range(dim) if d not in (9, 30, 41, 55)]
    assert torch.equal(out[:rows, :, rest], clean[:rows, :, rest]) and torch.equal(out[rows:], clean[rows:]) and torch.equal(lse, clean_lse)


@pytest.mark.parametrize("dt", list(TYPES))
@pytest.mark.parametrize("rows,cached,heads,dim", [(7, 40, 2, 64), (7, 40, 1, 72), (30, 200, 1, 128), (9, 1200, 2, 256), (200, 100, 1, 64), (300, 40, 1, 128), (300, 4200, 2, 128), (150, 1030, 1, 256)])
def test_an_infinite_value_of_no_probability_is_not_a_number(attn, rows, cached, heads, dim, dt):
    """0 times infinity, as in the formula, in steps that all rows see and in those that some do: of keys whose score is
    -infinity.  Others give that infinity."""
    case("no probability", rows, cached, heads, dim, dt)
    t = TYPES[dt]
    p = Paged(attn, 80, [(rows, cached), (2, 9)], 1, dim, 8, t)
    q = randn(81, p.tokens, heads, dim, scale=0.5).abs().to(t)   # all scores of the keys below are of one sign
    inf = float("inf")
    for key, channel, k in ((3, 9, -inf), (cached + 1, 20, -inf), (cached + rows // 2, 33, -inf), (cached + rows - 2, 5, -inf), (cached + rows // 2 + 1, 50, 0.0)):
        a = oa.place(0, key, p.table, 8, p.cache.k.shape[0])
        p.cache.k[a[0], :, a[1]] = k
        p.cache.v[a[0], :, a[1], channel] = inf
    out, _ = run_attention(attn, p, q)
    with np.errstate(invalid="ignore"):
        want, _ = oa.attention(f64(q), f64(p.cache.k), f64(p.cache.v), p.starts, p.lens, p.table, dim ** -0.5)
    got = f64(out)
    assert np.isnan(want[rows - 1, :, [5, 9, 20, 33]]).all() and np.isposinf(want[rows - 1, :, 50]).all() and np.isfinite(want[0, :, [5, 20, 33]]).all()
    assert np.array_equal(np.isnan(got), np.isnan(want)) and np.array_equal(np.isposinf(got), np.isposinf(want))
    assert not np.isneginf(got).any()


def test_strides_that_no_address_uses(attn):
    """Those of a single page, head or token: keys and values may differ in them, and an output from its input in place."""
    for pages, heads, page in ((6, 1, 16), (1, 3, 64), (1, 1, 64)):
        case("unused strides", pages, heads)
        k, v = (randn(i, pages, heads, page, 64).half().cuda() for i in (1, 2))
        table = ints([list(range(pages))])
        batch = attn.CacheBatch(ints([0, 1]), ints([pages * page - 3]), table)
        q = randn(3, 1, 2 * heads, 64).half().cuda()
        want = attn.littlebit_cache_attention_fwd(q, attn.LittleBitCache(k, v), batch)
        odd = [5 if n == 1 else s for n, s in zip(k.shape, k.stride())]
        for a, b in ((k.as_strided(k.shape, odd), v), (k, v.as_strided(v.shape, odd)), (k.as_strided(k.shape, odd), v.as_strided(v.shape, odd))):
            assert torch.equal(attn.littlebit_cache_attention_fwd(q, attn.LittleBitCache(a, b), batch), want)
    w = torch.ones(64, dtype=torch.float16, device="cuda")
    for shape, strides in (((1, 3, 64), (1000, 64, 1)), ((4, 1, 64), (64, 7, 1)), ((1, 1, 64), (3, 9, 1))):
        x = randn(4, *shape).half().cuda()
        want, _ = attn.littlebit_rope_fwd(x, None, q_weight=w)
        dx, _, dw, _ = attn.littlebit_rope_bwd(x, None, q=x, q_weight=w)
        y = x.clone()
        got, _, dw2, _ = attn.littlebit_rope_bwd(x, None, q=y, q_weight=w, dq_in=y.as_strided(shape, strides))
        assert torch.equal(y, dx) and torch.equal(dw2, dw)
        attn.littlebit_rope_fwd(x, None, q_weight=w, q_out=x.as_strided(shape, strides))
        assert torch.equal(x, want)
    with pytest.raises(ValueError, match="strides"):
        attn.LittleBitCache(torch.empty(2, 1, 64, 64, dtype=torch.float16, device="cuda"), torch.empty(2, 1, 64, 72, dtype=torch.float16, device="cuda")[..., :64]).c_struct()
