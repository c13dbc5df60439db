"""GPU parity of the dense operators around the LittleBit layers against the
float64 reference (oracle/head.py).

Bounds are counted in roundings.  u = 2^-24 is half a step of fp32, e = half a
step of the output's type (eps / 2); sub is half its smallest subnormal.
* A sum of N terms in fp32, however it is grouped, is off by at most
  (longest chain of additions) * u * sum |terms|; a chain here is at most
  the elements a thread holds, plus 6 in a wave, plus the waves and parts.
* exp(d) from the hardware's base-2 exponential: d / ln 2 is rounded once, so
  its value is off by |d| u, plus 2 u of the instruction: (|d| + 2) * 2 u.
"""

import itertools

import numpy as np
import pytest
import torch

from oracle import head as oh

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
TYPES = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}
SUB = {torch.float32: 2.0 ** -150, torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134}


@pytest.fixture(scope="module")
def head():
    from binary_rank_gemv_amd import head
    return head


def half_step(t):
    return torch.finfo(t).eps / 2


def f64(t):
    return t.detach().cpu().double().numpy()


def rows_of(t, pad=0, offset=0):
    """The same values in rows `pad` elements further apart, `offset` elements into their buffer."""
    rows, n = t.shape
    buf = torch.full((rows * (n + pad) + offset + pad,), 77, dtype=t.dtype, device="cuda")
    v = buf[offset:offset + rows * (n + pad)].view(rows, n + pad)[:, :n]
    v.copy_(t)
    return v


def randn(seed, *shape, scale=1.0):
    return torch.from_numpy(np.random.default_rng(seed).standard_normal(shape) * scale)


def case(*what):
    print("[case]", *what, flush=True)


# ----------------------------------------------------------------------------------------------------------- norm

NORM_SHAPES = [(1, 1), (1, 7), (3, 8), (5, 100), (4, 512), (2, 513), (3, 2048), (2, 2056), (1, 4096), (1, 5120), (3, 8192),
               (2, 8200), (1, 16384), (2, 16385), (1, 32768), (530, 2500), (270, 5000)]


def chain(n):
    return 32 + 6 + 16 + 4   # at most 32 elements a thread, 6 in a wave, 16 waves, sqrt / division / products


@pytest.mark.parametrize("dt", ["fp16", "bf16"])
@pytest.mark.parametrize("rows,n", NORM_SHAPES)
def test_norm_forward(head, rows, n, dt):
    t = TYPES[dt]
    for residual, pad, offset in ((True, 0, 0), (False, 3, 1), (True, 8, 5)):
        case("norm", rows, n, dt, residual, pad, offset)
        x, r = randn(n, rows, n).to(t), randn(n + 1, rows, n, scale=3.0).to(t)
        w = (1 + 0.2 * randn(n + 2, n)).to(t)
        xd, rd = rows_of(x, pad, offset), rows_of(r, pad, offset) if residual else None
        q, scale, h1 = head.littlebit_rmsnorm_q8(xd, w.cuda(), rd)
        y, h2 = head.littlebit_rmsnorm_fwd(xd, w.cuda(), rd)
        torch.cuda.synchronize()
        want_h = (x.double() + r.double()).to(t) if residual else x
        assert torch.equal(h1.cpu(), want_h) and torch.equal(h2.cpu(), want_h)
        want = oh.rmsnorm(f64(want_h), f64(w), 1e-5)
        err = chain(n) * U
        e = half_step(t)
        assert (np.abs(f64(y) - want) <= (e + err * (1 + e)) * np.abs(want) + SUB[t]).all()
        s = oh.q8_scale(want)
        assert (np.abs(f64(scale) - s) <= err * s).all()
        # a code is within half a step of the value, and one more step only where the value's own error reaches
        codes = q.cpu().numpy().astype(np.float64)
        assert np.abs(codes).max() <= 127 and (np.abs(codes).max(axis=1) == 127).all()
        assert (np.abs(codes - want / s[:, None]) <= 0.5 + 127 * err).all()


@pytest.mark.parametrize("dt", ["fp16", "bf16"])
def test_norm_codes_are_the_exact_quotients_rounded(head, dt):
    """The products h w and their largest are exact in fp32, so the codes are those of
    the exact quotients.  The kernel decides by a remainder of at most 1/2 that is rounded
    twice, 2 * 2^-26 = 3e-8 of a step: quotients within 1e-7 of a half are left out."""
    case("norm codes", dt)
    t = TYPES[dt]
    x, w = randn(5, 300, 5000).to(t), (1 + 0.3 * randn(6, 5000)).to(t)
    q, _, _ = head.littlebit_rmsnorm_q8(x.cuda(), w.cuda())
    hw = f64(x) * f64(w)
    want = 127 * hw / np.abs(hw).max(1, keepdims=True)
    clear = np.abs(np.abs(want - np.trunc(want)) - 0.5) > 1e-7
    assert clear.mean() > 0.999
    assert np.array_equal(f64(q)[clear], np.rint(want)[clear])
    q, _ = head.littlebit_q8_quantize(x.float().cuda())
    want = 127 * f64(x) / np.abs(f64(x)).max(1, keepdims=True)
    clear = np.abs(np.abs(want - np.trunc(want)) - 0.5) > 1e-7
    assert np.array_equal(f64(q)[clear], np.rint(want)[clear])


@pytest.mark.parametrize("dt", list(TYPES))
def test_codes_of_quotients_that_are_halves_go_to_the_even_code(head, dt):
    """Rows of multiples of half a step: every second quotient is a half.  127 v and a are exact
    in float64, and their quotient, 31 by 24 bits, is a half or 2^-33 from one at least: the
    reference's codes are exact, none is left out."""
    case("codes of halves", dt)
    t = TYPES[dt]
    rng = np.random.default_rng(8)
    half = torch.from_numpy(rng.integers(-254, 255, (500, 1000)) / 2.0)
    half[:, 5] = 127.0
    unit = torch.from_numpy(rng.integers(129, 256, (500, 1)) / 128.0)          # 8 bits
    quotients = []
    if dt == "fp32":
        x = (half * unit).float()
        quotients.append((x.double(), head.littlebit_q8_quantize(x.cuda())[0]))
        x = randn(9, 500, 3000).float()
        quotients.append((x.double(), head.littlebit_q8_quantize(x.cuda())[0]))
    else:
        x = half.to(t)
        for i in range(0, 500, 50):
            w = unit[i].expand(1000).to(t).contiguous()
            quotients.append((x.double() * w.double(), head.littlebit_rmsnorm_q8(x.cuda(), w.cuda())[0]))
        x = randn(9, 2000, 5000).to(t)
        w = (1 + 0.3 * randn(10, 5000)).to(t)
        quotients.append((x.double() * w.double(), head.littlebit_rmsnorm_q8(x.cuda(), w.cuda())[0]))
    for v, q in quotients:
        v = v.numpy()
        want = np.rint(127 * v / np.abs(v).max(1, keepdims=True))
        assert np.array_equal(f64(q), want)


@pytest.mark.parametrize("n", [40, 1000, 3000, 5000, 9001, 20000])
@pytest.mark.parametrize("size,eps", [(1e25, 1e-5), (3e36, 1e-5), (1e-20, 0.0), (1e-37, 0.0)])
def test_norm_rows_whose_squares_leave_fp32(head, n, size, eps):
    """bf16 alone has such values; between them are ordinary rows, that keep their bits."""
    case("norm out of range", n, size, eps)
    t = torch.bfloat16
    x, dy = randn(n, 700, n).to(t), randn(n + 1, 700, n).to(t)
    plain = x.clone()
    far = torch.arange(700) % 7 == 3
    x[far] = (x[far].double() * size).to(t)
    w = (1 + 0.2 * randn(n + 2, n)).to(t)
    h, W, DY = f64(x), f64(w), f64(dy)
    want = oh.rmsnorm(h, W, eps)
    err = chain(n) * U
    e = half_step(t)
    y, _ = head.littlebit_rmsnorm_fwd(x.cuda(), w.cuda(), eps=eps)
    assert (np.abs(f64(y) - want) <= (e + err * (1 + e)) * np.abs(want) + SUB[t]).all()
    assert torch.equal(y[~far], head.littlebit_rmsnorm_fwd(plain.cuda(), w.cuda(), eps=eps)[0][~far])
    q, scale, _ = head.littlebit_rmsnorm_q8(x.cuda(), w.cuda(), eps=eps)
    s = oh.q8_scale(want)
    assert (np.abs(f64(scale) - s) <= err * s).all()
    assert (np.abs(f64(q) - want / s[:, None]) <= 0.5 + 127 * err).all()
    dx, dw = head.littlebit_rmsnorm_bwd(dy.cuda(), x.cuda(), w.cuda(), eps=eps)
    want_dx, want_dw = oh.rmsnorm_backward(DY, h, W, eps)
    r = 1 / np.sqrt((h * h).mean(1, keepdims=True) + eps)
    part = np.abs(h * r) * r * np.mean(np.abs(W * DY * (h * r)), 1, keepdims=True)
    bound = (chain(n) + 8) * U * (r * np.abs(W * DY) + 2 * part)
    held = np.abs(want_dx) < 1e38          # gradients beyond the type are infinite
    off = np.abs(f64(dx) - want_dx) <= half_step(t) * (np.abs(want_dx) + bound) + bound + SUB[t]
    assert off[held].all()
    assert (np.abs(f64(dw) - want_dw) <= (700 + chain(n) + 64) * U * np.abs(DY * h * r).sum(0)).all()
    assert torch.equal(dx[~far], head.littlebit_rmsnorm_bwd(dy.cuda(), plain.cuda(), w.cuda(), eps=eps)[0][~far])


def test_norm_rows_of_zeros_nan_and_infinity(head):
    case("norm special rows")
    x = torch.ones(5, 300, dtype=torch.float16)
    x[0] = 0
    x[1, 7] = float("nan")
    x[2, 299] = float("inf")
    x[3] = 6e-8          # the smallest subnormal
    q, scale, _ = head.littlebit_rmsnorm_q8(x.cuda(), torch.ones(300, dtype=torch.float16, device="cuda"), eps=0.0)
    assert scale[1].isnan() and scale[2].isnan() and (q[1:3] == 0).all()
    assert scale[0].isnan() and (q[0] == 0).all()     # 0 / sqrt(0): without eps a row of zeros has no norm
    assert (q[3:] == 127).all() and torch.allclose(scale[3:], torch.tensor(1 / 127.0, device="cuda"), rtol=60 * U)
    q, scale, _ = head.littlebit_rmsnorm_q8(x[:1].cuda(), torch.ones(300, dtype=torch.float16, device="cuda"))
    assert scale[0] == 0 and (q == 0).all()
    y, _ = head.littlebit_rmsnorm_fwd(x[1:3].cuda(), torch.ones(300, dtype=torch.float16, device="cuda"))
    assert y[0].isnan().all() and y[1, 299].isnan() and (y[1, :299] == 0).all()
    # an fp16 sum beyond the type's range is an infinity of the stored hidden state
    big = torch.full((1, 8), 60000.0, dtype=torch.float16, device="cuda")
    _, scale, h = head.littlebit_rmsnorm_q8(big, torch.ones(8, dtype=torch.float16, device="cuda"), big)
    assert h.isinf().all() and scale.isnan().all()


@pytest.mark.parametrize("dt", ["fp16", "bf16"])
@pytest.mark.parametrize("n", [300, 2000, 5000, 9000, 20000])
def test_norm_of_a_weight_with_nan_or_infinity(head, n, dt):
    """A product h w that is NaN or infinite leaves no finite scale, wherever in the row it is,
    and the dense output holds it."""
    case("norm weight special", n, dt)
    t = TYPES[dt]
    x = randn(n, 4, n).to(t)
    for place in (0, n // 2, n - 1):
        for bad in (float("nan"), float("inf"), -float("inf")):
            x[:, place] = torch.tensor([1.0, 0.0, -2.0, 0.0])
            w = torch.ones(n, dtype=t)
            w[place] = bad
            q, scale, _ = head.littlebit_rmsnorm_q8(x.cuda(), w.cuda())
            y, _ = head.littlebit_rmsnorm_fwd(x.cuda(), w.cuda())
            assert scale.isnan().all() and (q == 0).all()
            with np.errstate(invalid="ignore"):
                want = f64(x)[:, place] * bad
            got = f64(y)[:, place]
            assert np.array_equal(np.isnan(got), np.isnan(want)) and (got[~np.isnan(want)] == want[~np.isnan(want)]).all()
            rest = torch.arange(n) != place
            assert torch.isfinite(y.cpu()[:, rest]).all()


def test_norm_hidden_in_place_and_untouched_surroundings(head):
    case("norm in place")
    t = torch.bfloat16
    x, r = randn(0, 9, 130).to(t), randn(1, 9, 130).to(t)
    w = torch.ones(130, dtype=t, device="cuda")
    for pick in (0, 1):
        buf = torch.full((9 * 150 + 20,), 5.0, dtype=t, device="cuda")
        views = [rows_of(x, 20), rows_of(r, 20)]
        inner = buf[10:10 + 9 * 150].view(9, 150)[:, :130]
        inner.copy_(views[pick])
        views[pick] = inner
        y, h = head.littlebit_rmsnorm_fwd(views[0], w, views[1], hidden=inner)
        assert h.data_ptr() == inner.data_ptr()
        assert torch.equal(inner.cpu(), (x.double() + r.double()).to(t))
        outside = torch.ones_like(buf, dtype=torch.bool)
        outside[10:10 + 9 * 150].view(9, 150)[:, :130] = False
        assert (buf[outside] == 5).all()
        assert torch.equal(y, head.littlebit_rmsnorm_fwd(x.cuda(), w, r.cuda())[0])


@pytest.mark.parametrize("dt", ["fp16", "bf16"])
@pytest.mark.parametrize("rows,n", [(1, 1), (2, 7), (3, 100), (5, 2048), (700, 300), (1500, 64), (3, 4096), (2, 5000),
                                    (2, 8192), (3, 9001), (2, 16384), (2, 32768)])
def test_norm_backward(head, rows, n, dt):
    t = TYPES[dt]
    for with_dh, pad, offset in ((True, 0, 0), (False, 8, 0), (True, 5, 3)):
        case("norm backward", rows, n, dt, with_dh, pad, offset)
        h, dy, dh = (randn(n + i, rows, n, scale=s).to(t) for i, s in ((0, 2.0), (1, 0.5), (2, 0.5)))
        w = (1 + 0.2 * randn(n + 3, n)).to(t)
        dx, dw = head.littlebit_rmsnorm_bwd(rows_of(dy, pad, offset), rows_of(h, pad, offset), w.cuda(),
                                            rows_of(dh, pad, offset) if with_dh else None)
        torch.cuda.synchronize()
        H, DY, W = f64(h), f64(dy), f64(w)
        want_dx, want_dw = oh.rmsnorm_backward(DY, H, W, 1e-5, f64(dh) if with_dh else None)
        r = 1 / np.sqrt((H * H).mean(1, keepdims=True) + 1e-5)
        part = np.abs(H) * r ** 3 * np.mean(np.abs(W * DY * H), 1, keepdims=True)
        size = r * np.abs(W * DY) + 2 * part + (np.abs(f64(dh)) if with_dh else 0)
        err = (chain(n) + 8) * U * size
        assert (np.abs(f64(dx) - want_dx) <= half_step(t) * (np.abs(want_dx) + err) + err + SUB[t]).all()
        # dweight: a group's rows in turn, 32 slices of groups, 32 of those
        terms = np.abs(DY * H * r).sum(0)
        assert (np.abs(f64(dw) - want_dw) <= (rows + chain(n) + 64) * U * terms).all()


@pytest.mark.parametrize("dt", ["fp16", "bf16"])
@pytest.mark.parametrize("rows,n", [(5, 300), (900, 1000), (600, 4000), (300, 5000), (3, 9000), (300, 20000)])
def test_norm_to_both_outputs(head, rows, n, dt):
    """y and q of one call are those of the two calls, ordinary rows and those out of range."""
    case("norm, both outputs", rows, n, dt)
    t = TYPES[dt]
    x, r, w = randn(1, rows, n).to(t).cuda(), randn(2, rows, n).to(t).cuda(), (1 + 0.2 * randn(3, n)).to(t).cuda()
    if dt == "bf16":
        x[::3] *= 1e25
        x[1::7] *= 1e35
        r[1::7] = 0
    y, h = head.littlebit_rmsnorm_fwd(x, w, r)
    q, scale, _ = head.littlebit_rmsnorm_q8(x, w, r)
    both = [torch.empty_like(h), torch.empty_like(y), torch.empty(rows, n, dtype=torch.int8, device="cuda"), torch.empty_like(scale)]
    status = head.LIB.littlebit_rmsnorm_fwd(
        x.data_ptr(), n, r.data_ptr(), n, w.data_ptr(), head._DTYPE[t], rows, n, 1e-5, both[0].data_ptr(), n,
        both[1].data_ptr(), n, both[2].data_ptr(), n, both[3].data_ptr(), torch.cuda.current_stream().cuda_stream)
    assert status == 0
    torch.cuda.synchronize()
    for got, want in zip(both, (h, y, q, scale)):     # NaN where both factors reached a row
        assert torch.allclose(got, want, rtol=0, atol=0, equal_nan=True)


@pytest.mark.parametrize("dt", ["fp16", "bf16"])
@pytest.mark.parametrize("rows,n", [(5, 300), (5000, 100), (3000, 1000), (1500, 4000), (700, 5000), (600, 9000), (600, 20000)])
def test_norm_backward_in_place(head, rows, n, dt):
    """dx may be dy, dhidden or hidden itself: many rows a workgroup, whose loads run ahead."""
    case("norm backward in place", rows, n, dt)
    t = TYPES[dt]
    dy, dh, h = (torch.randn(rows, n, device="cuda").to(t) for _ in range(3))
    if dt == "bf16":
        h[::5] *= 1e25
    w = (1 + 0.2 * randn(3, n)).to(t).cuda()
    want, want_dw = head.littlebit_rmsnorm_bwd(dy, h, w, dh)
    need = head.LIB.littlebit_rmsnorm_bwd_workspace_bytes(rows, n)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    for place in range(3):
        args = [t_.clone() for t_ in (dy, dh, h)]
        dw = torch.empty(n, device="cuda")
        status = head.LIB.littlebit_rmsnorm_bwd(
            args[0].data_ptr(), n, args[1].data_ptr(), n, args[2].data_ptr(), n, w.data_ptr(), head._DTYPE[t], rows, n, 1e-5,
            args[place].data_ptr(), n, dw.data_ptr(), ws.data_ptr(), need, torch.cuda.current_stream().cuda_stream)
        assert status == 0
        torch.cuda.synchronize()
        assert torch.equal(args[place], want) and torch.equal(dw, want_dw)


def test_norm_backward_no_rows(head):
    case("norm backward of no rows")
    e = torch.empty(0, 50, dtype=torch.float16, device="cuda")
    dx, dw = head.littlebit_rmsnorm_bwd(e, e, torch.ones(50, dtype=torch.float16, device="cuda"))
    assert dx.shape == (0, 50) and (dw == 0).all()


def test_norm_backward_repeats_bit_for_bit(head):
    case("norm backward twice")
    h, dy = randn(0, 3000, 520).bfloat16().cuda(), randn(1, 3000, 520).bfloat16().cuda()
    w = torch.ones(520, dtype=torch.bfloat16, device="cuda")
    a = head.littlebit_rmsnorm_bwd(dy, h, w)
    b = head.littlebit_rmsnorm_bwd(dy, h, w)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


# ------------------------------------------------------------------------------------------------------- quantiser

@pytest.mark.parametrize("dt", ["fp32", "fp16", "bf16"])
@pytest.mark.parametrize("rows,n", [(1, 1), (3, 5), (2, 512), (3, 1000), (2, 4100), (1, 8192), (2, 20000)])
def test_quantize(head, rows, n, dt):
    t = TYPES[dt]
    for pad, offset in ((0, 0), (3, 1)):
        case("quantize", rows, n, dt, pad, offset)
        x = randn(n, rows, n).to(t)
        q, scale = head.littlebit_q8_quantize(rows_of(x, pad, offset))
        s = oh.q8_scale(f64(x))
        assert (np.abs(f64(scale) - s) <= U * s).all()
        # 127 / max and the product with it: two roundings
        assert (np.abs(f64(q) - f64(x) / s[:, None]) <= 0.5 + 127 * 3 * U).all()


def test_quantize_ends_of_the_range(head):
    case("quantize special rows")
    x = torch.zeros(6, 40)
    x[1] = 1e-38 * torch.arange(40)
    x[2, 3] = float("inf")
    x[3, 39] = float("nan")
    x[4] = 3e38
    x[5] = -1e-45
    q, scale = head.littlebit_q8_quantize(x.cuda())
    assert scale[0] == 0 and (q[0] == 0).all()
    want = torch.round(x[1].double() / x[1].double().max() * 127)
    assert (q[1].cpu().double() - want).abs().max() <= 1
    assert scale[2].isnan() and scale[3].isnan() and (q[2:4] == 0).all()
    assert (q[4] == 127).all() and torch.isfinite(scale[4])
    assert (q[5] == -127).all()


# ------------------------------------------------------------------------------------------------------ 8-bit product

LINEAR = [(1, 1, 1), (1, 16, 64), (2, 17, 65), (3, 100, 128), (16, 33, 1000), (17, 64, 256), (31, 130, 320), (64, 48, 2048),
          (65, 129, 512), (100, 200, 511), (128, 256, 1024), (130, 300, 640), (257, 513, 192), (300, 1000, 4096),
          (520, 768, 128), (1, 4096, 13824), (5, 32000, 320), (16, 4500, 272), (7, 9001, 144), (3, 8200, 130), (1, 4112, 16),
          (16, 4200, 9600), (2, 33000, 48), (12, 4128, 4096), (40, 1100, 200), (90, 4300, 390), (260, 9000, 256), (600, 9000, 384)]


@pytest.mark.parametrize("batch,m,n", LINEAR)
def test_q8_linear(head, batch, m, n):
    rng = np.random.default_rng(batch + m + n)
    xq = torch.from_numpy(rng.integers(-128, 128, (batch, n), dtype=np.int8))
    wq = torch.from_numpy(rng.integers(-128, 128, (m, n), dtype=np.int8))
    xs = torch.from_numpy(rng.uniform(0.01, 0.1, batch).astype(np.float32))
    ws = torch.from_numpy((rng.uniform(0.5, 1.5, m) / (60 * np.sqrt(n))).astype(np.float32))
    want = oh.q8_linear(xq.numpy(), xs.numpy(), wq.numpy(), ws.numpy())
    for dt, (pad, offset) in itertools.product(TYPES, ((0, 0), (16, 16), (3, 1))):
        case("q8 linear", batch, m, n, dt, pad, offset)
        t = TYPES[dt]
        buf = torch.full((batch * (m + pad) + 2 * pad,), 9.0, dtype=t, device="cuda")
        out = buf[pad:pad + batch * (m + pad)].view(batch, m + pad)[:, :m]
        got = head.littlebit_q8_linear_fwd(rows_of(xq, pad, offset), xs.cuda(), rows_of(wq, pad, offset), ws.cuda(),
                                           out=out)
        torch.cuda.synchronize()
        # the sum as fp32, the scales' product, their product, the output
        assert (np.abs(f64(got) - want) <= (3 * U + half_step(t) * (1 + 4 * U)) * np.abs(want) + SUB[t]).all()
        outside = torch.ones_like(buf, dtype=torch.bool)
        outside[pad:pad + batch * (m + pad)].view(batch, m + pad)[:, :m] = False
        assert (buf[outside] == 9).all()


def test_q8_linear_at_the_largest_sum(head):
    case("q8 linear, largest sums")
    n = 131071
    x = torch.full((2, n), -128, dtype=torch.int8, device="cuda")
    w = torch.full((3, n), -128, dtype=torch.int8, device="cuda")
    w[1] = 127
    one = torch.ones(3, device="cuda")
    y = head.littlebit_q8_linear_fwd(x, one[:2], w, one, dtype=torch.float32)
    want = torch.tensor([128.0 * 128 * n, -128.0 * 127 * n, 128.0 * 128 * n], dtype=torch.float64).float()
    assert (y.cpu() == want).all()


def test_q8_linear_codes_of_other_rows_do_not_reach_a_row(head):
    """A padded batch: each token's output depends on its own codes alone."""
    case("q8 linear rows")
    rng = np.random.default_rng(0)
    xq = torch.from_numpy(rng.integers(-127, 128, (150, 512), dtype=np.int8)).cuda()
    wq = torch.from_numpy(rng.integers(-127, 128, (200, 512), dtype=np.int8)).cuda()
    xs, ws = torch.rand(150, device="cuda"), torch.rand(200, device="cuda")
    xs[7] = float("nan")
    y = head.littlebit_q8_linear_fwd(xq, xs, wq, ws, dtype=torch.float32)
    for t in (0, 6, 8, 149):
        one = head.littlebit_q8_linear_fwd(xq[t:t + 1], xs[t:t + 1], wq, ws, dtype=torch.float32)
        assert torch.equal(one[0], y[t])
    assert y[7].isnan().all()


# --------------------------------------------------------------------------------------------------- log probabilities

def check_logprobs(head, x, targets, top, what, pad=0, offset=0):
    """x: CPU tensor of logits."""
    case("logprobs", what, tuple(x.shape), x.dtype, top, pad, offset)
    xd = rows_of(x, pad, offset)
    lp, H, parts, tv, ti = head.littlebit_logprobs_fwd(xd, targets.cuda(), top)
    torch.cuda.synchronize()
    lse = parts.sum(0)
    X = f64(x)
    logp, wantH = oh.logprobs(X)
    want_lse = oh.logsumexp(X)
    fine = np.isfinite(want_lse)
    p = np.exp(logp)
    far = np.where(p > 0, np.abs(np.where(p > 0, X, 0) - np.where(fine, X.max(1), 0)[:, None]), 0)
    mean_far = (p * far).sum(1)
    # chain of additions of a thread, a wave, the waves, the parts, and of a move to a new maximum a chunk
    n = x.shape[1] / 256 + 16 + 6 + 4 + 32 + 2 * (x.shape[1] / 4096 + 1)
    rel = (n + 4 + 2 * mean_far) * U                      # of the sum of exponentials
    wl = np.where(fine, want_lse, 0)
    tol = 2 * rel + 4 * U * (np.abs(wl) + np.abs(np.where(fine, X.max(1), 0))) + 8 * U
    assert (np.abs(f64(lse) - wl)[fine] <= tol[fine]).all()
    assert (np.isneginf(f64(lse)) == np.isneginf(want_lse)).all()
    tolH = 2 * rel * (1 + 2 * mean_far) + 8 * U * (1 + wantH)
    assert (np.abs(f64(H) - wantH) <= tolH).all()
    tg = targets.numpy()
    for i in range(len(tg)):
        if tg[i] < 0:
            assert lp[i] == 0
        else:
            want = logp[i, tg[i]]
            assert (f64(lp[i]) == want if np.isneginf(want) else abs(f64(lp[i]) - want) <= tol[i] + 2 * U * abs(want))
    if top:
        places = oh.top(X, top)
        assert np.array_equal(ti.cpu().numpy(), places)
        want = np.take_along_axis(logp, places, 1)
        got = f64(tv)
        inf = np.isneginf(want)
        assert (np.isneginf(got) == inf).all()
        assert (np.abs(got - np.where(inf, 0, want))[~inf] <= (tol[:, None] + 2 * U * np.abs(np.where(inf, 0, want)))[~inf]).all()
    else:
        assert tv is None and ti is None
    return xd, lp, H, parts, tv, ti


def targets_of(seed, rows, vocab):
    t = torch.from_numpy(np.random.default_rng(seed).integers(0, vocab, rows))
    t[::5] = -100
    return t


@pytest.mark.parametrize("dt", list(TYPES))
@pytest.mark.parametrize("rows,vocab,top", [(1, 1, 1), (3, 2, 2), (4, 17, 17), (2, 64, 64), (5, 1000, 3), (2, 4096, 64),
                                            (3, 4097, 20), (1, 8191, 1), (7, 12345, 33), (2, 32000, 5), (1, 100003, 64),
                                            (600, 5000, 7), (1030, 300, 2), (3, 32000, 0)])
def test_logprobs(head, rows, vocab, top, dt):
    for pad, offset in ((0, 0), (3, 1)):
        x = randn(vocab + rows, rows, vocab, scale=3.0).to(TYPES[dt])
        check_logprobs(head, x, targets_of(rows, rows, vocab), top, "random", pad, offset)


@pytest.mark.parametrize("dt", list(TYPES))
@pytest.mark.parametrize("kind", ["equal", "few values", "rising", "falling", "masked", "one left", "nothing left",
                                  "lowest", "far apart", "zeros of both signs", "peak"])
def test_logprobs_hard_rows(head, kind, dt):
    t, vocab, top = TYPES[dt], 9001, 20
    low = torch.finfo(t).min
    rng = np.random.default_rng(5)
    x = randn(9, 3, vocab, scale=2.0)
    if kind == "equal":
        x[:] = 1.25
    elif kind == "few values":
        x = torch.from_numpy(rng.integers(0, 3, (3, vocab)).astype(np.float64))
    elif kind == "rising":
        x = torch.linspace(-8, 8, vocab, dtype=torch.float64).repeat(3, 1)
    elif kind == "falling":
        x = torch.linspace(8, -8, vocab, dtype=torch.float64).repeat(3, 1)
    elif kind == "masked":
        x[:, ::2] = -np.inf
        x[1, 5:] = -np.inf          # fewer left than are asked for
    elif kind == "one left":
        x[:] = -np.inf
        x[0, 0] = x[1, 4096] = x[2, vocab - 1] = 3.0
    elif kind == "nothing left":
        x[1] = -np.inf
    elif kind == "lowest":
        x[:, 1:] = low
        x[1] = low
    elif kind == "far apart":
        x *= 2000.0
    elif kind == "zeros of both signs":
        x[:] = 0.0
        x[:, ::3] = -0.0
    elif kind == "peak":
        x[:, 77] = 60.0
    check_logprobs(head, x.to(t), torch.tensor([4, 77, 9000]), top, kind)


def test_logprobs_nan_and_infinity(head):
    case("logprobs nan")
    x = randn(1, 4, 5000).float()
    x[0, 40] = float("nan")
    x[0, 4500] = -float("nan")
    x[1, 4999] = float("inf")
    targets = torch.tensor([0, 1, 5000, 2])
    lp, H, lse, tv, ti = head.littlebit_logprobs_fwd(x.cuda(), targets.cuda(), 4)
    assert lp[:3].isnan().all() and H[:2].isnan().all() and lse.sum(0)[:2].isnan().all()
    assert torch.isfinite(lp[3]) and torch.isfinite(H[2:]).all()
    assert np.array_equal(ti.cpu().numpy(), oh.top(f64(x), 4))


def test_logprobs_without_targets(head):
    case("logprobs without targets")
    x = randn(1, 4, 5000).half().cuda()
    a = head.littlebit_logprobs_fwd(x, None, 3)
    b = head.littlebit_logprobs_fwd(x, torch.zeros(4, dtype=torch.int64, device="cuda"), 3)
    assert a[0] is None and all(torch.equal(p, q) for p, q in zip(a[1:], b[1:]))


@pytest.mark.parametrize("rows,vocab,top", [(5, 1000, 0), (3, 9001, 7), (2, 100003, 5)])
def test_logprobs_without_entropy_or_targets(head, rows, vocab, top):
    """What is not asked for is not written; the rest is the same."""
    case("logprobs, NULL outputs", rows, vocab, top)
    x, targets = randn(1, rows, vocab).half().cuda(), targets_of(2, rows, vocab).cuda()
    want = head.littlebit_logprobs_fwd(x, targets, top)
    need = head.LIB.littlebit_logprobs_workspace_bytes(rows, vocab, head._DTYPE[x.dtype], top)
    for with_targets in (True, False):
        lp, lse = torch.full((rows,), 7.0, device="cuda"), torch.empty(2, rows, device="cuda")
        tv = torch.empty(rows, max(top, 1), device="cuda")
        ti = torch.empty(rows, max(top, 1), dtype=torch.int64, device="cuda")
        ws = torch.empty(need + 16, dtype=torch.uint8, device="cuda")
        status = head.LIB.littlebit_logprobs_fwd(
            x.data_ptr(), vocab, head._DTYPE[x.dtype], rows, vocab, targets.data_ptr() if with_targets else None,
            lp.data_ptr() if with_targets else None, None, lse.data_ptr(), top, tv.data_ptr() if top else None,
            ti.data_ptr() if top else None, ws.data_ptr() if need else None, need, torch.cuda.current_stream().cuda_stream)
        assert status == 0
        torch.cuda.synchronize()
        assert torch.equal(lse, want[2]) and (torch.equal(lp, want[0]) if with_targets else (lp == 7).all())
        if top:
            assert torch.equal(tv, want[3]) and torch.equal(ti, want[4])


@pytest.mark.parametrize("dt", list(TYPES))
@pytest.mark.parametrize("rows,vocab,top", [(1, 1, 1), (3, 2, 0), (4, 17, 5), (5, 1000, 64), (2, 8192, 4), (3, 8193, 3),
                                            (7, 20011, 0), (2, 50257, 20)])
def test_logprobs_backward(head, rows, vocab, top, dt):
    t = TYPES[dt]
    rng = np.random.default_rng(rows + vocab)
    for pad, offset, use in ((0, 0, "all"), (3, 1, "all"), (0, 0, "token"), (0, 0, "entropy")):
        x = randn(vocab, rows, vocab, scale=2.0).to(t)
        x[:, vocab // 2] = -np.inf if vocab > 2 else x[:, 0]
        targets = targets_of(rows, rows, vocab)
        xd, lp, H, lse, tv, ti = check_logprobs(head, x, targets, top, use, pad, offset)
        if top and use == "all":
            targets = torch.where(targets >= 0, ti[:, 0].cpu(), targets)       # the target is an alternative too
        g = torch.from_numpy(rng.standard_normal((2, rows)).astype(np.float32)).cuda()
        gt = torch.from_numpy(rng.standard_normal((rows, top)).astype(np.float32)).cuda() if top and use == "all" else None
        dlp, dH = (g[0] if use != "entropy" else None), (g[1] if use != "token" else None)
        case("logprobs backward", rows, vocab, top, dt, pad, use)
        d = head.littlebit_logprobs_bwd(xd, targets.cuda(), lse, H, dlp, dH, ti if gt is not None else None, gt)
        torch.cuda.synchronize()
        X = f64(x)
        want = oh.logprobs_backward(X, targets.numpy(), f64(dlp) if dlp is not None else None,
                                    f64(dH) if dH is not None else None, ti.cpu().numpy() if gt is not None else None,
                                    f64(gt) if gt is not None else None)
        logp, ent = oh.logprobs(X)
        p = np.exp(logp)
        y = np.where(p > 0, logp, 0)
        a = (np.abs(f64(dlp))[:, None] if dlp is not None else 0) + (np.abs(f64(gt)).sum(1, keepdims=True) if gt is not None else 0)
        b = np.abs(f64(dH))[:, None] if dH is not None else 0
        # lse and H are off as in the forward test: 3e-5 of 1 covers vocab / 256 additions of 50257; exp as above
        off = (vocab / 256 + 100) * U + 4 * U * (np.abs(y) + np.abs(np.where(p > 0, X, 0)) + np.abs(oh.logsumexp(X))[:, None])
        err = p * (2 * off * (a + b * (np.abs(y) + ent[:, None])) + b * (off * 8 * (1 + ent[:, None])) + 70 * U * a)
        err = err + 70 * U * (np.abs(want) + a * (p > 0))
        assert (np.abs(f64(d) - want) <= half_step(t) * (np.abs(want) + err) + err + SUB[t]).all()
        # in place, the same bits
        head.littlebit_logprobs_bwd(xd, targets.cuda(), lse, H, dlp, dH, ti if gt is not None else None, gt, out=xd)
        assert torch.equal(xd.cpu(), d.cpu())


def test_logprobs_backward_special_rows(head):
    case("logprobs backward special rows")
    x = randn(2, 4, 700).float()
    x[0] = -np.inf
    x[1, 3] = -np.inf
    targets = torch.tensor([2, 3, -100, 700]).cuda()
    lp, H, lse, tv, ti = head.littlebit_logprobs_fwd(x.cuda(), targets, 2)
    one = torch.ones(4, device="cuda")
    d = head.littlebit_logprobs_bwd(x.cuda(), targets, lse, H, one, None, ti, torch.zeros(4, 2, device="cuda"))
    assert (d[0] == 0).all()                       # nothing left: no gradient
    assert d[1, 3] == 1 and lp[1] == -np.inf       # a masked token: its own direct gradient, p is 0
    assert (d[2] == 0).all() and d[3].isnan().all()


@pytest.mark.parametrize("dt", list(TYPES))
def test_logprobs_backward_of_rows_masked_with_the_lowest_value(head, dt):
    """Equals, however far from 0: p is 1 / vocab everywhere, exact but for exp and log (8 U each)."""
    case("logprobs backward, lowest", dt)
    t = TYPES[dt]
    x = torch.full((2, 1000), torch.finfo(t).min, dtype=t)
    x[1, 7] = 0.0
    targets = torch.tensor([3, 7]).cuda()
    lp, H, lse, _, _ = head.littlebit_logprobs_fwd(x.cuda(), targets)
    d = head.littlebit_logprobs_bwd(x.cuda(), targets, lse, H, torch.ones(2, device="cuda"), torch.ones(2, device="cuda"))
    want = -torch.full((1000,), 1e-3, dtype=torch.float64)
    want[3] += 1
    assert ((d[0].cpu().double() - want).abs() <= (half_step(t) + 40 * U) * want.abs() + 40 * U * 1e-3 + SUB[t]).all()
    assert (d[1] == 0).all() and lp[1] == 0 and H[1] == 0
    assert abs(lp[0].item() + np.log(1000)) <= 8 * U * 7 and abs(H[0].item() - np.log(1000)) <= 40 * U * 7


def test_logprobs_backward_of_a_place_given_twice(head):
    """The target among the alternatives, and one alternative given twice: every gradient counts."""
    case("logprobs backward, places twice")
    x = randn(3, 2, 50)
    targets = torch.tensor([7, 7])
    lp, H, lse, _, _ = head.littlebit_logprobs_fwd(x.float().cuda(), targets.cuda())
    idx = torch.tensor([[7, 9, 9], [0, 49, 0]])
    g, gt = torch.tensor([0.5, -1.0]), torch.tensor([[1.0, 2.0, 3.0], [0.25, 0.5, 0.75]])
    d = head.littlebit_logprobs_bwd(x.float().cuda(), targets.cuda(), lse, None, g.cuda(), None, idx.cuda(), gt.cuda())
    want = oh.logprobs_backward(f64(x.float()), targets.numpy(), g.numpy(), None, idx.numpy(), gt.numpy())
    assert np.abs(f64(d) - want).max() <= 100 * U * 8


def test_logprobs_backward_leaves_what_lies_between_rows(head):
    case("logprobs backward, surroundings")
    buf = torch.full((5 * 140 + 20,), 3.0, dtype=torch.float16, device="cuda")
    out = buf[10:10 + 5 * 140].view(5, 140)[:, :133]
    x = randn(8, 5, 133).half().cuda()
    targets = torch.arange(5, device="cuda")
    lp, H, lse, _, _ = head.littlebit_logprobs_fwd(x, targets)
    one = torch.ones(5, device="cuda")
    got = head.littlebit_logprobs_bwd(x, targets, lse, H, one, one, out=out)
    assert got.data_ptr() == out.data_ptr()
    assert torch.equal(out, head.littlebit_logprobs_bwd(x, targets, lse, H, one, one))
    outside = torch.ones_like(buf, dtype=torch.bool)
    outside[10:10 + 5 * 140].view(5, 140)[:, :133] = False
    assert (buf[outside] == 3).all()


def test_rows_beyond_32_bits(head):
    """Rows whose offsets pass 2^31 (and 2^32 bytes): the same as the same rows close together."""
    case("rows far apart")
    far = torch.empty(5_000_000_000, dtype=torch.int8, device="cuda")   # 5 GB, read and written at the rows alone

    def spread(t, ld):
        v = torch.as_strided(far.view(t.dtype), t.shape, (ld, 1), 8)
        v.copy_(t)
        return v

    x, w = randn(1, 24, 640).half().cuda(), torch.ones(640, dtype=torch.float16, device="cuda")
    y, _ = head.littlebit_rmsnorm_fwd(spread(x, 100_000_000), w)
    assert torch.equal(y, head.littlebit_rmsnorm_fwd(x, w)[0])
    dx, dw = head.littlebit_rmsnorm_bwd(spread(x, 100_000_000), x, w)
    assert all(torch.equal(a, b) for a, b in zip((dx, dw), head.littlebit_rmsnorm_bwd(x, x, w)))
    q, s = head.littlebit_q8_quantize(spread(x, 100_000_000))
    assert torch.equal(q, head.littlebit_q8_quantize(x)[0])
    q = q.contiguous()
    for m in (24, 4800):       # channels as rows far apart; tokens as rows far apart
        W = torch.randint(-127, 128, (m, 640), dtype=torch.int8, device="cuda")
        ws = torch.rand(m, device="cuda")
        for batch in (3, 24):
            want = head.littlebit_q8_linear_fwd(q[:batch], s[:batch], W, ws)
            if m == 24:
                far_w = head.littlebit_q8_linear_fwd(q[:batch], s[:batch], spread(W, 200_000_000), ws)
                assert torch.equal(far_w, want)
            far_x = head.littlebit_q8_linear_fwd(spread(q[:batch], 200_000_000), s[:batch], W, ws)
            assert torch.equal(far_x, want)
            out = torch.as_strided(far.view(torch.float16), (batch, m), (100_000_000, 1), 8)
            assert torch.equal(head.littlebit_q8_linear_fwd(q[:batch], s[:batch], W, ws, out=out), want)
    lg, tg = randn(2, 24, 5000).half().cuda(), torch.arange(24, device="cuda")
    a = head.littlebit_logprobs_fwd(spread(lg, 100_000_000), tg, 3)
    b = head.littlebit_logprobs_fwd(lg, tg, 3)
    assert all(torch.equal(p, r) for p, r in zip(a, b))
    one = torch.ones(24, device="cuda")
    v = spread(lg, 100_000_000)
    d = head.littlebit_logprobs_bwd(v, tg, b[2], b[1], one, one, out=v)
    assert torch.equal(d, head.littlebit_logprobs_bwd(lg, tg, b[2], b[1], one, one))


def test_many_rows(head):
    """More logits than 2^31 in one call: the last rows are the rows themselves."""
    case("many rows")
    rows, vocab = 70_000, 32_000
    x = torch.empty(rows, vocab, dtype=torch.float16, device="cuda").normal_()
    targets = torch.randint(0, vocab, (rows,), device="cuda")
    a = head.littlebit_logprobs_fwd(x, targets, 2)
    for r in (0, 67_108, 67_109, 69_999):
        b = head.littlebit_logprobs_fwd(x[r:r + 1].clone(), targets[r:r + 1], 2)
        assert torch.equal(a[0][r:r + 1], b[0]) and torch.equal(a[1][r:r + 1], b[1])
        assert torch.equal(a[3][r:r + 1], b[3]) and torch.equal(a[4][r:r + 1], b[4])
    last = x[-1:].clone()
    one = torch.ones(rows, device="cuda")
    head.littlebit_logprobs_bwd(x, targets, a[2], a[1], one, one, out=x)
    b = head.littlebit_logprobs_fwd(last, targets[-1:])
    assert torch.equal(x[-1:], head.littlebit_logprobs_bwd(last, targets[-1:], b[2], b[1], one[:1], one[:1]))


def test_the_longest_row(head):
    """2^30 logits in a row: split over 512 workgroups, 8192 of them a thread."""
    case("the longest row")
    vocab = 1 << 30
    x = torch.empty(1, vocab, dtype=torch.float16, device="cuda").normal_()
    x[0, 123_456_789], x[0, vocab - 1], x[0, 77] = 30.0, 31.0, -np.inf
    total = torch.zeros((), dtype=torch.float64, device="cuda")
    for part in x[0].split(1 << 26):
        total += part.double().sub_(31).exp_().sum()
    lse = 31 + float(total.log())
    lp, H, parts, tv, ti = head.littlebit_logprobs_fwd(x, torch.tensor([vocab - 1], device="cuda"), 2)
    assert ti.tolist() == [[vocab - 1, 123_456_789]]
    tol = (8192 + 100) * 2 * U + 4 * U * 31
    assert abs(float(parts.sum()) - lse) <= tol and abs(float(lp) - (31 - lse)) <= tol
    assert abs(float(tv[0, 1]) - (30 - lse)) <= tol
    x.fill_(1.0)                      # all equal: the lowest places, 30 log 2
    lp, H, parts, tv, ti = head.littlebit_logprobs_fwd(x, torch.tensor([5], device="cuda"), 2)
    assert ti.tolist() == [[0, 1]]
    assert abs(float(lp) + 30 * np.log(2)) <= 2 * tol and abs(float(H) - 30 * np.log(2)) <= 2 * tol


# ------------------------------------------------------------------------------------------------------- together

def _model(head, n=512, vocab=2000, seed=3):
    rng = np.random.default_rng(seed)
    W = torch.from_numpy((rng.standard_normal((vocab, n)) / np.sqrt(n)).astype(np.float32)).cuda()
    norm = torch.from_numpy(rng.uniform(0.5, 1.5, n)).half().cuda()
    return W, norm, head.LittleBitHead.from_weights(norm, W)


def test_block_to_token_probabilities(head):
    """A LittleBit layer behind a norm, then the head: every operator as it is used,
    against the float64 formulas on the same stored intermediates."""
    case("layer, norm, head, log probabilities")
    import oracle
    from binary_rank_gemv_amd import littlebit as lb
    from binary_rank_gemv_amd import synth
    branches, x = synth.make_layer(synth.TINY, batch=6, seed=1)
    layer = lb.LittleBitLayer.from_latents(branches)
    W, norm, hd = _model(head)
    x0 = torch.from_numpy(x).cuda()
    res = torch.from_numpy(np.random.default_rng(2).standard_normal((6, 512))).half().cuda()
    y, h = head.littlebit_rmsnorm_fwd(x0, norm, res)
    z = lb.littlebit_linear_fwd(layer, y)
    want_z = oracle.linear_forward(f64(y).astype(np.float16), branches)
    assert np.linalg.norm(f64(z) - want_z) / np.linalg.norm(want_z) <= 2e-3
    z = (z.float() / z.float().std()).half()
    targets = torch.tensor([0, 1999, -100, 5, 6, 7]).cuda()
    lp, H, tv, ti = hd.logprobs(z, targets, h, top=3)
    # the same in float64 from the stored codes
    hh = (z.double() + h.double()).half()
    q, scale, h2 = head.littlebit_rmsnorm_q8(z, norm, h)
    assert torch.equal(h2, hh)
    vals = f64(q) * f64(scale)[:, None]
    want_y = oh.rmsnorm(f64(hh), f64(norm), 1e-5)
    assert np.abs(vals - want_y).max() <= oh.q8_scale(want_y).max() * 0.51
    logits = oh.q8_linear(q.cpu().numpy(), f64(scale), hd.linear.q.cpu().numpy(), f64(hd.linear.scale))
    logp, ent = oh.logprobs(logits)
    rows = np.arange(6)
    given = np.array([0, 1, 3, 4, 5])
    assert np.abs(f64(lp)[given] - logp[rows, targets.cpu().numpy()][given]).max() <= 2e-5 and lp[2] == 0
    assert np.abs(f64(H) - ent).max() <= 2e-5
    # and 8 bits against the dense head: each factor's codes are within half a step of its largest value / 127,
    # independent over the 512 inputs: their sum stays within six standard deviations
    dense = want_y @ f64(W).T
    sw, sx = oh.q8_scale(f64(W))[None, :], oh.q8_scale(want_y)[:, None]
    dev = np.sqrt(((want_y ** 2).sum(1)[:, None] * sw ** 2 + (f64(W) ** 2).sum(1)[None, :] * sx ** 2) / 12)
    assert (np.abs(logits - dense) <= 6 * dev).all()


def test_head_text_in_parts_is_the_text_at_once(head):
    case("head in parts")
    W, norm, hd = _model(head)
    x = randn(4, 75, 512).half().cuda()
    targets = targets_of(1, 75, 2000).cuda()
    whole = hd.logprobs(x, targets, top=2)
    parts = hd.logprobs(x, targets, top=2, max_logit_bytes=2000 * 4 * 16)
    for a, b in zip(whole, parts):
        assert a.shape == b.shape and (torch.equal(a, b) if a.dtype == torch.int64 else torch.allclose(a, b, rtol=0, atol=1e-5))
    e = hd.logprobs(x[:0], targets[:0], top=2)
    assert e[0].shape == (0,) and e[3].shape == (0, 2)


def test_perplexity_of_a_padded_text(head):
    """As the docstring has it: the same with padding as without."""
    case("perplexity")
    W, norm, hd = _model(head)
    x, targets = randn(4, 40, 512).half().cuda(), torch.arange(40, device="cuda")
    targets[25:] = -100
    def perplexity(x, targets):
        logprob = hd.logprobs(x, targets)[0]
        return (-logprob[targets >= 0].mean()).exp()
    # the logits of a row may be formed by another kernel (25 tokens or 40): the sums are exact, so the same bits
    assert torch.equal(perplexity(x, targets), perplexity(x[:25], targets[:25]))
    assert (hd.logprobs(x, targets)[0][25:] == 0).all()


def test_head_in_parts_refuses_a_residual_of_other_rows(head):
    """Also where every part of the residual has its part's shape."""
    case("head, other residuals")
    W, norm, hd = _model(head)
    x, targets = randn(4, 32, 512).half().cuda(), targets_of(1, 32, 2000).cuda()
    for r in (x.repeat(2, 1), x[:16], x.repeat(1, 2)[:, :511], x.bfloat16(), x[0]):
        with pytest.raises(ValueError):
            hd.logprobs(x, targets, r, max_logit_bytes=2000 * 4 * 16)
    for y in (x[0], x.float(), None):
        with pytest.raises(ValueError):
            hd.logprobs(y, targets)


def test_head_holds_one_part_of_the_logits(head):
    case("head memory")
    W, norm = randn(1, 32000, 64).half().cuda(), torch.ones(64, dtype=torch.float16, device="cuda")
    hd = head.LittleBitHead.from_weights(norm, W)
    x, targets = randn(2, 2500, 64).half().cuda(), targets_of(3, 2500, 32000).cuda()
    room = 500 * 32000 * 4
    for stream in (None, torch.cuda.Stream()):
        torch.cuda.synchronize()
        before = torch.cuda.memory_allocated()
        torch.cuda.reset_peak_memory_stats()
        hd.logprobs(x, targets, top=2, max_logit_bytes=room, stream=stream)
        torch.cuda.synchronize()
        # the allocator hands out large blocks whole, in steps of 2 MiB; besides the logits there are the codes, scales
        # and lse of 500 tokens (64 + 4 + 8 bytes each) and the results of 2500 (32 bytes each): 118000 bytes, and less
        # than 512 more for each of 25 tensors
        block = -(-room // (2 << 20)) * (2 << 20)
        assert torch.cuda.max_memory_allocated() - before <= block + (1 << 17)


def test_head_text_of_more_tokens_than_a_call_takes(head):
    rows = (1 << 21) + 5
    case("long text", rows)
    W, norm = randn(1, 6, 8).half().cuda(), torch.ones(8, dtype=torch.float16, device="cuda")
    hd = head.LittleBitHead.from_weights(norm, W)
    x = randn(2, 1000, 8).half().cuda()
    targets = targets_of(3, 1000, 6).cuda()
    at = torch.arange(rows, device="cuda") % 1000
    lp, H, tv, ti = hd.logprobs(x[at], targets[at], top=2)
    for got, want in zip((lp, H, tv, ti), hd.logprobs(x, targets, top=2)):
        assert got.shape[0] == rows and torch.equal(got, want[at])


def test_streams_and_graphs(head):
    """The chain captured once and replayed over new inputs, with the program's own
    eager work between the replays; two graphs share nothing."""
    case("graphs")
    W, norm, hd = _model(head, vocab=9000)
    lib_in = [torch.empty(3, 512, dtype=torch.float16, device="cuda") for _ in range(2)]
    targets = torch.tensor([5, 8999, -1]).cuda()

    def step(x):
        logits = hd.logits(x)
        lp, H, lse, tv, ti = head.littlebit_logprobs_fwd(logits, targets, 4)
        d = head.littlebit_logprobs_bwd(logits, targets, lse, H, torch.ones(3, device="cuda"), torch.ones(3, device="cuda"),
                                        ti, torch.ones(3, 4, device="cuda"))
        y, h = head.littlebit_rmsnorm_fwd(x, norm, x)
        dx, dw = head.littlebit_rmsnorm_bwd(y, h, norm)
        return [logits, lp, H, lse, tv, ti, d, dx, dw]

    graphs, outs = [], []
    s = torch.cuda.Stream()
    for x in lib_in:
        x.normal_()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            step(x)
        torch.cuda.current_stream().wait_stream(s)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            outs.append(step(x))
        graphs.append(g)
    for k in range(4):
        for i, x in enumerate(lib_in):
            x.copy_(randn(10 * k + i, 3, 512).half())
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        graphs[0].replay()
        with torch.cuda.stream(side):
            graphs[1].replay()
        torch.cuda.synchronize()
        for x, got in zip(lib_in, outs):
            want = step(x)
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(got, want))
    # an explicit stream
    with torch.cuda.stream(torch.cuda.Stream()):
        torch.cuda.synchronize()
    s.wait_stream(torch.cuda.current_stream())
    q, scale, _ = head.littlebit_rmsnorm_q8(lib_in[0], norm, stream=s)
    y = head.littlebit_q8_linear_fwd(q, scale, hd.linear.q, hd.linear.scale, dtype=torch.float32, stream=s)
    s.synchronize()
    assert torch.equal(y, outs[0][0])


def test_alternatives_beyond_the_limit_take_no_memory(head):
    case("refused top")
    from binary_rank_gemv_amd.littlebit import LittleBitError
    x = torch.zeros(2000, 300, dtype=torch.float16, device="cuda")
    before = torch.cuda.memory_allocated()
    torch.cuda.reset_peak_memory_stats()
    for top in (65, 300, 301, 1 << 30, (1 << 32) + 3):
        with pytest.raises(LittleBitError):
            head.littlebit_logprobs_fwd(x, None, top)
    assert torch.cuda.max_memory_allocated() - before <= 2 * 2000 * 16    # entropy and lse, 12 bytes a row


def test_tensors_freed_behind_a_call_on_another_stream(head):
    """The caller's tensors go out of use as soon as the call returns, while the stream it was
    given is still busy: what is allocated next does not take their memory."""
    case("freed behind a stream")
    rows, n, m = 64, 4096, 2048
    made = lambda k, *shape: randn(k, *shape).half().cuda()  # noqa: E731
    q, s = head.littlebit_q8_quantize(made(3, rows, n))
    wq, ws = head.littlebit_q8_quantize(made(4, m, n))
    lg, tg, f = made(5, rows, 9000), torch.arange(rows, device="cuda"), torch.rand(rows, device="cuda")
    _, H, lse, _, _ = head.littlebit_logprobs_fwd(lg, tg)
    calls = [(head.littlebit_rmsnorm_fwd, [made(0, rows, n), made(1, n), made(2, rows, n)]),
             (head.littlebit_rmsnorm_q8, [made(0, rows, n), made(1, n), made(2, rows, n)]),
             (head.littlebit_rmsnorm_bwd, [made(0, rows, n), made(2, rows, n), made(1, n), made(6, rows, n)]),
             (head.littlebit_q8_quantize, [made(0, rows, n)]), (head.littlebit_q8_linear_fwd, [q, s, wq, ws]),
             (head.littlebit_logprobs_fwd, [lg, tg]), (head.littlebit_logprobs_bwd, [lg, tg, lse, H, f, f])]
    side = torch.cuda.Stream()
    for call, args in calls:
        want = call(*args)
        want = want if isinstance(want, tuple) else (want,)
        torch.cuda.synchronize()
        temporary = [a.clone() for a in args]
        sizes = [(a.shape, a.dtype) for a in args]
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            torch.cuda._sleep(20_000_000)
        got = call(*temporary, stream=side)
        got = got if isinstance(got, tuple) else (got,)
        del temporary
        later = [torch.zeros(shape, dtype=t, device="cuda") for shape, t in sizes]
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert (a is None and b is None) or torch.equal(a, b), call.__name__
        del later, got
        # the same captured, the stream named
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            got = call(*args, stream=side)
        for _ in range(3):
            graph.replay()
            torch.cuda.synchronize()
            for a, b in zip(got if isinstance(got, tuple) else (got,), want):
                assert (a is None and b is None) or torch.equal(a, b), call.__name__
            torch.zeros(1 << 20, device="cuda").add_(1)
        del graph, got


def test_gradients_are_not_lost_in_silence(head):
    """While autograd records, a tensor that requires a gradient is refused; without recording, and
    inside a Function, the calls take it.  The Function's gradients are those of the formulas."""
    case("requires grad")
    x, r, w = randn(1, 6, 64).half().cuda(), randn(2, 6, 64).half().cuda(), (1 + 0.1 * randn(3, 64)).half().cuda()
    lg, tg, f, g2 = randn(4, 6, 90).cuda(), torch.arange(6, device="cuda"), torch.rand(6, device="cuda"), torch.rand(6, 2, device="cuda")
    lg = lg.float()
    q, s = head.littlebit_q8_quantize(x)
    lp, H, lse, tv, ti = head.littlebit_logprobs_fwd(lg, tg, 2)
    calls = [(head.littlebit_rmsnorm_fwd, [x, w, r]), (head.littlebit_rmsnorm_q8, [x, w, r]),
             (head.littlebit_rmsnorm_bwd, [x, r, w, x]), (head.littlebit_q8_quantize, [x]),
             (head.littlebit_q8_linear_fwd, [q, s, q, s]), (head.littlebit_logprobs_fwd, [lg, tg, 2]),
             (head.littlebit_logprobs_bwd, [lg, tg, lse, H, f, f, ti, g2])]
    for call, args in calls:
        want = call(*args)
        for i, a in enumerate(args):
            if not (torch.is_tensor(a) and a.is_floating_point()):
                continue
            leaf = [a.detach().clone().requires_grad_() if j == i else b for j, b in enumerate(args)]
            with pytest.raises(ValueError, match="gradient"):
                call(*leaf)
            with torch.no_grad():
                got = call(*leaf)
            for p, q_ in zip(got if isinstance(got, tuple) else [got], want if isinstance(want, tuple) else [want]):
                assert torch.equal(p, q_)
    # a model's own parameters, without no_grad
    hd = head.LittleBitHead.from_weights(torch.nn.Parameter(w), torch.nn.Parameter(lg[:, :64].half()))
    assert hd.logprobs(x, tg, r)[0].shape == (6,)

    class Norm(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, residual, weight):
            y, h = head.littlebit_rmsnorm_fwd(x, weight, residual)
            ctx.save_for_backward(h, weight)
            return y, h

        @staticmethod
        def backward(ctx, dy, dh):
            h, weight = ctx.saved_tensors
            dx, dw = head.littlebit_rmsnorm_bwd(dy.contiguous(), h, weight, dh.contiguous())
            return dx, dx, dw.to(weight.dtype)

    leaves = [t.detach().clone().requires_grad_() for t in (x, r, w)]
    y, h = Norm.apply(*leaves)
    dy, dh = randn(7, 6, 64).half().cuda(), randn(8, 6, 64).half().cuda()
    torch.autograd.backward([y, h], [dy, dh])
    dx, dw = head.littlebit_rmsnorm_bwd(dy, h.detach(), w, dh)
    assert torch.equal(leaves[0].grad, dx) and torch.equal(leaves[1].grad, dx) and torch.equal(leaves[2].grad, dw.half())


def test_refusals(head):
    case("refusals")
    x = torch.zeros(4, 64, dtype=torch.float16, device="cuda")
    w = x[0]
    f = torch.zeros(4, device="cuda")
    q = torch.zeros(4, 64, dtype=torch.int8, device="cuda")
    ti = torch.zeros(4, 2, dtype=torch.int64, device="cuda")
    lse = torch.zeros(2, 4, device="cuda")
    from binary_rank_gemv_amd.littlebit import LittleBitError
    for call in (lambda: head.littlebit_rmsnorm_q8(x.t(), w[:4]),
                 lambda: head.littlebit_rmsnorm_q8(x, w[:63]),
                 lambda: head.littlebit_rmsnorm_q8(x, w.bfloat16()),
                 lambda: head.littlebit_rmsnorm_q8(x, w, x[:3]),
                 lambda: head.littlebit_rmsnorm_q8(x, w, hidden=x),
                 lambda: head.littlebit_rmsnorm_q8(x[:1].expand(4, 64), w),
                 lambda: head.littlebit_rmsnorm_q8(x.cpu(), w),
                 lambda: head.littlebit_rmsnorm_bwd(x, x, w, x.float()),
                 lambda: head.littlebit_q8_linear_fwd(q, f, q[:, :32], f),
                 lambda: head.littlebit_q8_linear_fwd(q, f[:3], q, f),
                 lambda: head.littlebit_q8_linear_fwd(q, f, q, f, dtype=torch.int32),
                 lambda: head.littlebit_q8_linear_fwd(q, f, q, f, out=x),
                 lambda: head.littlebit_logprobs_fwd(x, ti[:, 0]),
                 lambda: head.littlebit_logprobs_fwd(x, f),
                 lambda: head.littlebit_logprobs_bwd(x, None, f),
                 lambda: head.littlebit_logprobs_bwd(x, None, lse, dlogprob=f),
                 lambda: head.littlebit_logprobs_bwd(x, None, lse, dtop=f.view(4, 1)),
                 lambda: head.littlebit_logprobs_bwd(x, None, lse, top_index=ti, dtop=torch.zeros(4, 3, device="cuda")),
                 lambda: head.littlebit_logprobs_bwd(x, None, lse, dentropy=f)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: head.littlebit_logprobs_fwd(x, None, 65), lambda: head.littlebit_logprobs_fwd(x, None, -1),
                 lambda: head.littlebit_rmsnorm_q8(x, w, eps=-1.0)):
        with pytest.raises(LittleBitError):
            call()
