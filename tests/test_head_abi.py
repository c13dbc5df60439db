"""The C ABI of the dense operators: exported symbols, refusals before anything
is launched, sizes.  Every call here fails validation on the host or has
nothing to do; no GPU is needed."""

import ctypes
import os
import re
import subprocess

import pytest
import torch

head = pytest.importorskip("binary_rank_gemv_amd.head",
                           reason="liblittlebit_head.so not built (run python -m binary_rank_gemv_amd.build)")
from binary_rank_gemv_amd import littlebit as lb  # noqa: E402

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "littlebit_head.h")
FAKE = 1 << 20   # non-null, aligned, never dereferenced
BAD, UNSUP, WS = lb.LB_ERR_INVALID_ARG, lb.LB_ERR_UNSUPPORTED, lb.LB_ERR_WORKSPACE
F32, F16, BF16 = lb.LB_F32, lb.LB_F16, head.LB_BF16


def test_every_declared_symbol_is_exported_and_bound():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"\b(littlebit_\w+)\s*\(", text))
    assert names == set(head.HEAD_EXPORTED)
    lib = ctypes.CDLL(head.HEAD_LIB_PATH)
    for n in names:
        assert hasattr(lib, n), n
    for line in open(HEADER):
        m = re.match(r"#define (LB_\w+) (\d+)$", line)
        if m:
            assert getattr(head, m.group(1)) == int(m.group(2))


def test_library_needs_no_vendor_kernels():
    deps = subprocess.run(["readelf", "-d", head.HEAD_LIB_PATH], capture_output=True, text=True).stdout
    needed = re.findall(r"\(NEEDED\).*\[(.*)\]", deps)
    assert needed and not any(k in d for d in needed for k in ("blas", "solver", "MIOpen"))


def _norm(x=FAKE, ldx=64, res=FAKE, ldr=64, weight=FAKE, dtype=F16, rows=2, n=64, eps=1e-5, hidden=2 * FAKE, ldh=64,
          y=3 * FAKE, ldy=64, q=None, ldq=64, scale=None):
    return head.LIB.littlebit_rmsnorm_fwd(x, ldx, res, ldr, weight, dtype, rows, n, eps, hidden, ldh, y, ldy, q, ldq,
                                          scale, None)


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), BAD), (dict(weight=None), BAD), (dict(dtype=F32), BAD), (dict(dtype=7), BAD),
    (dict(rows=-1), BAD), (dict(n=0), BAD), (dict(n=40000, ldx=40000, ldr=40000, ldh=40000, ldy=40000), UNSUP),
    (dict(rows=1 << 22), UNSUP), (dict(eps=-1.0), BAD), (dict(eps=float("nan")), BAD), (dict(ldx=63), BAD),
    (dict(ldr=63), BAD), (dict(ldh=63), BAD), (dict(ldy=63), BAD), (dict(x=FAKE + 1), BAD), (dict(y=None), BAD),
    (dict(q=FAKE), BAD), (dict(scale=FAKE), BAD), (dict(q=FAKE, scale=FAKE, ldq=63), BAD),
    (dict(q=FAKE, scale=FAKE + 2), BAD), (dict(res=None), BAD), (dict(hidden=None), BAD),
    (dict(hidden=FAKE, ldh=72), BAD), (dict(ldx=1 << 50), UNSUP),
])
def test_norm_refuses(kw, status):
    assert _norm(**kw) == status
    assert "littlebit_rmsnorm_fwd" in head.littlebit_head_last_error()


def test_no_rows_is_no_work():
    assert _norm(rows=0, x=None, res=None, hidden=None, weight=None) == lb.LB_OK
    assert head.LIB.littlebit_q8_quantize(None, 64, F32, 0, 64, None, 64, None, None) == lb.LB_OK
    assert head.LIB.littlebit_q8_linear_fwd(None, 64, None, None, 64, None, 0, 8, 64, None, 8, F16, None) == lb.LB_OK
    assert head.LIB.littlebit_logprobs_fwd(None, 9, F16, 0, 9, None, None, None, None, 0, None, None, None, 0,
                                           None) == lb.LB_OK
    assert head.LIB.littlebit_logprobs_bwd(None, 9, F16, 0, 9, None, None, None, None, None, 0, None, None, None, 9,
                                           None) == lb.LB_OK


def _bwd(dy=FAKE, lddy=64, dh=FAKE, lddh=64, hidden=FAKE, ldh=64, weight=FAKE, dtype=BF16, rows=3, n=64, eps=1e-5,
         dx=2 * FAKE, lddx=64, dw=FAKE, ws=FAKE, nws=1 << 20):
    return head.LIB.littlebit_rmsnorm_bwd(dy, lddy, dh, lddh, hidden, ldh, weight, dtype, rows, n, eps, dx, lddx, dw,
                                          ws, nws, None)


@pytest.mark.parametrize("kw,status", [
    (dict(dy=None), BAD), (dict(hidden=None), BAD), (dict(weight=None), BAD), (dict(dx=None), BAD), (dict(dw=None), BAD),
    (dict(dw=FAKE + 2), BAD), (dict(lddy=8), BAD), (dict(lddh=8), BAD), (dict(lddx=8), BAD), (dict(dtype=F32), BAD),
    (dict(ws=None), WS), (dict(ws=FAKE + 8), WS), (dict(nws=16), WS), (dict(rows=-3), BAD), (dict(n=0), BAD),
    (dict(dx=FAKE, lddx=72), BAD), (dict(eps=-1.0), BAD),
])
def test_norm_backward_refuses(kw, status):
    assert _bwd(**kw) == status


def _lin(xq=FAKE, ldx=64, xs=FAKE, wq=FAKE, ldw=64, ws=FAKE, batch=2, m=16, n=64, y=FAKE, ldy=16, dt=F16):
    return head.LIB.littlebit_q8_linear_fwd(xq, ldx, xs, wq, ldw, ws, batch, m, n, y, ldy, dt, None)


@pytest.mark.parametrize("kw,status", [
    (dict(xq=None), BAD), (dict(xs=None), BAD), (dict(wq=None), BAD), (dict(ws=None), BAD), (dict(y=None), BAD),
    (dict(ldx=63), BAD), (dict(ldw=63), BAD), (dict(ldy=15), BAD), (dict(batch=-1), BAD), (dict(m=0), BAD),
    (dict(n=0), BAD), (dict(n=131072, ldx=131072, ldw=131072), UNSUP), (dict(m=1 << 25, ldy=1 << 25), UNSUP),
    (dict(dt=9), BAD), (dict(y=FAKE + 1), BAD), (dict(xs=FAKE + 1), BAD),
    (dict(batch=1 << 20, m=1 << 20, ldy=1 << 20), UNSUP),
])
def test_linear_refuses(kw, status):
    assert _lin(**kw) == status


def _lp(x=FAKE, ld=100, dt=F16, rows=2, vocab=100, t=FAKE, lp=FAKE, H=FAKE, lse=FAKE, top=0, tv=None, ti=None, ws=None,
        nws=0):
    return head.LIB.littlebit_logprobs_fwd(x, ld, dt, rows, vocab, t, lp, H, lse, top, tv, ti, ws, nws, None)


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), BAD), (dict(ld=99), BAD), (dict(dt=4), BAD), (dict(rows=-1), BAD), (dict(vocab=0), BAD),
    (dict(t=None), BAD), (dict(lp=None), BAD), (dict(lse=None), BAD), (dict(t=FAKE + 4), BAD), (dict(top=-1), BAD),
    (dict(top=101, tv=FAKE, ti=FAKE), BAD), (dict(top=65, tv=FAKE, ti=FAKE), UNSUP), (dict(top=3, ti=FAKE), BAD),
    (dict(top=3, tv=FAKE), BAD), (dict(x=FAKE + 1), BAD), (dict(vocab=1 << 31, ld=1 << 31), UNSUP),
    (dict(vocab=100000, ld=100000), WS), (dict(vocab=100000, ld=100000, ws=FAKE + 4, nws=1 << 20), WS),
])
def test_logprobs_refuses(kw, status):
    assert _lp(**kw) == status


def _lpb(x=FAKE, ld=100, dt=F16, rows=2, vocab=100, t=FAKE, lse=FAKE, H=FAKE, dlp=FAKE, dH=FAKE, top=0, ti=None,
         dt_=None, d=FAKE, ldd=100):
    return head.LIB.littlebit_logprobs_bwd(x, ld, dt, rows, vocab, t, lse, H, dlp, dH, top, ti, dt_, d, ldd, None)


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), BAD), (dict(d=None), BAD), (dict(lse=None), BAD), (dict(t=None), BAD), (dict(dlp=None), BAD),
    (dict(H=None), BAD), (dict(dH=None), BAD), (dict(top=2, ti=FAKE), BAD), (dict(top=2, dt_=FAKE), BAD),
    (dict(top=65, ti=FAKE, dt_=FAKE), UNSUP), (dict(ldd=104), BAD), (dict(ldd=50, d=2 * FAKE), BAD),
    (dict(rows=1 << 20, vocab=1 << 20, ld=1 << 20, ldd=1 << 20), UNSUP),
])
def test_logprobs_backward_refuses(kw, status):
    assert _lpb(**kw) == status


def test_workspace_sizes():
    W = head.LIB.littlebit_logprobs_workspace_bytes
    assert W(1, 100, F16, 5) == 0 and W(5000, 128000, F16, 5) == 0     # one workgroup a row: nothing to join
    assert 0 < W(1, 128000, F16, 0) < W(1, 128000, F16, 20)
    assert W(0, 100, F16, 0) == 0 and W(1, 0, F16, 0) == 0 and W(1, 1 << 31, F16, 0) == 0
    B = head.LIB.littlebit_rmsnorm_bwd_workspace_bytes
    assert B(0, 64) == 0 and B(1, 64) >= 256 and B(10, 40000) == 0


def test_binding_refuses_what_is_not_on_a_gpu():
    x = torch.zeros(2, 8, dtype=torch.float16)
    for call in (lambda: head.littlebit_rmsnorm_q8(x, x[0]), lambda: head.littlebit_rmsnorm_fwd(x.float(), x[0]),
                 lambda: head.littlebit_rmsnorm_bwd(x, x, x[0]), lambda: head.littlebit_q8_quantize(x),
                 lambda: head.littlebit_q8_linear_fwd(x, x, x, x), lambda: head.littlebit_logprobs_fwd(x),
                 lambda: head.littlebit_logprobs_bwd(x, None, x[0])):
        with pytest.raises(ValueError):
            call()
