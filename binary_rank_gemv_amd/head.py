"""ctypes binding of ``include/littlebit_head.h`` (argument marshalling only):
the dense operators around the LittleBit layers, in ``_lib/liblittlebit_head.so``.

* ``littlebit_rmsnorm_q8(x, weight, residual)`` -> (q, scale, hidden): the norm
  with the residual's addition, as int8 codes with one scale a token
* ``littlebit_rmsnorm_fwd(x, weight, residual)`` -> (y, hidden): the same, dense
  (what ``littlebit_linear_fwd`` and ``littlebit_block_fwd`` read)
* ``littlebit_rmsnorm_bwd(dy, hidden, weight)`` -> (dx, dweight)
* ``littlebit_q8_quantize(x)`` -> (q, scale), by row
* ``littlebit_q8_linear_fwd(xq, xscale, wq, wscale)`` -> y
* ``littlebit_logprobs_fwd(logits, targets, top)`` -> (logprob, entropy, lse,
  top_logprob, top_index)
* ``littlebit_logprobs_bwd(logits, targets, lse, entropy, ...)`` -> dlogits
* ``Q8Linear`` holds an 8-bit weight; ``LittleBitHead`` a model's last norm and
  its 8-bit head, with the logits or the log probabilities of a text

Work is enqueued on ``stream`` (default: the current stream of the tensors'
device), which the caller lets wait for what the tensors' own stream still
writes; their memory is not reused before ``stream`` has passed the call.  The
tensors of a call lie on one device, which need not be the current one.

Nothing is recorded for autograd: the backward passes are calls of their own,
and while gradients are recorded a tensor that requires one is refused (call
under ``torch.no_grad()``, as the methods of a ``torch.autograd.Function`` are).

Importing this module raises if the library has not been built
(``python -m binary_rank_gemv_amd.build``): there is no fallback path.
"""

from __future__ import annotations

import contextlib
import ctypes
import os
from dataclasses import dataclass
from typing import Optional, Tuple

import torch

from .littlebit import LB_F16, LB_F32, LB_OK, LittleBitError

HEAD_LIB_PATH = os.environ.get("LITTLEBIT_HEAD_LIBRARY") or os.path.join(
    os.path.dirname(os.path.abspath(__file__)), "_lib", "liblittlebit_head.so")

LB_BF16 = 2
LB_NORM_MAX_N = 32768
LB_TOP_MAX = 64

HEAD_EXPORTED = (
    "littlebit_rmsnorm_fwd", "littlebit_rmsnorm_bwd_workspace_bytes", "littlebit_rmsnorm_bwd",
    "littlebit_q8_quantize", "littlebit_q8_linear_fwd", "littlebit_logprobs_workspace_bytes",
    "littlebit_logprobs_fwd", "littlebit_logprobs_bwd", "littlebit_head_last_error",
)

_DTYPE = {torch.float32: LB_F32, torch.float16: LB_F16, torch.bfloat16: LB_BF16}
_HALF = {torch.float16: LB_F16, torch.bfloat16: LB_BF16}
_INT8 = {torch.int8: 0}


def _load():
    if not os.path.exists(HEAD_LIB_PATH):
        raise ImportError(f"{HEAD_LIB_PATH} is missing: build it with `python -m binary_rank_gemv_amd.build`")
    lib = ctypes.CDLL(HEAD_LIB_PATH)
    vp, i64, i32, f32, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
    sigs = {
        "littlebit_rmsnorm_fwd": (i32, [vp, i64, vp, i64, vp, i32, i64, i64, f32, vp, i64, vp, i64, vp, i64, vp, vp]),
        "littlebit_rmsnorm_bwd_workspace_bytes": (sz, [i64, i64]),
        "littlebit_rmsnorm_bwd": (i32, [vp, i64, vp, i64, vp, i64, vp, i32, i64, i64, f32, vp, i64, vp, vp, sz, vp]),
        "littlebit_q8_quantize": (i32, [vp, i64, i32, i64, i64, vp, i64, vp, vp]),
        "littlebit_q8_linear_fwd": (i32, [vp, i64, vp, vp, i64, vp, i64, i64, i64, vp, i64, i32, vp]),
        "littlebit_logprobs_workspace_bytes": (sz, [i64, i64, i32, i32]),
        "littlebit_logprobs_fwd": (i32, [vp, i64, i32, i64, i64, vp, vp, vp, vp, i32, vp, vp, vp, sz, vp]),
        "littlebit_logprobs_bwd": (i32, [vp, i64, i32, i64, i64, vp, vp, vp, vp, vp, i32, vp, vp, vp, i64, vp]),
        "littlebit_head_last_error": (ctypes.c_char_p, []),
    }
    for name, (res, args) in sigs.items():
        f = getattr(lib, name)
        f.restype, f.argtypes = res, args
    return lib


LIB = _load()


def littlebit_head_last_error() -> str:
    return LIB.littlebit_head_last_error().decode()


def _check(status: int):
    if status != LB_OK:
        raise LittleBitError(status, littlebit_head_last_error())


_HERE = contextlib.nullcontext()
_empty = torch.empty_strided   # the cheapest way to an uninitialised tensor: these calls are short
_raw_stream = torch._C._cuda_getCurrentRawStream


def _on(device, stream):
    """(context, stream pointer): `device` current, allocations on `stream`."""
    if stream is not None:
        if stream.device != device:
            raise ValueError(f"stream is on {stream.device}, the tensors are on {device}")
        return torch.cuda.stream(stream), int(stream.cuda_stream)
    index = device.index
    return (_HERE if index == torch.cuda.current_device() else torch.cuda.device(index)), _raw_stream(index)


def _matrix(name: str, t: torch.Tensor, dtype, device, shape) -> int:
    """Checks a row-major matrix argument (unit column stride, any row stride)
    and returns its row stride; of a single row, at least its length."""
    if torch.is_tensor(t) and t.dtype is dtype and t.device == device and t.shape == shape and device.type == "cuda":
        rows, cols = shape
        if t.is_contiguous():
            return cols
        if (cols == 1 or t.stride(1) == 1) and (rows == 1 or t.stride(0) >= cols):
            return max(t.stride(0), cols)
        raise ValueError(f"{name} must have unit column stride and rows that do not overlap")
    if not torch.is_tensor(t) or t.dim() != 2 or not t.is_cuda:
        raise ValueError(f"{name} must be a 2-D CUDA tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, is {t.dtype}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, the call is on {device}")
    raise ValueError(f"{name} must have shape {tuple(shape)}, has {tuple(t.shape)}")


def _first(name: str, t: torch.Tensor, dtypes):
    """(dtype code, shape, device) of the argument that the others are held to."""
    code = dtypes.get(t.dtype) if torch.is_tensor(t) else None
    if code is None:
        raise ValueError(f"{name} must be a tensor of {' or '.join(str(d) for d in dtypes)}")
    if t.dim() != 2:
        raise ValueError(f"{name} must be a 2-D CUDA tensor")
    return code, t.shape, t.device


def _vector(name: str, t: torch.Tensor, dtype, device, n: int):
    if not torch.is_tensor(t) or t.dtype is not dtype or t.device != device or t.dim() != 1:
        raise ValueError(f"{name} must be a 1-D {dtype} tensor on {device}")
    if t.shape[0] != n or not t.is_contiguous():
        raise ValueError(f"{name} must be {n} contiguous values")


def _table(name: str, t: torch.Tensor, dtype, device, shape):
    if not torch.is_tensor(t) or t.dtype != dtype or t.device != device or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)} on {device}")


def _keep(stream, *tensors):
    """Tensors that a call reads or writes on a stream given by name: freed ones are
    not handed out again on their own stream while that one still runs."""
    for t in tensors:
        if t is not None:
            t.record_stream(stream)


_recording = torch.is_grad_enabled


def _no_history(*tensors):
    for t in tensors:
        if t is not None and t.requires_grad:
            raise ValueError("a tensor of the call requires a gradient, which would be lost: these calls record nothing for "
                             "autograd; call under torch.no_grad() and take the gradient by the littlebit_*_bwd calls")


def _new(rows: int, n: int, dtype, device) -> torch.Tensor:
    return _empty((rows, n), (n, 1), dtype=dtype, device=device)


def _codes(rows: int, n: int, device):
    """Room for int8 codes and its row stride: rows 16 bytes aligned (the product's fast case)."""
    ld = (n + 15) // 16 * 16
    if ld == n:
        return _new(rows, n, torch.int8, device), n
    return _new(rows, ld, torch.int8, device)[:, :n], ld


# ------------------------------------------------------------------------------------------------------- norm

def _norm(x, weight, residual, eps, hidden, dense, stream):
    code, shape, device = _first("x", x, _HALF)
    dtype = x.dtype
    ldx = _matrix("x", x, dtype, device, shape)
    rows, n = shape
    _vector("weight", weight, dtype, device, n)
    ldr = ldh = ldy = ldq = 0
    if residual is not None:
        ldr = _matrix("residual", residual, dtype, device, shape)
        if hidden is not None:
            ldh = _matrix("hidden", hidden, dtype, device, shape)
    elif hidden is not None:
        raise ValueError("hidden is an output of the residual's addition: give a residual")
    if _recording():
        _no_history(x, weight, residual, hidden)
    ctx, sp = _on(device, stream)
    with ctx:
        if residual is not None and hidden is None:
            hidden, ldh = _new(rows, n, dtype, device), n
        y = q = scale = None
        if dense:
            y, ldy = _new(rows, n, dtype, device), n
        else:
            q, ldq = _codes(rows, n, device)
            scale = _empty((rows,), (1,), dtype=torch.float32, device=device)
        _check(LIB.littlebit_rmsnorm_fwd(
            x.data_ptr(), ldx, None if residual is None else residual.data_ptr(), ldr, weight.data_ptr(), code, rows, n,
            eps, None if hidden is None else hidden.data_ptr(), ldh, None if y is None else y.data_ptr(), ldy,
            None if q is None else q.data_ptr(), ldq, None if scale is None else scale.data_ptr(), sp))
    if stream is not None:
        _keep(stream, x, weight, residual, hidden)
    return y, q, scale, x if residual is None else hidden


def littlebit_rmsnorm_q8(x: torch.Tensor, weight: torch.Tensor, residual: Optional[torch.Tensor] = None,
                         eps: float = 1e-5, hidden: Optional[torch.Tensor] = None,
                         stream=None) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """(q, scale, hidden): hidden = x + residual rounded to their type (x itself
    without a residual), and the int8 codes q of its weighted root-mean-square
    norm, one fp32 scale a row (q * scale[:, None] stands for the norm).
    ``hidden`` may name the output, x or residual themselves included."""
    _, q, scale, hidden = _norm(x, weight, residual, eps, hidden, False, stream)
    return q, scale, hidden


def littlebit_rmsnorm_fwd(x: torch.Tensor, weight: torch.Tensor, residual: Optional[torch.Tensor] = None,
                          eps: float = 1e-5, hidden: Optional[torch.Tensor] = None,
                          stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """(y, hidden) of the dense norm, both in x's type; hidden as for
    littlebit_rmsnorm_q8."""
    y, _, _, hidden = _norm(x, weight, residual, eps, hidden, True, stream)
    return y, hidden


def littlebit_rmsnorm_bwd(dy: torch.Tensor, hidden: torch.Tensor, weight: torch.Tensor,
                          dhidden: Optional[torch.Tensor] = None, eps: float = 1e-5,
                          stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """(dx, dweight): the gradient of x (and of the residual: it is the same)
    from the gradients of y and, where it has one, of hidden; dweight in fp32.
    For the 8-bit output, dy is the gradient of the values its codes stand for,
    and the rounding is passed straight through."""
    code, shape, device = _first("hidden", hidden, _HALF)
    dtype = hidden.dtype
    ldh = _matrix("hidden", hidden, dtype, device, shape)
    rows, n = shape
    lddy = _matrix("dy", dy, dtype, device, shape)
    _vector("weight", weight, dtype, device, n)
    lddh = 0 if dhidden is None else _matrix("dhidden", dhidden, dtype, device, shape)
    if _recording():
        _no_history(dy, hidden, weight, dhidden)
    ctx, sp = _on(device, stream)
    with ctx:
        dx = _new(rows, n, dtype, device)
        dweight = _empty((n,), (1,), dtype=torch.float32, device=device)
        need = LIB.littlebit_rmsnorm_bwd_workspace_bytes(rows, n)
        ws = _empty((need,), (1,), dtype=torch.uint8, device=device)
        _check(LIB.littlebit_rmsnorm_bwd(
            dy.data_ptr(), lddy, None if dhidden is None else dhidden.data_ptr(), lddh, hidden.data_ptr(), ldh,
            weight.data_ptr(), code, rows, n, eps, dx.data_ptr(), n, dweight.data_ptr(), ws.data_ptr(), need, sp))
    if stream is not None:
        _keep(stream, dy, hidden, weight, dhidden)
    return dx, dweight


# -------------------------------------------------------------------------------------------------- 8-bit product

def littlebit_q8_quantize(x: torch.Tensor, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """(q, scale): int8 codes of each row with one fp32 scale, largest value 127."""
    code, shape, device = _first("x", x, _DTYPE)
    ldx = _matrix("x", x, x.dtype, device, shape)
    rows, n = shape
    if _recording():
        _no_history(x)
    ctx, sp = _on(device, stream)
    with ctx:
        q, ldq = _codes(rows, n, device)
        scale = _empty((rows,), (1,), dtype=torch.float32, device=device)
        _check(LIB.littlebit_q8_quantize(x.data_ptr(), ldx, code, rows, n, q.data_ptr(), ldq, scale.data_ptr(), sp))
    if stream is not None:
        _keep(stream, x)
    return q, scale


def littlebit_q8_linear_fwd(xq: torch.Tensor, xscale: torch.Tensor, wq: torch.Tensor, wscale: torch.Tensor,
                            dtype: torch.dtype = torch.float16, out: Optional[torch.Tensor] = None,
                            stream=None) -> torch.Tensor:
    """y[t, o] = xscale[t] * wscale[o] * sum_k xq[t, k] * wq[o, k] in `dtype`
    (that of `out`, where it is given)."""
    _, (batch, n), device = _first("xq", xq, _INT8)
    ldx = _matrix("xq", xq, torch.int8, device, (batch, n))
    m = _first("wq", wq, _INT8)[1][0]
    ldw = _matrix("wq", wq, torch.int8, device, (m, n))
    _vector("xscale", xscale, torch.float32, device, batch)
    _vector("wscale", wscale, torch.float32, device, m)
    ldy = m
    if out is not None:
        dtype = out.dtype
        ldy = _matrix("out", out, dtype, device, (batch, m))
    code = _DTYPE.get(dtype)
    if code is None:
        raise ValueError("the output must be float32, float16 or bfloat16")
    if _recording():
        _no_history(xscale, wscale, out)
    ctx, sp = _on(device, stream)
    with ctx:
        y = out if out is not None else _new(batch, m, dtype, device)
        _check(LIB.littlebit_q8_linear_fwd(xq.data_ptr(), ldx, xscale.data_ptr(), wq.data_ptr(), ldw,
                                           wscale.data_ptr(), batch, m, n, y.data_ptr(), ldy, code, sp))
    if stream is not None:
        _keep(stream, xq, xscale, wq, wscale, out)
    return y


# --------------------------------------------------------------------------------------------------- log probabilities

def littlebit_logprobs_fwd(logits: torch.Tensor, targets: Optional[torch.Tensor] = None, top: int = 0,
                           stream=None) -> Tuple[Optional[torch.Tensor], ...]:
    """(logprob, entropy, lse, top_logprob, top_index) of each row of logits.
    logprob is None without targets; the last two are None for top = 0.  A
    negative target stands for no token (logprob 0).  lse holds each row's
    maximum and, behind it, log sum exp(x - maximum): lse.sum(0) is the
    logarithm of the sum of exponentials."""
    code, shape, device = _first("logits", logits, _DTYPE)
    ld = _matrix("logits", logits, logits.dtype, device, shape)
    rows, vocab = shape
    if targets is not None:
        _vector("targets", targets, torch.int64, device, rows)
    if _recording():
        _no_history(logits)
    ctx, sp = _on(device, stream)
    with ctx:
        logprob = values = places = ws = None
        if targets is not None:
            logprob = _empty((rows,), (1,), dtype=torch.float32, device=device)
        entropy = _empty((rows,), (1,), dtype=torch.float32, device=device)
        lse = _new(2, rows, torch.float32, device)
        if 0 < top <= LB_TOP_MAX:   # the call refuses others
            values = _new(rows, top, torch.float32, device)
            places = _new(rows, top, torch.int64, device)
        need = LIB.littlebit_logprobs_workspace_bytes(rows, vocab, code, top)
        if need:
            ws = _empty((need,), (1,), dtype=torch.uint8, device=device)
        _check(LIB.littlebit_logprobs_fwd(
            logits.data_ptr(), ld, code, rows, vocab, None if targets is None else targets.data_ptr(),
            None if logprob is None else logprob.data_ptr(), entropy.data_ptr(), lse.data_ptr(), top,
            None if values is None else values.data_ptr(), None if places is None else places.data_ptr(),
            None if ws is None else ws.data_ptr(), need, sp))
    if stream is not None:
        _keep(stream, logits, targets)
    return logprob, entropy, lse, values, places


def littlebit_logprobs_bwd(logits: torch.Tensor, targets: Optional[torch.Tensor], lse: torch.Tensor,
                           entropy: Optional[torch.Tensor] = None, dlogprob: Optional[torch.Tensor] = None,
                           dentropy: Optional[torch.Tensor] = None, top_index: Optional[torch.Tensor] = None,
                           dtop: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                           stream=None) -> torch.Tensor:
    """The gradient of the logits, in their type, from the gradients of
    littlebit_logprobs_fwd's logprob, entropy and top_logprob (None: it has
    none).  lse, entropy and top_index are that call's outputs.  ``out`` may be
    the logits themselves."""
    code, shape, device = _first("logits", logits, _DTYPE)
    ld = _matrix("logits", logits, logits.dtype, device, shape)
    rows, vocab = shape
    _table("lse", lse, torch.float32, device, (2, rows))
    if dlogprob is not None:
        if targets is None:
            raise ValueError("dlogprob needs targets")
        _vector("targets", targets, torch.int64, device, rows)
        _vector("dlogprob", dlogprob, torch.float32, device, rows)
    if dentropy is not None:
        if entropy is None:
            raise ValueError("dentropy needs entropy")
        _vector("entropy", entropy, torch.float32, device, rows)
        _vector("dentropy", dentropy, torch.float32, device, rows)
    top = 0
    if dtop is not None:
        if top_index is None or not torch.is_tensor(dtop) or dtop.dim() != 2:
            raise ValueError("dtop needs top_index, one row of each a token")
        top = dtop.shape[1]
        _table("top_index", top_index, torch.int64, device, (rows, top))
        _table("dtop", dtop, torch.float32, device, (rows, top))
    ldd = vocab if out is None else _matrix("out", out, logits.dtype, device, shape)
    if _recording():
        _no_history(logits, lse, entropy, dlogprob, dentropy, dtop, out)
    ctx, sp = _on(device, stream)
    with ctx:
        d = _new(rows, vocab, logits.dtype, device) if out is None else out
        _check(LIB.littlebit_logprobs_bwd(
            logits.data_ptr(), ld, code, rows, vocab, None if dlogprob is None else targets.data_ptr(), lse.data_ptr(),
            None if dentropy is None else entropy.data_ptr(), None if dlogprob is None else dlogprob.data_ptr(),
            None if dentropy is None else dentropy.data_ptr(), top, top_index.data_ptr() if top else None,
            dtop.data_ptr() if top else None, d.data_ptr(), ldd, sp))
    if stream is not None:
        _keep(stream, logits, targets, lse, entropy, dlogprob, dentropy, top_index, dtop, out)
    return d


# -------------------------------------------------------------------------------------------------------- the head

@dataclass
class Q8Linear:
    """A dense weight in 8 bits, one scale an output channel (m x n codes)."""
    q: torch.Tensor
    scale: torch.Tensor

    @staticmethod
    def from_weight(weight: torch.Tensor) -> "Q8Linear":
        """Quantises a dense m x n weight (fp32, fp16 or bf16, on the GPU; a parameter's values)."""
        with torch.no_grad():
            return Q8Linear(*littlebit_q8_quantize(weight))

    def __call__(self, xq, xscale, dtype=torch.float16, out=None, stream=None) -> torch.Tensor:
        return littlebit_q8_linear_fwd(xq, xscale, self.q, self.scale, dtype, out, stream)


@dataclass
class LittleBitHead:
    """The end of a model whose blocks are LittleBit layers: the last norm and
    the head, kept dense in 8 bits."""
    norm: torch.Tensor
    linear: Q8Linear
    eps: float = 1e-5

    @staticmethod
    def from_weights(norm: torch.Tensor, weight: torch.Tensor, eps: float = 1e-5) -> "LittleBitHead":
        return LittleBitHead(norm=norm.detach(), linear=Q8Linear.from_weight(weight), eps=eps)

    def logits(self, x: torch.Tensor, residual: Optional[torch.Tensor] = None, dtype=torch.float32,
               stream=None) -> torch.Tensor:
        """Logits of the tokens x (the last block's output, before it joins the residual stream)."""
        q, scale, _ = littlebit_rmsnorm_q8(x, self.norm, residual, self.eps, stream=stream)
        return self.linear(q, scale, dtype, stream=stream)

    def logprobs(self, x: torch.Tensor, targets: torch.Tensor, residual: Optional[torch.Tensor] = None, top: int = 0,
                 dtype=torch.float32, max_logit_bytes: int = 1 << 30, stream=None):
        """(logprob, entropy, top_logprob, top_index) of the given tokens over a
        text of any length: the logits are formed for as many tokens at a time
        as fit in `max_logit_bytes`, and never kept.  The perplexity of the text is
        exp(-logprob[targets >= 0].mean()): tokens that are not given (negative
        targets) have logprob 0 and are no part of the mean."""
        _, shape, device = _first("x", x, _HALF)
        rows = shape[0]
        if residual is not None:   # whole: a part of a longer one would fit its part of x
            _matrix("residual", residual, x.dtype, device, shape)
        _vector("targets", targets, torch.int64, device, rows)
        vocab = self.linear.q.shape[0]
        step = max_logit_bytes // (vocab * torch.empty((), dtype=dtype).element_size())
        step = min(max(1, step), 1 << 20)   # a call takes 2^21 rows at most
        parts = []
        for t in range(0, max(rows, 1), step):
            r = None if residual is None else residual[t:t + step]
            logits = self.logits(x[t:t + step], r, dtype, stream)
            logprob, entropy, _, values, places = littlebit_logprobs_fwd(logits, targets[t:t + step], top, stream)
            del logits   # before the next part's are formed
            parts.append((logprob, entropy, values, places))
        if len(parts) == 1:
            return parts[0]
        ctx = torch.cuda.stream(stream) if stream is not None else _HERE
        with ctx:
            return tuple(torch.cat(p) if p[0] is not None else None for p in zip(*parts))
