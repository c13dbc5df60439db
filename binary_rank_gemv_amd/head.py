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
device); the tensors of a call lie on one device, which need not be the
current one.  Importing this module raises if the library has not been built
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


def _on(t: torch.Tensor, stream):
    """(context, stream pointer): the device of `t` current, allocations on `stream`."""
    if stream is not None:
        if stream.device != t.device:
            raise ValueError(f"stream is on {stream.device}, the tensors are on {t.device}")
        return torch.cuda.stream(stream), int(stream.cuda_stream)
    index = t.device.index
    here = torch.cuda.current_device()
    return (_HERE if index == here else torch.cuda.device(index)), torch.cuda.current_stream(index).cuda_stream


def _matrix(name: str, t: torch.Tensor, dtype, device, shape=None):
    """Checks a row-major matrix argument (unit column stride, any row stride)."""
    if not torch.is_tensor(t) or t.dim() != 2 or not t.is_cuda:
        raise ValueError(f"{name} must be a 2-D CUDA tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, is {t.dtype}")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, the call is on {device}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, has {tuple(t.shape)}")
    rows, cols = t.shape
    if cols > 1 and t.stride(1) != 1 or rows > 1 and t.stride(0) < cols:
        raise ValueError(f"{name} must have unit column stride and rows that do not overlap")


def _vector(name: str, t: torch.Tensor, dtype, device, n: int):
    if not torch.is_tensor(t) or t.dim() != 1 or not t.is_cuda or t.dtype != dtype or t.device != device:
        raise ValueError(f"{name} must be a 1-D {dtype} tensor on {device}")
    if t.shape[0] != n or n > 1 and t.stride(0) != 1:
        raise ValueError(f"{name} must be {n} contiguous values")


def _table(name: str, t: torch.Tensor, dtype, device, shape):
    if not torch.is_tensor(t) or t.dtype != dtype or t.device != device or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)} on {device}")


def _ld(t: torch.Tensor) -> int:
    """Row stride; of a single row, whatever its stride says, at least its length."""
    return max(t.stride(0), t.shape[1])


def _codes(rows: int, n: int, device) -> torch.Tensor:
    """Room for int8 codes, rows 16 bytes aligned (the product's fast case)."""
    return torch.empty((rows, (n + 15) // 16 * 16), dtype=torch.int8, device=device)[:, :n] if n % 16 else \
        torch.empty((rows, n), dtype=torch.int8, device=device)


# ------------------------------------------------------------------------------------------------------- norm

def _norm(x, weight, residual, eps, hidden, dense, stream):
    dtype = _HALF.get(x.dtype) if torch.is_tensor(x) else None
    if dtype is None:
        raise ValueError("x must be a float16 or bfloat16 tensor")
    _matrix("x", x, x.dtype, None)
    rows, n = x.shape
    device = x.device
    _vector("weight", weight, x.dtype, device, n)
    if residual is not None:
        _matrix("residual", residual, x.dtype, device, x.shape)
    elif hidden is not None:
        raise ValueError("hidden is an output of the residual's addition: give a residual")
    if hidden is not None:
        _matrix("hidden", hidden, x.dtype, device, x.shape)
    ctx, sp = _on(x, stream)
    with ctx:
        if residual is not None and hidden is None:
            hidden = torch.empty((rows, n), dtype=x.dtype, device=device)
        if dense:
            y, q, scale = torch.empty((rows, n), dtype=x.dtype, device=device), None, None
        else:
            y, q, scale = None, _codes(rows, n, device), torch.empty(rows, dtype=torch.float32, device=device)
        _check(LIB.littlebit_rmsnorm_fwd(
            x.data_ptr(), _ld(x), residual.data_ptr() if residual is not None else None,
            _ld(residual) if residual is not None else 0, weight.data_ptr(), dtype, rows, n, eps,
            hidden.data_ptr() if hidden is not None else None, _ld(hidden) if hidden is not None else 0,
            y.data_ptr() if dense else None, n, q.data_ptr() if q is not None else None,
            _ld(q) if q is not None else 0, scale.data_ptr() if scale is not None else None, sp))
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
    dtype = _HALF.get(hidden.dtype) if torch.is_tensor(hidden) else None
    if dtype is None:
        raise ValueError("hidden must be a float16 or bfloat16 tensor")
    _matrix("hidden", hidden, hidden.dtype, None)
    rows, n = hidden.shape
    device = hidden.device
    _matrix("dy", dy, hidden.dtype, device, hidden.shape)
    _vector("weight", weight, hidden.dtype, device, n)
    if dhidden is not None:
        _matrix("dhidden", dhidden, hidden.dtype, device, hidden.shape)
    ctx, sp = _on(hidden, stream)
    with ctx:
        dx = torch.empty((rows, n), dtype=hidden.dtype, device=device)
        dweight = torch.empty(n, dtype=torch.float32, device=device)
        need = LIB.littlebit_rmsnorm_bwd_workspace_bytes(rows, n)
        ws = torch.empty(need, dtype=torch.uint8, device=device)
        _check(LIB.littlebit_rmsnorm_bwd(
            dy.data_ptr(), _ld(dy), dhidden.data_ptr() if dhidden is not None else None,
            _ld(dhidden) if dhidden is not None else 0, hidden.data_ptr(), _ld(hidden), weight.data_ptr(), dtype,
            rows, n, eps, dx.data_ptr(), n, dweight.data_ptr(), ws.data_ptr(), need, sp))
    return dx, dweight


# -------------------------------------------------------------------------------------------------- 8-bit product

def littlebit_q8_quantize(x: torch.Tensor, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """(q, scale): int8 codes of each row with one fp32 scale, largest value 127."""
    dtype = _DTYPE.get(x.dtype) if torch.is_tensor(x) else None
    if dtype is None:
        raise ValueError("x must be a float32, float16 or bfloat16 tensor")
    _matrix("x", x, x.dtype, None)
    rows, n = x.shape
    ctx, sp = _on(x, stream)
    with ctx:
        q = _codes(rows, n, x.device)
        scale = torch.empty(rows, dtype=torch.float32, device=x.device)
        _check(LIB.littlebit_q8_quantize(x.data_ptr(), _ld(x), dtype, rows, n, q.data_ptr(), _ld(q),
                                         scale.data_ptr(), sp))
    return q, scale


def littlebit_q8_linear_fwd(xq: torch.Tensor, xscale: torch.Tensor, wq: torch.Tensor, wscale: torch.Tensor,
                            dtype: torch.dtype = torch.float16, out: Optional[torch.Tensor] = None,
                            stream=None) -> torch.Tensor:
    """y[t, o] = xscale[t] * wscale[o] * sum_k xq[t, k] * wq[o, k] in `dtype`
    (that of `out`, where it is given)."""
    _matrix("xq", xq, torch.int8, None)
    device = xq.device
    _matrix("wq", wq, torch.int8, device)
    batch, n = xq.shape
    m = wq.shape[0]
    if wq.shape[1] != n:
        raise ValueError(f"wq has rows of {wq.shape[1]}, xq of {n}")
    _vector("xscale", xscale, torch.float32, device, batch)
    _vector("wscale", wscale, torch.float32, device, m)
    if out is not None:
        dtype = out.dtype
        _matrix("out", out, dtype, device, (batch, m))
    code = _DTYPE.get(dtype)
    if code is None:
        raise ValueError("the output must be float32, float16 or bfloat16")
    ctx, sp = _on(xq, stream)
    with ctx:
        y = out if out is not None else torch.empty((batch, m), dtype=dtype, device=device)
        _check(LIB.littlebit_q8_linear_fwd(xq.data_ptr(), _ld(xq), xscale.data_ptr(), wq.data_ptr(), _ld(wq),
                                           wscale.data_ptr(), batch, m, n, y.data_ptr(), _ld(y), code, sp))
    return y


# --------------------------------------------------------------------------------------------------- log probabilities

def littlebit_logprobs_fwd(logits: torch.Tensor, targets: Optional[torch.Tensor] = None, top: int = 0,
                           stream=None) -> Tuple[Optional[torch.Tensor], ...]:
    """(logprob, entropy, lse, top_logprob, top_index) of each row of logits.
    logprob is None without targets; the last two are None for top = 0.  A
    negative target stands for no token (logprob 0).  lse holds each row's
    maximum and, behind it, log sum exp(x - maximum): lse.sum(0) is the
    logarithm of the sum of exponentials."""
    code = _DTYPE.get(logits.dtype) if torch.is_tensor(logits) else None
    if code is None:
        raise ValueError("logits must be a float32, float16 or bfloat16 tensor")
    _matrix("logits", logits, logits.dtype, None)
    rows, vocab = logits.shape
    device = logits.device
    if targets is not None:
        _vector("targets", targets, torch.int64, device, rows)
    ctx, sp = _on(logits, stream)
    with ctx:
        stats = torch.empty((4, rows), dtype=torch.float32, device=device)
        logprob, entropy, lse = stats[0], stats[1], stats[2:]
        values = places = None
        if top > 0:
            values = torch.empty((rows, top), dtype=torch.float32, device=device)
            places = torch.empty((rows, top), dtype=torch.int64, device=device)
        need = LIB.littlebit_logprobs_workspace_bytes(rows, vocab, code, top)
        ws = torch.empty(need, dtype=torch.uint8, device=device) if need else None
        _check(LIB.littlebit_logprobs_fwd(
            logits.data_ptr(), _ld(logits), code, rows, vocab, targets.data_ptr() if targets is not None else None,
            logprob.data_ptr() if targets is not None else None, entropy.data_ptr(), lse.data_ptr(), top,
            values.data_ptr() if values is not None else None, places.data_ptr() if places is not None else None,
            ws.data_ptr() if ws is not None else None, need, sp))
    return logprob if targets is not None else None, entropy, lse, values, places


def littlebit_logprobs_bwd(logits: torch.Tensor, targets: Optional[torch.Tensor], lse: torch.Tensor,
                           entropy: Optional[torch.Tensor] = None, dlogprob: Optional[torch.Tensor] = None,
                           dentropy: Optional[torch.Tensor] = None, top_index: Optional[torch.Tensor] = None,
                           dtop: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                           stream=None) -> torch.Tensor:
    """The gradient of the logits, in their type, from the gradients of
    littlebit_logprobs_fwd's logprob, entropy and top_logprob (None: it has
    none).  lse, entropy and top_index are that call's outputs.  ``out`` may be
    the logits themselves."""
    code = _DTYPE.get(logits.dtype) if torch.is_tensor(logits) else None
    if code is None:
        raise ValueError("logits must be a float32, float16 or bfloat16 tensor")
    _matrix("logits", logits, logits.dtype, None)
    rows, vocab = logits.shape
    device = logits.device
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
        if top_index is None or dtop.dim() != 2:
            raise ValueError("dtop needs top_index, one row of each a token")
        top = dtop.shape[1]
        _table("top_index", top_index, torch.int64, device, (rows, top))
        _table("dtop", dtop, torch.float32, device, (rows, top))
    if out is not None:
        _matrix("out", out, logits.dtype, device, logits.shape)
    ctx, sp = _on(logits, stream)
    with ctx:
        d = out if out is not None else torch.empty((rows, vocab), dtype=logits.dtype, device=device)
        _check(LIB.littlebit_logprobs_bwd(
            logits.data_ptr(), _ld(logits), code, rows, vocab,
            targets.data_ptr() if dlogprob is not None else None, lse.data_ptr(),
            entropy.data_ptr() if dentropy is not None else None,
            dlogprob.data_ptr() if dlogprob is not None else None,
            dentropy.data_ptr() if dentropy is not None else None, top,
            top_index.data_ptr() if top else None, dtop.data_ptr() if top else None, d.data_ptr(), _ld(d), sp))
    return d


# -------------------------------------------------------------------------------------------------------- the head

@dataclass
class Q8Linear:
    """A dense weight in 8 bits, one scale an output channel (m x n codes)."""
    q: torch.Tensor
    scale: torch.Tensor

    @staticmethod
    def from_weight(weight: torch.Tensor) -> "Q8Linear":
        """Quantises a dense m x n weight (fp32, fp16 or bf16, on the GPU)."""
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
        return LittleBitHead(norm=norm, linear=Q8Linear.from_weight(weight), eps=eps)

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
        exp(-mean logprob)."""
        rows = x.shape[0]
        _vector("targets", targets, torch.int64, x.device, rows)
        vocab = self.linear.q.shape[0]
        step = max(1, max_logit_bytes // (vocab * torch.empty((), dtype=dtype).element_size()))
        parts = []
        for t in range(0, max(rows, 1), step):
            r = None if residual is None else residual[t:t + step]
            logits = self.logits(x[t:t + step], r, dtype, stream)
            logprob, entropy, _, values, places = littlebit_logprobs_fwd(logits, targets[t:t + step], top, stream)
            parts.append((logprob, entropy, values, places))
        if len(parts) == 1:
            return parts[0]
        ctx = torch.cuda.stream(stream) if stream is not None else _HERE
        with ctx:
            return tuple(torch.cat(p) if p[0] is not None else None for p in zip(*parts))
