"""ctypes binding of ``include/littlebit_attn.h`` (argument marshalling only):
what lies between a block's query, key and value projections and its output
projection, in ``_lib/liblittlebit_attn.so``.

* ``littlebit_rope_fwd(q, k, positions, inv_freq, q_weight, k_weight)`` ->
  (q_out, k_out): each head normed and turned to its position
* ``littlebit_rope_bwd(dq, dk, positions, inv_freq, q, k, q_weight, k_weight)``
  -> (dq_in, dk_in, dq_weight, dk_weight)
* ``littlebit_cache_append(cache, batch, k, v, q, positions, inv_freq, ...)`` ->
  q_out: the same, keys and values into a paged cache
* ``littlebit_cache_attention_fwd(q, cache, batch, tree)`` -> out: the attention
  over the cache, of single tokens, prompts, or trees of drafted tokens
* ``littlebit_cache_accept(cache, batch, path)``: a verified tree's accepted
  tokens moved together in the cache
* ``LittleBitCache`` holds the pages, ``CacheBatch`` the sequences of a call;
  ``LittleBitAttention`` is the whole of it, from a block's input to its output
  projection, around four LittleBit layers

Queries, keys and values are tokens x heads x dim tensors (fp16 or bf16) whose
channels lie together; views into a fused projection's output are taken as
they are.

Work is enqueued on ``stream`` (default: the current stream of the tensors'
device), which the caller lets wait for what the tensors' own stream still
writes; their memory is not reused before ``stream`` has passed the call.  The
tensors of a call lie on one device, which need not be the current one.

Nothing is recorded for autograd: the backward pass is a call of its own, and
while gradients are recorded a tensor that requires one is refused.

Importing this module raises if the library has not been built
(``python -m binary_rank_gemv_amd.build``): there is no fallback path.
"""

from __future__ import annotations

import ctypes
import math
import os
from dataclasses import dataclass
from typing import Optional, Tuple

import torch

from .littlebit import LB_F16, LB_OK, LittleBitError, LittleBitLayer, littlebit_linear_fwd

ATTN_LIB_PATH = os.environ.get("LITTLEBIT_ATTN_LIBRARY") or os.path.join(
    os.path.dirname(os.path.abspath(__file__)), "_lib", "liblittlebit_attn.so")

LB_BF16 = 2
LB_HEAD_MAX_DIM = 256
LB_TREE_MAX = 64

ATTN_EXPORTED = (
    "littlebit_rope_fwd", "littlebit_rope_bwd_workspace_bytes", "littlebit_rope_bwd", "littlebit_cache_append",
    "littlebit_cache_attention_workspace_bytes", "littlebit_cache_attention_fwd", "littlebit_cache_accept",
    "littlebit_attn_last_error",
)

_HALF = {torch.float16: LB_F16, torch.bfloat16: LB_BF16}

_vp, _i64, _i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32


class _Heads(ctypes.Structure):
    _fields_ = [("p", _vp), ("token_stride", _i64), ("head_stride", _i64), ("heads", _i32)]


class _Rope(ctypes.Structure):
    _fields_ = [("positions", _vp), ("inv_freq", _vp), ("rot", _i32), ("interleaved", _i32), ("q_weight", _vp),
                ("k_weight", _vp), ("eps", ctypes.c_float)]


class _Cache(ctypes.Structure):
    _fields_ = [("k", _vp), ("v", _vp), ("page_stride", _i64), ("head_stride", _i64), ("slot_stride", _i64),
                ("pages", _i32), ("heads", _i32), ("page_size", _i32), ("dim", _i32), ("dtype", _i32)]


class _Batch(ctypes.Structure):
    _fields_ = [("starts", _vp), ("lens", _vp), ("table", _vp), ("table_stride", _i64), ("seqs", _i32),
                ("columns", _i32)]


def _load():
    if not os.path.exists(ATTN_LIB_PATH):
        raise ImportError(f"{ATTN_LIB_PATH} is missing: build it with `python -m binary_rank_gemv_amd.build`")
    lib = ctypes.CDLL(ATTN_LIB_PATH)
    # structs and optional pointers alike are handed over as addresses
    sigs = {
        "littlebit_rope_fwd": (_i32, [_vp, _vp, _vp, _i32, _i64, _i32, _vp, _vp, _vp]),
        "littlebit_rope_bwd_workspace_bytes": (ctypes.c_size_t, [_i64, _i32, _i32, _i32]),
        "littlebit_rope_bwd": (_i32, [_vp, _vp, _vp, _vp, _vp, _i32, _i64, _i32, _vp, _vp, _vp, _vp, _vp, ctypes.c_size_t,
                                      _vp]),
        "littlebit_cache_append": (_i32, [_vp, _vp, _i64, _vp, _vp, _vp, _vp, _vp, _vp]),
        "littlebit_cache_attention_workspace_bytes": (ctypes.c_size_t, [_vp, _vp, _i64, _i32]),
        "littlebit_cache_attention_fwd": (_i32, [_vp, _vp, _i64, _vp, _vp, ctypes.c_float, _vp, _vp, _vp, ctypes.c_size_t,
                                                 _vp]),
        "littlebit_cache_accept": (_i32, [_vp, _vp, _vp, _i32, _vp]),
        "littlebit_attn_last_error": (ctypes.c_char_p, []),
    }
    for name, (res, args) in sigs.items():
        f = getattr(lib, name)
        f.restype, f.argtypes = res, args
    return lib


LIB = _load()


def littlebit_attn_last_error() -> str:
    return LIB.littlebit_attn_last_error().decode()


def _check(status: int):
    if status != LB_OK:
        raise LittleBitError(status, littlebit_attn_last_error())


class _Here:
    def __enter__(self):
        return None

    def __exit__(self, *_):
        return False


_HERE = _Here()
_empty = torch.empty_strided
_raw_stream = torch._C._cuda_getCurrentRawStream
_ref = ctypes.byref
_recording = torch.is_grad_enabled
_current = torch._C._cuda_getDevice


def _on(index, stream):
    """(context, stream pointer): device `index` current, allocations on `stream`."""
    if stream is not None:
        if stream.device.index != index:
            raise ValueError(f"stream is on {stream.device}, the tensors are on cuda:{index}")
        return torch.cuda.stream(stream), int(stream.cuda_stream)
    return (_HERE if index == _current() else torch.cuda.device(index)), _raw_stream(index)


def _keep(stream, *tensors):
    """Tensors that a call reads or writes on a stream given by name: freed ones are
    not handed out again on their own stream while that one still runs."""
    for t in tensors:
        if t is not None:
            t.record_stream(stream)


def _no_history(*tensors):
    for t in tensors:
        if t is not None and t.requires_grad:
            raise ValueError("a tensor of the call requires a gradient, which would be lost: these calls record nothing for "
                             "autograd; call under torch.no_grad() and take the gradient by littlebit_rope_bwd")


# The checks ask for everything at once, and for the reason only where something is wrong: these calls are short.

def _first(name: str, t: torch.Tensor):
    """(type code, device index) of the tensor that the others are held to."""
    code = _HALF.get(t.dtype) if torch.is_tensor(t) else None
    if code is None:
        raise ValueError(f"{name} must be a tensor of {' or '.join(str(d) for d in _HALF)}")
    index = t.get_device()
    if index < 0 or t.dim() != 3:
        raise ValueError(f"{name} must be a tokens x heads x dim CUDA tensor")
    return code, index


def _heads(name: str, t: torch.Tensor, dtype, index: int, tokens: int, dim: int, heads: int = 0) -> _Heads:
    """A tokens x heads x dim argument; any number of heads for heads = 0."""
    if torch.is_tensor(t) and t.dim() == 3:
        n, h, d = t.shape
        st, sh, sd = t.stride()
        if n == tokens and d == dim and t.dtype is dtype and t.get_device() == index and (h == heads or not heads) \
                and (sd == 1 or d == 1):
            return _Heads(t.data_ptr(), st, sh, h)
        if t.dtype is not dtype:
            raise ValueError(f"{name} must be {dtype}, is {t.dtype}")
        if t.get_device() != index:
            raise ValueError(f"{name} is on {t.device}, the call is on cuda:{index}")
        if n == tokens and d == dim and (h == heads or not heads):
            raise ValueError(f"the channels of {name} must lie together")
        raise ValueError(f"{name} must have shape ({tokens}, {heads or h}, {dim}), has {tuple(t.shape)}")
    raise ValueError(f"{name} must be a tokens x heads x dim CUDA tensor")


def _ints(name: str, t: torch.Tensor, index: int, n: int, dtype=torch.int32) -> int:
    if torch.is_tensor(t) and t.dtype is dtype and t.get_device() == index and t.dim() == 1:
        if t.shape[0] == n and t.is_contiguous():
            return t.data_ptr()
        raise ValueError(f"{name} must be {n} contiguous values")
    raise ValueError(f"{name} must be a 1-D {dtype} tensor on cuda:{index}")


def _rope(positions, inv_freq, q_weight, k_weight, eps, interleaved, dtype, index, tokens, dim) -> _Rope:
    half, pos, inv = 0, None, None
    if inv_freq is not None:
        half = inv_freq.shape[0] if torch.is_tensor(inv_freq) and inv_freq.dim() == 1 else 0
        inv = _ints("inv_freq", inv_freq, index, half, torch.float32)
        if positions is None:
            raise ValueError("inv_freq needs positions")
        pos = _ints("positions", positions, index, tokens)
    return _Rope(pos, inv, 2 * half, 1 if interleaved else 0,
                 None if q_weight is None else _ints("q_weight", q_weight, index, dim, dtype),
                 None if k_weight is None else _ints("k_weight", k_weight, index, dim, dtype), eps)


def _new_heads(tokens, heads, dim, dtype, index):
    """A new tensor of heads, and its argument."""
    row = heads * dim
    t = _empty((tokens, heads, dim), (row, dim, 1), dtype=dtype, device=index)
    return t, _Heads(t.data_ptr(), row, dim, heads)


def _out(name, t, dtype, index, tokens, dim, heads):
    """An output that is given, or a new one, and its argument."""
    if t is None:
        return _new_heads(tokens, heads, dim, dtype, index)
    return t, _heads(name, t, dtype, index, tokens, dim, heads)


# --------------------------------------------------------------------------------------- head norm and rotation

def littlebit_rope_fwd(q: Optional[torch.Tensor], k: Optional[torch.Tensor], positions: Optional[torch.Tensor] = None,
                       inv_freq: Optional[torch.Tensor] = None, q_weight: Optional[torch.Tensor] = None,
                       k_weight: Optional[torch.Tensor] = None, eps: float = 1e-5, interleaved: bool = False,
                       q_out: Optional[torch.Tensor] = None, k_out: Optional[torch.Tensor] = None,
                       stream=None) -> Tuple[Optional[torch.Tensor], Optional[torch.Tensor]]:
    """(q_out, k_out): every head normed (where its weight is given) and its first
    2 len(inv_freq) channels turned by positions * inv_freq (where that is).  q or
    k may be None.  ``q_out`` and ``k_out`` may name the outputs, q and k
    themselves included."""
    one = q if q is not None else k
    code, index = _first("q" if q is not None else "k", one)
    dtype, (tokens, _, dim) = one.dtype, one.shape
    hq = None if q is None else _heads("q", q, dtype, index, tokens, dim)
    hk = None if k is None else _heads("k", k, dtype, index, tokens, dim)
    if (q is None and q_out is not None) or (k is None and k_out is not None):
        raise ValueError("an output without its input")
    rope = _rope(positions, inv_freq, q_weight, k_weight, eps, interleaved, dtype, index, tokens, dim)
    if _recording():
        _no_history(q, k, inv_freq, q_weight, k_weight, q_out, k_out)
    ctx, sp = _on(index, stream)
    with ctx:
        oq = ok = None
        if q is not None:
            q_out, oq = _out("q_out", q_out, dtype, index, tokens, dim, hq.heads)
        if k is not None:
            k_out, ok = _out("k_out", k_out, dtype, index, tokens, dim, hk.heads)
        _check(LIB.littlebit_rope_fwd(hq and _ref(hq), hk and _ref(hk), _ref(rope), code, tokens, dim, oq and _ref(oq),
                                      ok and _ref(ok), sp))
    if stream is not None:
        _keep(stream, q, k, positions, inv_freq, q_weight, k_weight, q_out, k_out)
    return q_out, k_out


def littlebit_rope_bwd(dq: Optional[torch.Tensor], dk: Optional[torch.Tensor], positions: Optional[torch.Tensor] = None,
                       inv_freq: Optional[torch.Tensor] = None, q: Optional[torch.Tensor] = None,
                       k: Optional[torch.Tensor] = None, q_weight: Optional[torch.Tensor] = None,
                       k_weight: Optional[torch.Tensor] = None, eps: float = 1e-5, interleaved: bool = False,
                       dq_in: Optional[torch.Tensor] = None, dk_in: Optional[torch.Tensor] = None,
                       stream=None) -> Tuple[Optional[torch.Tensor], ...]:
    """(dq_in, dk_in, dq_weight, dk_weight): from the gradients of
    littlebit_rope_fwd's outputs (either may be None) those of its inputs, and the
    weights' in fp32 (None without a weight).  q and k are that call's inputs;
    they are needed with a weight only.  ``dq_in`` and ``dk_in`` may name the
    outputs, dq and dk themselves included."""
    one = dq if dq is not None else dk
    code, index = _first("dq" if dq is not None else "dk", one)
    dtype, (tokens, _, dim) = one.dtype, one.shape
    if dq is None:
        q = q_weight = None
    if dk is None:
        k = k_weight = None
    hdq = None if dq is None else _heads("dq", dq, dtype, index, tokens, dim)
    hdk = None if dk is None else _heads("dk", dk, dtype, index, tokens, dim)
    if (dq is None and dq_in is not None) or (dk is None and dk_in is not None):
        raise ValueError("an output without its input")
    rope = _rope(positions, inv_freq, q_weight, k_weight, eps, interleaved, dtype, index, tokens, dim)
    hq = _heads("q", q, dtype, index, tokens, dim, hdq.heads) if q_weight is not None else None
    hk = _heads("k", k, dtype, index, tokens, dim, hdk.heads) if k_weight is not None else None
    if _recording():
        _no_history(dq, dk, q, k, inv_freq, q_weight, k_weight, dq_in, dk_in)
    ctx, sp = _on(index, stream)
    with ctx:
        oq = ok = dqw = dkw = ws = None
        need = 0
        if dq is not None:
            dq_in, oq = _out("dq_in", dq_in, dtype, index, tokens, dim, hdq.heads)
        if dk is not None:
            dk_in, ok = _out("dk_in", dk_in, dtype, index, tokens, dim, hdk.heads)
        if q_weight is not None:
            dqw = _empty((dim,), (1,), dtype=torch.float32, device=index)
        if k_weight is not None:
            dkw = _empty((dim,), (1,), dtype=torch.float32, device=index)
        if dqw is not None or dkw is not None:
            need = LIB.littlebit_rope_bwd_workspace_bytes(tokens, hdq.heads if hdq else 0, hdk.heads if hdk else 0, dim)
            ws = _empty((need,), (1,), dtype=torch.uint8, device=index)
        _check(LIB.littlebit_rope_bwd(
            hdq and _ref(hdq), hdk and _ref(hdk), hq and _ref(hq), hk and _ref(hk), _ref(rope), code, tokens, dim,
            oq and _ref(oq), ok and _ref(ok), None if dqw is None else dqw.data_ptr(),
            None if dkw is None else dkw.data_ptr(), ws.data_ptr() if need else None, need, sp))
    if stream is not None:
        _keep(stream, dq, dk, q, k, positions, inv_freq, q_weight, k_weight, dq_in, dk_in)
    return dq_in, dk_in, dqw, dkw


# ---------------------------------------------------------------------------------------------------- the cache

def _used(shape, strides):
    """Strides with those of dimensions of size one, which no address uses, as in a contiguous tensor."""
    out, inner = list(strides), 1
    for i in range(len(shape) - 1, -1, -1):
        if shape[i] == 1:
            out[i] = inner
        inner = max(inner, out[i] * shape[i])
    return tuple(out)


@dataclass
class LittleBitCache:
    """Pages of keys and of values, pages x heads x slots x dim each (fp16 or
    bf16).  Views with other strides work where the two agree and channels lie
    together, such as pages x slots x heads x dim, transposed."""
    k: torch.Tensor
    v: torch.Tensor

    @staticmethod
    def empty(pages: int, heads: int, dim: int, page_size: int = 64, dtype=torch.float16, device="cuda") -> "LittleBitCache":
        new = lambda: torch.empty(pages, heads, page_size, dim, dtype=dtype, device=device)  # noqa: E731
        return LittleBitCache(new(), new())

    def c_struct(self) -> _Cache:
        k, v = self.k, self.v
        code = _HALF.get(k.dtype) if torch.is_tensor(k) else None
        if code is None or not torch.is_tensor(v) or k.dim() != 4 or k.get_device() < 0:
            raise ValueError("a cache is two pages x heads x slots x dim CUDA tensors of float16 or bfloat16")
        if v.dtype is not k.dtype or v.get_device() != k.get_device() or v.shape != k.shape:
            raise ValueError("the cache's values must have the keys' type, device and shape")
        strides, others = k.stride(), v.stride()
        if strides != others or 1 in k.shape:
            strides, others = _used(k.shape, strides), _used(k.shape, others)
            if strides != others:
                raise ValueError("the cache's values must have the keys' strides")
        if strides[3] != 1:
            raise ValueError("the cache's channels must lie together")
        return _Cache(k.data_ptr(), v.data_ptr(), *strides[:3], *k.shape, code)


@dataclass
class CacheBatch:
    """The sequences of a call, int32 tensors on the cache's device: sequence i has
    the rows starts[i] to starts[i + 1] - 1, lens[i] keys in the cache (its rows'
    included, which are its last), and its pages in table[i].  Rows before
    starts[0] and from starts[-1] on belong to no sequence: every call leaves
    them as they are (in a new output: unset)."""
    starts: torch.Tensor
    lens: torch.Tensor
    table: torch.Tensor

    def c_struct(self, index: int) -> _Batch:
        starts, lens, table = self.starts, self.lens, self.table
        if torch.is_tensor(lens) and torch.is_tensor(table) and lens.dim() == 1 and table.dim() == 2:
            seqs, columns = table.shape
            stride, one = table.stride()
            if table.dtype is torch.int32 and table.get_device() == index and (one == 1 or columns == 1):
                return _Batch(_ints("starts", starts, index, seqs + 1), _ints("lens", lens, index, seqs), table.data_ptr(),
                              stride if seqs > 1 else columns, seqs, columns)
        raise ValueError(f"lens must be a 1-D and table a 2-D torch.int32 tensor on cuda:{index}, entries of a row together")


def littlebit_cache_append(cache: LittleBitCache, batch: CacheBatch, k: torch.Tensor, v: torch.Tensor,
                           q: Optional[torch.Tensor] = None, positions: Optional[torch.Tensor] = None,
                           inv_freq: Optional[torch.Tensor] = None, q_weight: Optional[torch.Tensor] = None,
                           k_weight: Optional[torch.Tensor] = None, eps: float = 1e-5, interleaved: bool = False,
                           q_out: Optional[torch.Tensor] = None, stream=None) -> Optional[torch.Tensor]:
    """Writes the keys (normed and turned as by littlebit_rope_fwd) and values of
    the batch's rows into its pages; returns the queries, normed and turned (None
    without q).  ``q_out`` may name that output, q itself included."""
    c = cache.c_struct()
    dtype, index, dim = cache.k.dtype, cache.k.get_device(), c.dim
    b = batch.c_struct(index)
    _first("k", k)
    tokens = k.shape[0]
    hk = _heads("k", k, dtype, index, tokens, dim, c.heads)
    hv = _heads("v", v, dtype, index, tokens, dim, c.heads)
    hq = None if q is None else _heads("q", q, dtype, index, tokens, dim)
    if q is None and (q_out is not None or q_weight is not None):
        raise ValueError("q_out and q_weight need q")
    rope = _rope(positions, inv_freq, q_weight, k_weight, eps, interleaved, dtype, index, tokens, dim)
    if _recording():
        _no_history(cache.k, cache.v, k, v, q, inv_freq, q_weight, k_weight, q_out)
    ctx, sp = _on(index, stream)
    with ctx:
        oq = None
        if q is not None:
            q_out, oq = _out("q_out", q_out, dtype, index, tokens, dim, hq.heads)
        _check(LIB.littlebit_cache_append(_ref(c), _ref(b), tokens, _ref(hk), _ref(hv), hq and _ref(hq), _ref(rope),
                                          oq and _ref(oq), sp))
    if stream is not None:
        _keep(stream, cache.k, cache.v, batch.starts, batch.lens, batch.table, k, v, q, positions, inv_freq, q_weight,
              k_weight, q_out)
    return q_out


def littlebit_cache_attention_fwd(q: torch.Tensor, cache: LittleBitCache, batch: CacheBatch,
                                  tree: Optional[torch.Tensor] = None, scale: Optional[float] = None,
                                  out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                                  stream=None) -> torch.Tensor:
    """The attention of q's rows over their sequences' keys in the cache, those of
    the rows themselves included (append first): causal, or, with ``tree`` (int64,
    one word a row), row t of a sequence sees the sequence's row j where bit j of
    its word is set, and all keys before the rows.  ``scale`` is 1 / sqrt(dim) by
    default.  ``lse`` (fp32, tokens x heads) receives the logarithm of each row's
    sum of exponentials."""
    c = cache.c_struct()
    dtype, index, dim = cache.k.dtype, cache.k.get_device(), c.dim
    b = batch.c_struct(index)
    _first("q", q)
    tokens, heads = q.shape[0], q.shape[1]
    hq = _heads("q", q, dtype, index, tokens, dim)
    word = None if tree is None else _ints("tree", tree, index, tokens, torch.int64)
    if lse is not None and (not torch.is_tensor(lse) or lse.dtype is not torch.float32 or lse.get_device() != index
                            or lse.shape != (tokens, heads) or not lse.is_contiguous()):
        raise ValueError(f"lse must be a contiguous torch.float32 tensor of shape {(tokens, heads)} on cuda:{index}")
    if _recording():
        _no_history(cache.k, cache.v, q, out, lse)
    ctx, sp = _on(index, stream)
    with ctx:
        out, ho = _out("out", out, dtype, index, tokens, dim, heads)
        need = LIB.littlebit_cache_attention_workspace_bytes(_ref(c), _ref(b), tokens, heads)
        ws = _empty((need,), (1,), dtype=torch.uint8, device=index)
        _check(LIB.littlebit_cache_attention_fwd(
            _ref(c), _ref(b), tokens, _ref(hq), word, 1.0 / math.sqrt(dim) if scale is None else scale, _ref(ho),
            None if lse is None else lse.data_ptr(), ws.data_ptr() if need else None, need, sp))
    if stream is not None:
        _keep(stream, cache.k, cache.v, batch.starts, batch.lens, batch.table, q, tree, out, lse)
    return out


def littlebit_cache_accept(cache: LittleBitCache, batch: CacheBatch, path: torch.Tensor, stream=None) -> None:
    """Of each sequence of the batch (that of the call which appended the tree),
    keys and values of row path[i][j] to the place of row j; negative entries end
    or skip.  path is int32, one row a sequence."""
    c = cache.c_struct()
    index = cache.k.get_device()
    b = batch.c_struct(index)
    if not torch.is_tensor(path) or path.dtype is not torch.int32 or path.get_device() != index or path.dim() != 2 \
            or path.shape[0] != b.seqs or not path.is_contiguous():
        raise ValueError(f"path must be a contiguous torch.int32 tensor of {b.seqs} rows on cuda:{index}")
    if _recording():
        _no_history(cache.k, cache.v)
    ctx, sp = _on(index, stream)
    with ctx:
        _check(LIB.littlebit_cache_accept(_ref(c), _ref(b), path.data_ptr(), path.shape[1], sp))
    if stream is not None:
        _keep(stream, cache.k, cache.v, batch.starts, batch.lens, batch.table, path)


# -------------------------------------------------------------------------------------------------- a block's part

@dataclass
class LittleBitAttention:
    """The attention of a block whose four projections are LittleBit layers:
    from the normed hidden states to the output projection's result."""
    q: LittleBitLayer
    k: LittleBitLayer
    v: LittleBitLayer
    o: LittleBitLayer
    dim: int                               # channels of a head
    inv_freq: Optional[torch.Tensor]       # fp32, half the rotated channels
    q_norm: Optional[torch.Tensor] = None  # fp16 weights of the head norms
    k_norm: Optional[torch.Tensor] = None
    eps: float = 1e-5
    interleaved: bool = False
    scale: Optional[float] = None

    def __call__(self, x: torch.Tensor, cache: LittleBitCache, batch: CacheBatch, positions: Optional[torch.Tensor] = None,
                 tree: Optional[torch.Tensor] = None) -> torch.Tensor:
        """x (tokens x n, fp16) of the batch's rows -> tokens x o.m.  Appends the
        rows' keys and values to the cache.  positions (int32) is what inv_freq needs."""
        rows = lambda layer: littlebit_linear_fwd(layer, x).view(x.shape[0], layer.m // self.dim, self.dim)  # noqa: E731
        with torch.cuda.device_of(x):   # the layers run on the current device
            q, k, v = rows(self.q), rows(self.k), rows(self.v)
            q = littlebit_cache_append(cache, batch, k, v, q, positions, self.inv_freq, self.q_norm, self.k_norm, self.eps,
                                       self.interleaved, q_out=q)
            out = torch.zeros_like(q)   # rows of no sequence stay 0
            littlebit_cache_attention_fwd(q, cache, batch, tree, self.scale, out=out)
            return littlebit_linear_fwd(self.o, out.view(x.shape[0], -1))
