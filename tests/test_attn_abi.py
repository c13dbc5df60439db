"""The C ABI between the projections: exported symbols, refusals before anything
is launched, sizes.  Every call here fails validation on the host or has
nothing to do; no GPU is needed."""

import ctypes
import os
import re
import subprocess

import pytest
import torch

attn = pytest.importorskip("binary_rank_gemv_amd.attn",
                           reason="liblittlebit_attn.so not built (run python -m binary_rank_gemv_amd.build)")
from binary_rank_gemv_amd import littlebit as lb  # noqa: E402

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "littlebit_attn.h")
FAKE = 1 << 20   # non-null, aligned, never dereferenced
BAD, UNSUP, WS = lb.LB_ERR_INVALID_ARG, lb.LB_ERR_UNSUPPORTED, lb.LB_ERR_WORKSPACE
F32, F16, BF16 = lb.LB_F32, lb.LB_F16, attn.LB_BF16
ref = ctypes.byref


def test_every_declared_symbol_is_exported_and_bound():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"\b(littlebit_\w+)\s*\(", text))
    assert names == set(attn.ATTN_EXPORTED)
    lib = ctypes.CDLL(attn.ATTN_LIB_PATH)
    for n in names:
        assert hasattr(lib, n), n
    for line in open(HEADER):
        m = re.match(r"#define (LB_\w+) (\d+)$", line)
        if m:
            assert getattr(attn, m.group(1)) == int(m.group(2))


def test_library_needs_no_vendor_kernels():
    deps = subprocess.run(["readelf", "-d", attn.ATTN_LIB_PATH], capture_output=True, text=True).stdout
    needed = re.findall(r"\(NEEDED\).*\[(.*)\]", deps)
    assert needed and not any(k in d for d in needed for k in ("blas", "solver", "MIOpen"))


def H(p=FAKE, token=256, head=64, heads=4):
    return attn._Heads(p, token, head, heads)


def rope(positions=FAKE, inv=FAKE, rot=64, inter=0, qw=FAKE, kw=FAKE, eps=1e-5):
    return attn._Rope(positions, inv, rot, inter, qw, kw, eps)


def r(x):
    return None if x is None else ref(x)


OUT = 2 * FAKE


def _fwd(q=H(), k=H(), rp=rope(), dtype=F16, tokens=3, dim=64, qo=H(OUT), ko=H(OUT)):
    return attn.LIB.littlebit_rope_fwd(r(q), r(k), r(rp), dtype, tokens, dim, r(qo), r(ko), None)


HEADS = [
    (dict(q=H(None)), BAD), (dict(q=H(FAKE + 1)), BAD), (dict(q=H(token=-1)), BAD), (dict(q=H(head=-64)), BAD),
    (dict(q=H(token=1 << 50)), UNSUP), (dict(q=H(heads=0), qo=H(OUT, heads=0)), BAD), (dict(q=H(heads=2000)), UNSUP),
    (dict(qo=H(OUT, heads=3)), BAD), (dict(qo=H(FAKE, token=512)), BAD), (dict(qo=H(OUT, token=200)), BAD),
    (dict(qo=H(OUT, head=32)), BAD), (dict(qo=H(OUT, token=64, head=128)), BAD), (dict(q=None), BAD), (dict(qo=None), BAD),
]


@pytest.mark.parametrize("kw,status", HEADS + [
    (dict(dtype=F32), BAD), (dict(dtype=9), BAD), (dict(tokens=-1), BAD), (dict(tokens=1 << 22), UNSUP), (dict(dim=0), BAD),
    (dict(dim=63), BAD), (dict(dim=258), UNSUP), (dict(rp=None), BAD), (dict(rp=rope(rot=63)), BAD), (dict(rp=rope(rot=66)), BAD),
    (dict(rp=rope(rot=-2)), BAD), (dict(rp=rope(eps=-1.0)), BAD), (dict(rp=rope(eps=float("nan"))), BAD),
    (dict(rp=rope(eps=float("inf"))), BAD), (dict(rp=rope(positions=None)), BAD), (dict(rp=rope(inv=None)), BAD),
    (dict(rp=rope(positions=FAKE + 2)), BAD), (dict(rp=rope(inv=FAKE + 2)), BAD), (dict(rp=rope(qw=FAKE + 1)), BAD),
    (dict(q=None, k=None, qo=None, ko=None), BAD), (dict(k=None), BAD), (dict(ko=None), BAD),
])
def test_rope_refuses(kw, status):
    assert _fwd(**kw) == status
    assert "littlebit_rope_fwd" in attn.littlebit_attn_last_error()


def _bwd(dq=H(), dk=H(), q=H(), k=H(), rp=rope(), dtype=BF16, tokens=3, dim=64, qo=H(OUT), ko=H(OUT), qw=FAKE, kw=FAKE, ws=FAKE,
         nws=1 << 20):
    return attn.LIB.littlebit_rope_bwd(r(dq), r(dk), r(q), r(k), r(rp), dtype, tokens, dim, r(qo), r(ko), qw, kw, ws, nws, None)


@pytest.mark.parametrize("kw,status", [
    (dict(dq=H(None)), BAD), (dict(q=None), BAD), (dict(k=None), BAD), (dict(q=H(heads=3)), BAD), (dict(qo=None), BAD),
    (dict(qw=None), BAD), (dict(kw=None), BAD), (dict(qw=FAKE + 2), BAD), (dict(rp=rope(qw=None)), BAD), (dict(ws=None), WS),
    (dict(ws=FAKE + 8), WS), (dict(nws=16), WS), (dict(dq=None), BAD), (dict(dq=None, qo=None), BAD), (dict(dtype=F32), BAD),
    (dict(q=H(OUT, token=512)), BAD), (dict(dq=None, dk=None), BAD), (dict(tokens=-1), BAD), (dict(dim=7), BAD),
    (dict(rp=None), BAD),
])
def test_rope_backward_refuses(kw, status):
    assert _bwd(**kw) == status
    assert "littlebit_rope_bwd" in attn.littlebit_attn_last_error()


def C(k=FAKE, v=FAKE, page=2 * 16 * 64, head=16 * 64, slot=64, pages=9, heads=2, size=16, dim=64, dtype=F16):
    return attn._Cache(k, v, page, head, slot, pages, heads, size, dim, dtype)


def B(starts=FAKE, lens=FAKE, table=FAKE, stride=4, seqs=2, columns=4):
    return attn._Batch(starts, lens, table, stride, seqs, columns)


CACHES = [
    (dict(c=None), BAD), (dict(c=C(k=None)), BAD), (dict(c=C(v=FAKE + 8)), BAD), (dict(c=C(page=2 * 16 * 64 + 4)), BAD),
    (dict(c=C(head=1000)), BAD), (dict(c=C(head=8)), BAD), (dict(c=C(slot=56)), BAD), (dict(c=C(slot=1 << 25)), UNSUP),
    (dict(c=C(pages=0)), BAD), (dict(c=C(heads=0)), BAD), (dict(c=C(heads=2000)), UNSUP), (dict(c=C(size=4)), BAD),
    (dict(c=C(size=24)), BAD), (dict(c=C(size=1 << 17)), BAD), (dict(c=C(dim=60)), BAD), (dict(c=C(dim=264)), UNSUP),
    (dict(c=C(dtype=F32)), BAD), (dict(c=C(page=0)), BAD), (dict(c=C(page=-2048)), BAD), (dict(b=None), BAD), (dict(b=B(starts=None)), BAD), (dict(b=B(lens=FAKE + 2)), BAD),
    (dict(b=B(table=None)), BAD), (dict(b=B(seqs=0)), BAD), (dict(b=B(seqs=1 << 16)), UNSUP), (dict(b=B(columns=0)), BAD),
    (dict(b=B(columns=1 << 26, stride=1 << 26)), UNSUP), (dict(b=B(stride=3)), BAD),
]
KV = H(heads=2, token=128)


def _append(c=C(), b=B(), tokens=3, k=KV, v=KV, q=H(), rp=rope(), qo=H(OUT)):
    return attn.LIB.littlebit_cache_append(r(c), r(b), tokens, r(k), r(v), r(q), r(rp), r(qo), None)


@pytest.mark.parametrize("kw,status", CACHES + [
    (dict(k=None), BAD), (dict(v=None), BAD), (dict(k=H()), BAD), (dict(v=H(None, heads=2)), BAD), (dict(q=None), BAD),
    (dict(qo=None), BAD), (dict(qo=H(OUT, token=100)), BAD), (dict(rp=rope(rot=66)), BAD), (dict(tokens=-1), BAD), (dict(tokens=1 << 22), UNSUP),
])
def test_append_refuses(kw, status):
    assert _append(**kw) == status
    assert "littlebit_cache_append" in attn.littlebit_attn_last_error()


LONG = B(columns=100, stride=100)   # more keys than one workgroup takes at least


def _attend(c=C(), b=B(), tokens=3, q=H(), tree=None, scale=0.1, out=H(OUT), lse=None, ws=FAKE, nws=1 << 30):
    return attn.LIB.littlebit_cache_attention_fwd(r(c), r(b), tokens, r(q), tree, scale, r(out), lse, ws, nws, None)


@pytest.mark.parametrize("kw,status", CACHES + HEADS[:7] + [
    (dict(out=H(OUT, heads=2)), BAD), (dict(out=H()), BAD), (dict(out=None), BAD), (dict(q=H(heads=3), out=H(OUT, heads=3)), BAD),
    (dict(scale=float("nan")), BAD), (dict(tree=FAKE + 4), BAD), (dict(lse=FAKE + 2), BAD),
    (dict(b=LONG, ws=None), WS), (dict(b=LONG, ws=FAKE + 8), WS), (dict(b=LONG, nws=100), WS), (dict(tokens=-1), BAD),
    (dict(c=C(heads=512, head=1024, page=512 * 1024), q=H(heads=1024, token=1 << 16), out=H(OUT, heads=1024, token=1 << 16), tokens=1 << 21), UNSUP),
])
def test_attention_refuses(kw, status):
    kw = {("out" if k == "qo" else k): v for k, v in kw.items()}
    assert _attend(**kw) == status
    assert "littlebit_cache_attention_fwd" in attn.littlebit_attn_last_error()


def _accept(c=C(), b=B(), path=FAKE, columns=5):
    return attn.LIB.littlebit_cache_accept(r(c), r(b), path, columns, None)


@pytest.mark.parametrize("kw,status", CACHES + [
    (dict(path=None), BAD), (dict(path=FAKE + 2), BAD), (dict(columns=0), BAD), (dict(columns=65), BAD)])
def test_accept_refuses(kw, status):
    assert _accept(**kw) == status
    assert "littlebit_cache_accept" in attn.littlebit_attn_last_error()


def test_no_tokens_is_no_work():
    none, kv = H(None), H(None, heads=2)
    assert _fwd(q=none, k=none, qo=none, ko=none, tokens=0, rp=rope(None, None)) == lb.LB_OK
    assert _append(k=kv, v=kv, q=none, qo=none, tokens=0) == lb.LB_OK
    assert _attend(q=none, out=none, tokens=0, ws=None, nws=0) == lb.LB_OK
    assert _bwd(dq=none, dk=none, qo=none, ko=none, rp=rope(None, None, qw=None, kw=None), q=None, k=None, qw=None, kw=None, tokens=0, ws=None,
                nws=0) == lb.LB_OK


def test_workspace_sizes():
    W = attn.LIB.littlebit_rope_bwd_workspace_bytes
    assert W(0, 4, 4, 64) == 0 and W(1, 4, 4, 300) == 0 and W(-1, 4, 4, 64) == 0 and W(1, 5000, 1, 64) == 0
    assert 0 < W(1, 4, 4, 64) <= W(100, 4, 4, 64) and W(100, 0, 4, 64) > 0
    A = lambda c, b, t, h: attn.LIB.littlebit_cache_attention_workspace_bytes(r(c), r(b), t, h)  # noqa: E731
    assert A(C(), B(), 0, 4) == 0 and A(C(), B(), 3, 3) == 0 and A(None, B(), 3, 4) == 0 and A(C(), None, 3, 4) == 0
    assert A(C(heads=0), LONG, 3, 4) == 0 and A(C(), B(seqs=0), 3, 4) == 0 and A(C(), LONG, 3, 4) > 0
    assert A(C(), B(), 3, 4) == 0   # short sequences: nothing to join
    assert A(C(), B(seqs=1 << 16), 3, 4) == 0 and 0 < A(C(), B(seqs=200), 300, 4) <= A(C(), B(seqs=60000), 300, 4)   # many: places to add up


def test_binding_refuses_what_is_not_on_a_gpu():
    x, i = torch.zeros(2, 1, 64, dtype=torch.float16), torch.zeros(2, dtype=torch.int32)
    cache, batch = attn.LittleBitCache(*[torch.zeros(1, 1, 8, 64, dtype=torch.float16)] * 2), attn.CacheBatch(i, i[:1], i[None])
    for call in (lambda: attn.littlebit_rope_fwd(x, x), lambda: attn.littlebit_rope_bwd(x, x),
                 lambda: attn.littlebit_cache_append(cache, batch, x, x), lambda: attn.littlebit_cache_attention_fwd(x, cache, batch),
                 lambda: attn.littlebit_cache_accept(cache, batch, i[None])):
        with pytest.raises(ValueError):
            call()


def test_a_block_calls_its_layers_on_the_device_of_its_tensors(monkeypatch):
    """The layers run on the current device: the block makes that of x current, also where it is another."""
    inside, calls = [], []

    class Device:
        def __enter__(self):
            inside.append(True)

        def __exit__(self, *_):
            inside.pop()

    def layer(name, m):
        return type("Layer", (), {"name": name, "m": m})()

    def linear(layer, x):
        calls.append((layer.name, bool(inside)))
        return x.new_zeros(x.shape[0], layer.m)

    monkeypatch.setattr(torch.cuda, "device_of", lambda x: Device())
    monkeypatch.setattr(attn, "littlebit_linear_fwd", linear)
    monkeypatch.setattr(attn, "littlebit_cache_append", lambda cache, batch, k, v, q, *rest, q_out: q_out)
    monkeypatch.setattr(attn, "littlebit_cache_attention_fwd", lambda q, *rest, out: out)
    block = attn.LittleBitAttention(layer("q", 16), layer("k", 8), layer("v", 8), layer("o", 12), 8, None)
    assert block(torch.zeros(3, 12), None, None).shape == (3, 12)
    assert sorted(calls) == [("k", True), ("o", True), ("q", True), ("v", True)] and not inside
