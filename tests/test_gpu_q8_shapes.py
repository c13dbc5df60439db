"""Every tile shape of the 8-bit product (csrc/q8.hip), at every place where its
ring of LDS stages and of register buffers turns over.

Which shape a size takes is read off the kernel's own table, so that a change of
the table that leaves a shape without a case here fails."""

import os
import re

import numpy as np
import pytest
import torch

from oracle import head as oh

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
U = 2.0 ** -24
TYPES = {torch.float32: 2.0 ** -150, torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134}  # half the smallest subnormal

# (channels, tokens) of a tile: a (tokens, channels) size that takes it
SIZES = {(32, 64): (50, 70), (64, 64): (20, 9000), (64, 128): (130, 6000), (128, 64): (40, 20000),
         (128, 128): (130, 11000), (128, 256): (500, 11000), (256, 256): (1000, 16300)}


def shapes():
    """[(channels, tokens, cost)] and the LDS stages of each, as the source has them."""
    text = open(os.path.join(ROOT, "binary_rank_gemv_amd", "csrc", "q8.hip")).read()
    table = re.search(r"\bshapes\[\] = \{(.*?)\};", text, re.S).group(1)
    rows = [tuple(map(int, r)) for r in re.findall(r"\{(\d+), (\d+), (\d+)\}", table)]
    calls = [tuple(map(int, c)) for c in
             re.findall(r"launch_tile<Y, (\d+), (\d+), (\d+), (\d+), (\d+)>\(a, stream\)", text)]
    assert [(16 * wm * mw, 16 * wn * nw) for wm, wn, mw, nw, _ in calls] == [r[:2] for r in rows]
    return rows, {r[:2]: c[4] for r, c in zip(rows, calls)}


def chosen(rows, batch, m, compute_units):
    def cost(r):
        workgroups = -(-m // r[0]) * -(-batch // r[1])
        return -(-workgroups // compute_units) * r[2]
    return min(rows, key=cost)[:2]


def test_every_shape_has_a_size():
    rows, stages = shapes()
    assert set(SIZES) == {r[:2] for r in rows} == set(stages)
    for shape, (batch, m) in SIZES.items():
        assert batch > 16 and chosen(rows, batch, m, 256) == shape


@pytest.mark.gpu
@pytest.mark.parametrize("pad,offset", [(0, 0), (3, 1)])
@pytest.mark.parametrize("shape", list(SIZES), ids=lambda s: f"{s[0]}x{s[1]}")
def test_products_of_a_shape(shape, pad, offset):
    from binary_rank_gemv_amd import head
    rows, stages = shapes()
    batch, m = SIZES[shape]
    assert chosen(rows, batch, m, torch.cuda.get_device_properties(0).multi_processor_count) == shape
    st = stages[shape]
    # chunks of 128 inputs: fewer than the stages, as many, one more, and every remainder of two whole turns
    chunks = sorted({1, st - 1, st, st + 1} | set(range(2 * st + 1, 4 * st + 2)))
    most = 128 * chunks[-1] + 80
    rng = np.random.default_rng(shape[0] + shape[1])
    codes = [torch.from_numpy(rng.integers(-128, 128, (r, most + pad), dtype=np.int8)) for r in (batch, m)]
    xs = torch.from_numpy(rng.uniform(0.01, 0.1, batch).astype(np.float32))
    ws = torch.from_numpy((rng.uniform(0.5, 1.5, m) / 1000).astype(np.float32))
    xq, wq = (c[:, offset:] for c in codes)
    xd, wd = (c.cuda()[:, offset:] for c in codes)
    sums = 0
    done = 0
    for c in chunks:
        for n in (128 * c, 128 * c + 77):
            print("[case]", shape, pad, batch, m, n, flush=True)
            # whole numbers below 2^53: the sums are exact, and a longer row's are a shorter one's and the rest
            rest = oh.q8_linear(xq[:, done:n].numpy(), np.ones(batch), wq[:, done:n].numpy(), np.ones(m))
            sums, done = sums + rest, n
            want = torch.from_numpy(sums * xs.double().numpy()[:, None] * ws.double().numpy()).cuda()
            for t in TYPES if n == chunks[-1] * 128 + 77 else (torch.float32,):
                got = head.littlebit_q8_linear_fwd(xd[:, :n], xs.cuda(), wd[:, :n], ws.cuda(), dtype=t)
                # the sum as fp32, the scales' product, their product, the output: half a step each
                tol = (3 * U + torch.finfo(t).eps / 2 * (1 + 4 * U)) * want.abs() + TYPES[t]
                assert ((got.double() - want).abs() <= tol).all()
