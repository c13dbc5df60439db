"""The attention's split of a batch against its plan, on the CPU: every block of
rows and part of keys that the kernels number has a workgroup, and every part
that is joined a place in the workspace.  The split is computed by the kernels'
own arithmetic (csrc/attn_split.h), compiled for the host."""

import ctypes
import os
import random
import subprocess

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def split(tmp_path_factory):
    from binary_rank_gemv_amd import build
    if not os.path.exists(build.ATTN_LIB):
        pytest.skip("library not built (python -m binary_rank_gemv_amd.build)")
    out = str(tmp_path_factory.mktemp("split") / "libsplit.so")
    subprocess.run([build.HIPCC, "--offload-host-only", "-x", "hip", "-O1", "-std=c++17", "-fPIC", "-shared",
                    "-I", os.path.join(ROOT, "include"), "-I", build.CSRC, os.path.join(ROOT, "tests", "attn_split_host.hip"),
                    "-L", build.LIBDIR, "-l:" + os.path.basename(build.ATTN_LIB), "-Wl,-rpath," + build.LIBDIR, "-o", out],
                   check=True, capture_output=True, timeout=300)
    lib = ctypes.CDLL(out)

    def call(counts, heads, kv, dim, page=64, spare=0):
        """(items, joined, workgroups, slots, height) of sequences of (rows, keys)."""
        rows, keys = (np.array([c[i] for c in counts], dtype=np.int32) for i in (0, 1))
        columns = max(1, -(-int(keys.max()) // page))
        result = np.zeros(5, dtype=np.int64)
        as_p = lambda a: ctypes.c_void_p(a.ctypes.data)  # noqa: E731
        lib.attn_split(ctypes.c_int64(int(rows.sum()) + spare), len(counts), ctypes.c_int64(columns * page), heads, kv, dim, as_p(rows), as_p(keys),
                       as_p(result))
        return [int(v) for v in result]
    return call


def hold(got, *what):
    items, joined, workgroups, slots, height = got
    assert items <= workgroups, (what, got)
    assert joined <= slots, (what, got)


@pytest.mark.parametrize("counts,heads,kv,dim", [
    ([(5600, 9000)] + [(1, 1000)] * 69, 4, 1, 64), ([(7839, 7839)] + [(1, 1)] * 71, 3, 1, 64),
    ([(10943, 10943)] + [(1, 1)] * 69, 2, 1, 64), ([(20000, 20000)] + [(1, 1)] * 69, 1, 1, 64),
    ([(20000, 20000)] + [(10, 10)] * 64, 1, 1, 64), ([(16128, 16128)] + [(1, 1)] * 64, 1, 1, 128),
    ([(8192, 8192)] + [(0, 0)] * 64, 4, 1, 128), ([(8064, 8064)] + [(0, 0)] * 64, 4, 2, 64),
    ([(9000, 9000)] + [(1, 70)] * 140, 2, 1, 64), ([(6000, 6100)] + [(3, 40)] * 200, 4, 1, 256),
    # rows whose keys were never counted
    ([(9000, 9000)] + [(100, 0)] * 70, 1, 1, 64)])
def test_long_prompts_among_many_sequences(split, counts, heads, kv, dim):
    for order in (counts, counts[::-1]):
        got = split(order, heads, kv, dim)
        assert got[4] > 32   # blocks of many rows
        hold(got, heads, kv, dim)


@pytest.mark.parametrize("seed", range(8))
def test_random_batches(split, seed):
    """1 to 300 sequences: alike, one long among short ones, of all lengths, empty ones, keys that are fewer than the rows."""
    rng = random.Random(seed)
    spread = lambda low, high: int(round(low * (high / low) ** rng.random()))  # noqa: E731
    many = several = 0
    for _ in range(400):
        kv = rng.choice([1, 1, 1, 2, 2, 4, 8, 40])
        heads, dim, page = kv * rng.choice([1, 1, 2, 3, 4, 6, 8]), rng.choice([8, 64, 80, 96, 128, 192, 256]), rng.choice([8, 16, 64, 1024])
        seqs = rng.choice([1, 2, 63, 64, 65, 66, 128, 129, spread(1, 300)])
        kind = rng.choice(["long", "long", "alike", "any", "one"])
        counts = []
        for i in range(seqs):
            rows = {"long": rng.randint(0, 2), "alike": 300, "any": rng.choice([0, 1, spread(1, 3000)]), "one": 1}[kind]
            counts.append((rows, rows + rng.choice([0, 0, spread(1, 4000)])))
        if kind == "long":
            rows = spread(100, 30000)
            counts[rng.randrange(seqs)] = (rows, rows + rng.choice([0, 0, spread(1, 30000)]))
        if rng.random() < 0.1:
            counts = [(r, rng.randint(0, n)) for r, n in counts]
        if sum(r for r, _ in counts) == 0:
            counts[0] = (1, 1)
        got = split(counts, heads, kv, dim, page, spare=rng.choice([0, 0, 5]))
        hold(got, counts[:3], seqs, heads, kv, dim, page)
        many += got[4] > 32 and seqs > 64
        several += got[1] > 0
    assert many > 20 and several > 20   # the draw reaches what it is for
