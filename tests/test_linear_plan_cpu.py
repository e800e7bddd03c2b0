"""The grouped products' rules that need no GPU (csrc/linear_plan.h), compiled here with the
host's C++ compiler."""
import ctypes as C
import os
import subprocess

import numpy as np
import pytest

from atomic_expert_routing_b200 import build as libbuild
from linear_cases import GRAD_W, GRAD_W_IDS, ROW_IDS, ROWS

SHIM = r"""
#include "linear_plan.h"
using namespace omni;
extern "C" {
// the zeroing warp's walk: tiles of blocks[i] blocks, waits where tail[i]; the limits of each wait
void wait_limits(int n, const int32_t* blocks, const uint8_t* tail, uint32_t* limits) {
  WaitSpan span;
  for (int i = 0; i < n; ++i) {
    span.tile(blocks[i]);
    limits[i] = 0;
    if (tail[i]) {
      limits[i] = span.limits();
      span.waited();
    }
  }
}
int shape(int64_t I, int64_t rows, int64_t G, int sms) { return pick_shape(I, rows, G, sms); }
int pairs(int64_t in, int64_t out, int64_t rows, int64_t G, int sms) {
  return grad_w_pairs(in, out, rows, G, sms);
}
}
"""


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    d = tmp_path_factory.mktemp("plan")
    src, so = d / "shim.cc", d / "shim.so"
    src.write_text(SHIM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-Wall", "-Werror", "-I",
                    libbuild.CSRC, "-o", str(so), str(src)], check=True)
    lib = C.CDLL(str(so))
    lib.shape.argtypes = [C.c_int64] * 3 + [C.c_int]
    lib.pairs.argtypes = [C.c_int64] * 4 + [C.c_int]
    return lib


# what a block of 64 rows and a tile's way out take at most, in seconds: a CTA's share of the
# memory's rate, 6.5 TB/s / 148, for 32 KB a block (0.75 us; the products alone take 0.4), and
# 128 KB of dW for a tile
BLOCK, WAY_OUT = 32768 / (6.5e12 / 148), 131072 / (5e12 / 148)


def _walk(rows, per_group, slots, slot):
    """A CTA's tiles: (blocks, has rows to zero) of every slots-th of the groups' tiles."""
    group = np.repeat(np.arange(len(rows)), per_group)[slot::slots]
    r = np.asarray(rows, dtype=np.int64)[group]
    return ((r + 63) // 64).astype(np.int32), ((r % 16 != 0) & (r > 0)).astype(np.uint8)


WALKS = {
    # the first group alone takes a CTA past the limit of one second
    "a long group, then ten rows": ([1 << 29] + [16] * 147 + [10], 1, 148),
    "two wide experts": ([499_968, 500_010], 256 * 256, 74),
    "no group but the last": ([65_536] * 1023 + [1], 16, 148),
    "every group": ([1 + 37 * q % 83 for q in range(1000)], 16, 74),
    "empty groups": ([0] * 1000 + [5], 4096, 74),
    "one group": ([(1 << 30) - 1], 1, 148),
}


@pytest.mark.parametrize("name", list(WALKS))
def test_a_wait_for_rows_to_zero_outlasts_what_the_cta_sums_before(plan, name):
    rows, per_group, slots = WALKS[name]
    waits = 0
    for slot in range(slots):
        blocks, tail = _walk(rows, per_group, slots, slot)
        limits = np.zeros(len(blocks), dtype=np.uint32)
        plan.wait_limits(len(blocks), blocks.ctypes.data_as(C.c_void_p),
                         tail.ctypes.data_as(C.c_void_p), limits.ctypes.data_as(C.c_void_p))
        since = np.cumsum(blocks * BLOCK + WAY_OUT)
        at = np.nonzero(tail)[0]
        lasts = np.diff(since[at], prepend=0.0) if len(at) else since[:0]
        assert (limits[at] > 2 * lasts).all()
        # and stays near it, so that a wait that nothing ends is given up
        assert (limits[at] <= 2 + 10 * lasts).all()
        waits += len(at)
    assert waits


# ---- which kernel a product takes -----------------------------------------------------

SMS, WIDTHS = 148, (32, 64, 128, 256)


@pytest.mark.parametrize("width,several,sizes,I,K", ROWS, ids=ROW_IDS)
def test_rows_cases_reach_their_kernel(plan, width, several, sizes, I, K):
    assert WIDTHS[plan.shape(I, sum(sizes), len(sizes), SMS)] == width
    pair = 2 if width == 256 else 1
    tiles = sum(-(-r // width) for r in sizes) * -(-I // (128 * pair))
    assert (tiles > SMS // pair) == several
    assert any(r % 32 for r in sizes) and K % 64  # ends inside a tile and inside a k-block


@pytest.mark.parametrize("pairs,several,sizes,n_in,n_out", GRAD_W, ids=GRAD_W_IDS)
def test_grad_w_cases_reach_their_kernel(plan, pairs, several, sizes, n_in, n_out):
    assert bool(plan.pairs(n_in, n_out, sum(sizes), len(sizes), SMS)) == pairs
    m = 256 if pairs else 128
    tiles = -(-n_in // m) * -(-n_out // m) * len(sizes)
    assert (tiles > SMS // (2 if pairs else 1)) == several
    assert any(r % 16 for r in sizes)  # with rows to zero


def test_every_kernel_has_cases():
    assert {w for w, *_ in ROWS} == set(WIDTHS) and {p for p, *_ in GRAD_W} == {False, True}
    for w in WIDTHS:
        assert {s for v, s, *_ in ROWS if v == w} == {False, True}
    for p in (False, True):
        assert {s for v, s, *_ in GRAD_W if v == p} == {False, True}
    assert any(k > 512 for *_, k in ROWS)
