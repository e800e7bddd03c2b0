"""The draining warps of the grouped products when a wait runs out.  Four warps share barriers
that have no time limit, and each decides by itself that its wait has run out: the phase can end
between two warps' last looks.  A warp that then left would leave the others in a barrier for
good.  A model of the protocol, and a look at the source that it is the one the kernel keeps."""
import ctypes as C
import itertools
import os
import re
import subprocess

import pytest

from atomic_expert_routing_b200 import build as libbuild


def _warp(tiles, runs_out, keeps_on):
    """A warp's walk: per tile one wait, then that tile's barriers.  runs_out: the waits that this
    warp, if it still waits then, gives up."""
    ok = True
    for t, barriers in enumerate(tiles):
        if ok and t in runs_out:
            ok = False
            if not keeps_on:
                return
        for _ in range(barriers):
            yield


def _all_end(tiles, outs, keeps_on):
    """Four warps with a barrier of all four: whether every warp reaches its end."""
    warps = [_warp(tiles, o, keeps_on) for o in outs]
    while True:
        at_barrier = [next(w, "end") != "end" for w in warps]
        if not any(at_barrier):
            return True
        if not all(at_barrier):
            return False  # some wait for warps that have gone


# barriers of a tile: two for each chunk that leaves through shared memory; none where the group's
# end cuts it or the columns lie past the matrix
TILES = [[2], [0, 2], [2, 0, 4], [4, 4, 2, 0], [0, 0, 0]]


@pytest.mark.parametrize("tiles", TILES, ids=str)
def test_every_warp_ends_whichever_waits_run_out(tiles):
    some = [set(c) for r in range(3) for c in itertools.combinations(range(len(tiles)), r)]
    stuck = 0
    for outs in itertools.product(some, repeat=4):
        assert _all_end(tiles, outs, keeps_on=True)
        stuck += not _all_end(tiles, outs, keeps_on=False)
    assert (stuck > 0) == any(tiles)  # and leaving at a time-out would not have been enough


SHIM = r"""
#include "linear_plan.h"
extern "C" {
int whole(int clipped, int left) { return omni::DrainRule{clipped != 0, false, 16}.whole(left); }
int two(int pairs, int gap, int left) { return omni::DrainRule{false, pairs != 0, gap}.two(left); }
int barriers(int clipped, int pairs, int gap, int n, int c) {
  return omni::DrainRule{clipped != 0, pairs != 0, gap}.barriers(n, c);
}
}
"""


def test_the_barriers_of_a_tile_are_counted_as_its_chunks_take_them(tmp_path):
    src, so = tmp_path / "shim.cc", tmp_path / "shim.so"
    src.write_text(SHIM)
    subprocess.run(["g++", "-std=c++17", "-shared", "-fPIC", "-Wall", "-Werror", "-I",
                    libbuild.CSRC, "-o", str(so), str(src)], check=True)
    lib = C.CDLL(str(so))

    def walk(clipped, pairs, gap, n, c):
        """The barriers one after another: the kernel's two ways out, two of its chunks a time."""
        taken = 0
        while c < n:
            both = c + gap < n
            if both and lib.two(pairs, gap, n - c):
                taken += 2
            else:
                for at in (c, c + gap) if both else (c,):
                    taken += 2 if lib.whole(clipped, n - at) else 0
            c += 2 * gap
        return taken

    for clipped, pairs, gap, n in itertools.product((0, 1), (0, 1), (16, 32), range(1, 257)):
        for c in (0,) if gap == 16 else (0, 16):
            assert lib.barriers(clipped, pairs, gap, n, c) == walk(clipped, pairs, gap, n, c)


def test_the_kernel_comes_to_every_barrier():
    text = open(os.path.join(libbuild.CSRC, "linear_tc.cu")).read()
    a = text.index("if (warp < kEpiWarps) {")
    part = re.sub(r"//[^\n]*", "", text[a:text.index("// this thread's stores are done", a)])
    walk, rest = part.split("if (!ok)\n      for (; t < tiles; t += step) {")
    # the walk over the tiles: left early only where a wait ran out, before the tile's barriers
    assert "for (; t < tiles; t += step) {" in walk and walk.count("half_sync(half)") == 4
    assert re.findall(r"[^;{}]*break;", walk) and all(
        re.search(r"if \(!ok\) break;", b) for b in re.findall(r"[^;{}]*break;", walk))
    assert walk.rindex("if (!ok) break;") < walk.index("leave_two(c, z0, z1)")
    assert [r for r in re.findall(r"[^;{}]*\breturn;", walk)] == ["\n        if (ic >= I) return;"]
    # then the barriers of the tiles that are left
    assert "walk.at(t)" in rest and "rule.barriers(tl.n, first_c)" in rest
    assert rest.count("half_sync(half)") == 1 and "break" not in rest and "return" not in rest


def test_dw_beside_dx_reads_no_array_through_l1():
    """dW may start without a wait of its own: group arrays and row numbers come from L2."""
    text = open(os.path.join(libbuild.CSRC, "linear.cuh")).read()
    table = text[text.index("void build_groups("):]
    table = table[:table.index("// What the products of one launch read and write")]
    assert "__ldcg" in text
    for array in ("off", "ids", "n_groups"):
        reads = re.findall(rf"\*\s*P\.{array}\b|P\.{array}\[", table)
        assert not reads and f"fresh(P.{array}" in table
    text = open(os.path.join(libbuild.CSRC, "linear_tc.cu")).read()
    grad = text[text.index("if constexpr (C::kGradW) {\n        uint32_t tails"):]
    grad = grad[:grad.index("} else if (gathers) {")]
    assert "a.rows[" not in grad and grad.count("fresh(a.rows") == 2
