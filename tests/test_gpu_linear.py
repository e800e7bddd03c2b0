"""GPU parity of the wide-expert products, their gradients and the 8-bit products against their
definitions in 64 bits.

Tolerances, element by element.  A sum of K products of bf16 values in fp32, in any order and with
every addition off by at most one unit in the last place (2^-23 relative to the partial sum,
which the sum of the magnitudes S bounds): K * 2^-23 * S.  Rounding the result v to bf16 adds
2^-8 * |v|, to fp32 2^-24 * |v|.  SiLU changes its argument's error by a factor of at most 1.1
and adds a few fp32 roundings (8 * 2^-24 * |v|).  Integer sums are exact; their conversion to
fp32 and the two scales add 3 * 2^-24 * |v|.
"""
import numpy as np
import pytest
import torch

import atomic_expert_routing_b200 as omni
from atomic_expert_routing_b200 import _lib

pytestmark = pytest.mark.gpu

ULP = 2.0 ** -23
BF, F32 = torch.bfloat16, torch.float32


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, *shape, std=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(BF)


def _i32(v):
    return torch.tensor(np.asarray(v, dtype=np.int32), device="cuda")


def _silu(v):
    return v * torch.sigmoid(v)


def _close(got, ref, err, silu=False):
    """|got - ref| <= the sum's error err (of ref before SiLU), carried on, plus the roundings."""
    v = _silu(ref) if silu else ref
    if silu:
        err = 1.1 * err + 8 * 2.0 ** -24 * v.abs()
    half = 2.0 ** -8 if got.dtype == BF else 2.0 ** -24
    tol = err + half * (v.abs() + err) + 1e-37
    off = (got.double() - v).abs()
    assert bool(torch.isfinite(got).all())
    assert bool((off <= tol).all()), float((off / tol).max())


# group sizes, in, out; the sizes hold groups without rows, of one row, ends inside a tile of
# any size and past several, and rows behind the last group (`more`)
SHAPES = [
    ([1], 8, 8, 0),
    ([0, 1, 0], 64, 64, 0),
    ([1] * 8, 2048, 1024, 0),
    ([0, 0, 0], 64, 72, 5),
    ([3, 0, 17, 1, 0, 130, 33], 200, 328, 9),
    ([257, 15, 16, 17, 31, 32, 33, 0], 72, 1000, 0),
    ([63, 64, 65, 127, 128, 129], 1000, 136, 1),
    ([700, 3], 512, 264, 2),
    ([2, 1300, 0, 255, 256], 520, 520, 0),
    ([5] * 70, 128, 256, 3),
    # several tiles to a CTA, most groups ending inside a block of 64 and of 16 rows
    ([1 + 37 * q % 83 for q in range(60)], 520, 1032, 0),
]
IDS = [f"{len(s[0])}x{sum(s[0])}-{s[1]}-{s[2]}" for s in SHAPES]


def _off(sizes):
    return np.concatenate(([0], np.cumsum(sizes)))


def _groups(sizes, listed, E_more=0, seed=0):
    """The group arrays of a call.  listed: only the groups with rows, their ids among more
    matrices, behind them entries that must not be used.  (kwargs, group_off, E, id of group)"""
    if not listed:
        return {}, _i32(_off(sizes)), len(sizes), np.arange(len(sizes))
    live = [s for s in sizes if s > 0]
    E = len(sizes) + 3
    ids = np.sort(np.random.default_rng(seed).choice(E, len(live), replace=False))
    pad = 2
    off = np.concatenate((_off(live), [7] * pad))
    kw = {"ids": _i32(np.concatenate((ids, [1 << 30] * pad))), "n_groups": _i32([len(live)])}
    return kw, _i32(off), E, ids


def _rows(g, M, T, on):
    return torch.randint(0, T, (M,), generator=g, device="cuda", dtype=torch.int32) if on else None


def _spans(sizes, ids, listed):
    sizes = [s for s in sizes if s > 0] if listed else sizes
    off = _off(sizes)
    return [(int(off[i]), int(off[i + 1]), int(ids[i])) for i in range(len(sizes))]


@pytest.mark.parametrize("f32", [False, True], ids=["bf16", "f32"])
@pytest.mark.parametrize("listed,gather,silu", [(False, False, False), (True, True, False),
                                                (True, False, True), (False, True, True)])
@pytest.mark.parametrize("sizes,n_in,n_out,more", SHAPES, ids=IDS)
def test_forward(sizes, n_in, n_out, more, listed, gather, silu, f32):
    g = _gen(1)
    kw, off, E, ids = _groups(sizes, listed)
    M = sum(sizes) + more
    T = max(1, M // 3) if gather else M
    rows = _rows(g, M, T, gather)
    x, W = _normal(g, T, n_in), _normal(g, E, n_out, n_in, std=n_in ** -0.5)
    y = torch.full((M, n_out), 7.5, dtype=F32 if f32 else BF, device="cuda")
    counts = omni.new_counts("cuda")
    out = omni.grouped_linear(x, W, off, rows=rows, silu=silu, y=y, counts=counts, **kw)
    assert out is y
    xr = (x if rows is None else x[rows.long()]).double()
    done = torch.zeros(M, dtype=torch.bool, device="cuda")
    for a, b, e in _spans(sizes, ids, listed):
        w = W[e].double()
        _close(y[a:b], xr[a:b] @ w.T, n_in * ULP * (xr[a:b].abs() @ w.abs().T), silu)
        done[a:b] = True
    assert bool((y[~done] == 7.5).all())  # rows in no group: left as they were
    assert counts.tolist() == [0, 0, 0, 0]


@pytest.mark.parametrize("f32", [False, True], ids=["bf16", "f32"])
@pytest.mark.parametrize("listed,gather", [(False, False), (True, True)])
@pytest.mark.parametrize("sizes,n_in,n_out,more", SHAPES, ids=IDS)
def test_backward(sizes, n_in, n_out, more, listed, gather, f32):
    g = _gen(2)
    kw, off, E, ids = _groups(sizes, listed)
    M = sum(sizes) + more
    T = max(1, M // 3) if gather else M
    rows = _rows(g, M, T, gather)
    x, W = _normal(g, T, n_in), _normal(g, E, n_out, n_in, std=n_in ** -0.5)
    dy = _normal(g, M, n_out)
    if more:  # rows of no group may hold anything
        dy[-more:] = float("nan")
    dx = torch.full((M, n_in), 7.5, dtype=F32 if f32 else BF, device="cuda")
    counts = omni.new_counts("cuda")
    r = omni.grouped_linear_backward(x, W, dy, off, rows=rows, dx=dx, counts=counts, **kw)
    base = torch.randn(W.shape, generator=g, device="cuda")
    added, over = base.clone(), base.clone()
    omni.grouped_linear_backward(x, W, dy, off, rows=rows, dW=added, need_dx=False, **kw)
    omni.grouped_linear_backward(x, W, dy, off, rows=rows, dW=over, need_dx=False,
                                 accumulate=False, **kw)
    xr, d = (x if rows is None else x[rows.long()]).double(), dy.double()
    done = torch.zeros(M, dtype=torch.bool, device="cuda")
    seen = set()
    for a, b, e in _spans(sizes, ids, listed):
        w = W[e].double()
        _close(dx[a:b], d[a:b] @ w, n_out * ULP * (d[a:b].abs() @ w.abs()))
        done[a:b] = True
        ref = d[a:b].T @ xr[a:b]
        err = (b - a) * ULP * (d[a:b].abs().T @ xr[a:b].abs())
        _close(r["dW"][e], ref, err)
        assert torch.equal(over[e], r["dW"][e])
        sum_ = ref + base[e].double()
        _close(added[e], sum_, err + 2.0 ** -24 * sum_.abs())
        seen.add(e)
    assert bool((dx[~done] == 7.5).all())
    for e in set(range(E)) - seen:  # matrices of no group
        assert bool((r["dW"][e] == 0).all())
        assert torch.equal(added[e], base[e]) and torch.equal(over[e], base[e])
    assert counts.tolist() == [0, 0, 0, 0]


def test_long_groups_keep_fp32_sums():
    """fp32 results over long axes are summed in pieces of 512 products: with terms of one sign,
    a piece is off by at most 512 units in the last place of itself, and adding up n/512 pieces
    by n/512 more: (512 + n/512) * 2^-23 relative, where one running sum would be allowed n."""
    g = _gen(3)
    n = M = 20000
    w = 128
    x = (torch.rand((M, w), generator=g, device="cuda") + 0.5).to(BF)
    dy = (torch.rand((M, w), generator=g, device="cuda") + 0.5).to(BF)
    W = _normal(g, 1, w, w)
    r = omni.grouped_linear_backward(x, W, dy, _i32([0, M]), need_dx=False)
    ref = dy.double().T @ x.double()
    assert float(((r["dW"][0].double() - ref) / ref).abs().max()) <= (512 + n // 512 + 1) * ULP
    # and a product over a long axis, in fp32
    n = 16384
    x = (torch.rand((40, 16384), generator=g, device="cuda") + 0.5).to(BF)
    W = (torch.rand((1, 64, 16384), generator=g, device="cuda") + 0.5).to(BF)
    y = omni.grouped_linear(x, W, _i32([0, 40]), out_dtype=F32)
    ref = x.double() @ W[0].double().T
    assert float(((y.double() - ref) / ref).abs().max()) <= (512 + n // 512 + 1) * ULP


def test_gradients_against_differences():
    """The product is linear in x and in W: on small integers every sum is exact, and a difference
    of two products equals the gradient's inner product with the step exactly."""
    g = _gen(4)
    sizes, n_in, n_out = [37, 0, 90, 5], 72, 40
    off, M = _i32(_off(sizes)), 132

    def ints(*shape):
        return torch.randint(-3, 4, shape, generator=g, device="cuda").to(BF)

    x, W, dy = ints(M, n_in), ints(4, n_out, n_in), ints(M, n_out)
    r = omni.grouped_linear_backward(x, W, dy, off, out_dtype=F32)

    def loss(x, W):
        y = omni.grouped_linear(x, W, off, out_dtype=F32)
        return float((y.double() * dy.double()).sum())

    for _ in range(3):
        hx, hW = ints(M, n_in), ints(4, n_out, n_in)
        assert loss(x + hx, W) - loss(x, W) == float((r["dx"].double() * hx.double()).sum())
        assert loss(x, W + hW) - loss(x, W) == float((r["dW"].double() * hW.double()).sum())


def test_values_of_other_groups_do_not_leak():
    """NaN and infinity stay with their rows and matrices, in tiles that span group ends too."""
    g = _gen(5)
    sizes, n_in, n_out = [5, 40, 130, 1, 70], 200, 136
    off = _i32(_off(sizes))
    M = sum(sizes)
    x, W, dy = _normal(g, M, n_in), _normal(g, 5, n_out, n_in), _normal(g, M, n_out)
    y0 = omni.grouped_linear(x, W, off)
    r0 = omni.grouped_linear_backward(x, W, dy, off)
    bad = 1  # the group of rows [5, 45)
    x2, W2, dy2 = x.clone(), W.clone(), dy.clone()
    x2[5:45], W2[bad], dy2[5:45] = float("nan"), float("inf"), float("nan")
    y = omni.grouped_linear(x2, W2, off)
    r = omni.grouped_linear_backward(x2, W2, dy2, off)
    keep = torch.ones(M, dtype=torch.bool, device="cuda")
    keep[5:45] = False
    others = [0, 2, 3, 4]
    assert torch.equal(y[keep], y0[keep]) and not bool(torch.isfinite(y[~keep]).any())
    assert torch.equal(r["dx"][keep], r0["dx"][keep])
    assert torch.equal(r["dW"][others], r0["dW"][others])
    assert bool(torch.isnan(r["dW"][bad]).all())
    # one infinite activation: its row only
    x3 = x.clone()
    x3[60, 7] = float("inf")
    y = omni.grouped_linear(x3, W, off)
    same = torch.arange(M, device="cuda") != 60
    assert torch.equal(y[same], y0[same]) and not bool(torch.isfinite(y[60]).any())


def _bad_arrays():
    """(group_off, ids, n_groups, rows of the groups that still count) on 40 rows, 4 matrices."""
    return [
        ([0, 10, 5, 20, 40], None, None, [(0, 10, 0), (20, 40, 3)]),     # an end before its start
        ([0, 10, 20, 30, 41], None, None, [(0, 10, 0), (10, 20, 1), (20, 30, 2)]),  # past M
        ([-1, 10, 20, 30, 40], None, None, [(10, 20, 1), (20, 30, 2), (30, 40, 3)]),
        ([0, 10, 20, 30, 40], [0, 2, 1, 3], None, [(0, 10, 0), (10, 20, 2), (30, 40, 3)]),
        ([0, 10, 20, 30, 40], [0, 1, 1, 3], None, [(0, 10, 0), (10, 20, 1), (30, 40, 3)]),
        ([0, 10, 20, 30, 40], [-1, 1, 2, 4], None, [(10, 20, 1), (20, 30, 2)]),
        ([0, 10, 20, 30, 40], None, 9, [(0, 10, 0), (10, 20, 1), (20, 30, 2), (30, 40, 3)]),
        ([0, 10, 20, 30, 40], None, -3, []),
    ]


@pytest.mark.parametrize("off,ids,n,spans", _bad_arrays())
def test_bad_group_arrays_are_reported(off, ids, n, spans):
    g = _gen(6)
    x, W, dy = _normal(g, 40, 64), _normal(g, 4, 72, 64), _normal(g, 40, 72)
    kw = {"ids": None if ids is None else _i32(ids), "n_groups": None if n is None else _i32([n])}
    y = torch.full((40, 72), 7.5, dtype=F32, device="cuda")
    counts, bcounts = omni.new_counts("cuda"), omni.new_counts("cuda")
    omni.grouped_linear(x, W, _i32(off), y=y, counts=counts, **kw)
    dW = torch.full((4, 72, 64), 7.5, device="cuda")
    r = omni.grouped_linear_backward(x, W, dy, _i32(off), dW=dW, accumulate=True, counts=bcounts,
                                     **kw)
    assert counts.tolist() == [0, 0, _lib.OMNI_DEV_BAD_INDEX, 0] == bcounts.tolist()
    done = torch.zeros(40, dtype=torch.bool, device="cuda")
    for a, b, e in spans:
        _close(y[a:b], x[a:b].double() @ W[e].double().T,
               64 * ULP * (x[a:b].double().abs() @ W[e].double().abs().T))
        done[a:b] = True
    assert bool((y[~done] == 7.5).all())
    for e in set(range(4)) - {e for *_, e in spans}:
        assert bool((r["dW"][e] == 7.5).all())


def test_bad_rows_are_reported():
    g = _gen(7)
    x, W, dy = _normal(g, 10, 64), _normal(g, 1, 72, 64), _normal(g, 40, 72)
    rows = torch.randint(0, 10, (40,), generator=g, device="cuda", dtype=torch.int32)
    wrong = rows.clone()
    wrong[3], wrong[39] = -1, 10
    right = wrong.clone()
    right[3] = right[39] = 0  # what a bad entry is taken as
    off = _i32([0, 40])
    for r, bit in ((right, 0), (wrong, _lib.OMNI_DEV_BAD_INDEX)):
        counts, bcounts = omni.new_counts("cuda"), omni.new_counts("cuda")
        y = omni.grouped_linear(x, W, off, rows=r, counts=counts)
        b = omni.grouped_linear_backward(x, W, dy, off, rows=r, need_dx=False, counts=bcounts)
        assert counts.tolist() == [0, 0, bit, 0] == bcounts.tolist()
        if bit == 0:
            y0, dW0 = y, b["dW"]
    assert torch.equal(y, y0) and torch.equal(b["dW"], dW0)


def test_many_groups():
    """The largest number of groups, many of them empty or of a few rows."""
    g = _gen(40)
    sizes = np.random.default_rng(41).integers(0, 7, 1024)
    off, M = _i32(_off(sizes)), int(sizes.sum())
    x, W, dy = _normal(g, M, 16), _normal(g, 1024, 24, 16), _normal(g, M, 24)
    counts = omni.new_counts("cuda")
    y = omni.grouped_linear(x, W, off, out_dtype=F32, counts=counts)
    r = omni.grouped_linear_backward(x, W, dy, off, out_dtype=F32, counts=counts)
    e = torch.repeat_interleave(torch.arange(1024, device="cuda"),
                                torch.from_numpy(sizes).cuda())
    X, Y, w = x.double(), dy.double(), W.double()[e]
    _close(y, torch.einsum("mi,moi->mo", X, w),
           16 * ULP * torch.einsum("mi,moi->mo", X.abs(), w.abs()))
    _close(r["dx"], torch.einsum("mo,moi->mi", Y, w),
           24 * ULP * torch.einsum("mo,moi->mi", Y.abs(), w.abs()))
    outer = torch.einsum("mo,mi->moi", Y, X)
    ref = torch.zeros((1024, 24, 16), dtype=torch.float64, device="cuda")
    mag = ref.clone().index_add_(0, e, outer.abs())
    _close(r["dW"], ref.index_add_(0, e, outer), 8 * ULP * mag)
    assert counts.tolist() == [0, 0, 0, 0]


def test_offsets_past_32_bits():
    """Outputs and matrices of more than 2^31 elements: the last rows, the last expert."""
    g = _gen(42)
    M, n_out = 1_050_003, 2056
    x, W = _normal(g, M, 8), _normal(g, 2, n_out, 8)
    y = omni.grouped_linear(x, W, _i32([0, 5, M]))
    ref = x[-40:].double() @ W[1].double().T
    _close(y[-40:], ref, 8 * ULP * (x[-40:].double().abs() @ W[1].double().abs().T))
    del y
    W = torch.zeros((2060, 1024, 1024), dtype=BF, device="cuda")
    W[2059] = _normal(g, 1024, 1024)
    x, dy = _normal(g, 33, 1024), _normal(g, 33, 1024)
    kw = {"ids": _i32([0, 2059])}
    y = omni.grouped_linear(x, W, _i32([0, 1, 33]), out_dtype=F32, **kw)
    w, X = W[2059].double(), x[1:].double()
    _close(y[1:], X @ w.T, 1024 * ULP * (X.abs() @ w.abs().T))
    dW = torch.zeros((2060, 1024, 1024), device="cuda")
    omni.grouped_linear_backward(x, W, dy, _i32([0, 1, 33]), dW=dW, need_dx=False, **kw)
    Y = dy[1:].double()
    _close(dW[2059], Y.T @ X, 32 * ULP * (Y.abs().T @ X.abs()))
    assert not bool(dW[1:2059].any())


def test_backward_calls_in_a_row_add_up():
    """dx and dW of a call may run side by side; calls behind one another may not.  On small
    integers every sum is exact, so the total of many calls is too."""
    g = _gen(43)
    sizes = [3, 70, 0, 129, 1, 40]
    off, M = _i32(_off(sizes)), sum(sizes)

    def ints(*shape):
        return torch.randint(-3, 4, shape, generator=g, device="cuda").to(BF)

    x, W, dy = ints(M, 264), ints(6, 136, 264), ints(M, 136)
    one = omni.grouped_linear_backward(x, W, dy, off, out_dtype=F32)
    total = torch.zeros_like(one["dW"])
    for _ in range(40):
        r = omni.grouped_linear_backward(x, W, dy, off, dW=total, out_dtype=F32)
        x2 = r["dx"].to(BF)  # the kernel behind reads dx
        assert x2.shape == (M, 264)
    assert torch.equal(total, 40 * one["dW"]) and torch.equal(r["dx"], one["dx"])


def test_no_rows():
    W = torch.ones((3, 64, 64), dtype=BF, device="cuda")
    x = torch.empty((0, 64), dtype=BF, device="cuda")
    off = _i32([0, 0, 0, 0])
    assert omni.grouped_linear(x, W, off).shape == (0, 64)
    r = omni.grouped_linear_backward(x, W, x, off)
    assert r["dx"].shape == (0, 64) and not bool(r["dW"].any())
    dW = torch.ones_like(r["dW"])
    omni.grouped_linear_backward(x, W, x, off, dW=dW, need_dx=False)
    assert bool((dW == 1).all())
    omni.grouped_linear_backward(x, W, x, off, dW=dW, need_dx=False, accumulate=False)
    assert not bool(dW.any())
    q, s = omni.quantize_rows(x)
    assert q.shape == (0, 64) and s.shape == (0,)


# ---- 8 bits ---------------------------------------------------------------------

def _quantize_ref(x):
    s = (x.double().abs().amax(-1) / 127.0).float()
    q = torch.round(x.double() / s.double()[..., None]).clamp(-127, 127)
    return torch.where(s[..., None] == 0, torch.zeros_like(q), q), s


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("n,width", [(1, 16), (5, 48), (64, 2048), (1003, 1040), (3, 65536),
                                     (5001, 1040), (4999, 2048), (4800, 16)])
def test_quantize_rows(n, width, dtype):
    g = _gen(8)
    x = torch.randn((n, width), generator=g, device="cuda")
    x = (x * torch.exp(4 * torch.randn((n, 1), generator=g, device="cuda"))).to(dtype)
    q, s = omni.quantize_rows(x)
    rq, rs = _quantize_ref(x)
    assert torch.equal(s, rs) and torch.equal(q.double(), rq)


def test_quantize_rows_at_the_borders():
    """Quotients on and beside the middle between two integers; rows of zeros, of the smallest and
    largest values; rows with an infinity or a NaN."""
    mid = torch.arange(-126, 126, device="cuda").double() + 0.5
    rows = []
    for scale in (1.0, 0.75, 1.0 / 3.0, 1e-30, 3e-39, 1e-44, 2.6e36):
        s = float(torch.tensor(127.0 * scale).float())
        v = (mid * (s / 127.0)).float()
        for ulps in (-1, 0, 1):
            r = torch.zeros(256, device="cuda")
            r[:252] = (v.view(torch.int32) + ulps).view(F32)
            r[255] = s
            rows.append(r)
    x = torch.stack(rows)
    q, s = omni.quantize_rows(x)
    rq, rs = _quantize_ref(x)
    assert torch.equal(s, rs) and torch.equal(q.double(), rq)
    z = torch.zeros((4, 32), device="cuda")
    z[1, 3], z[2, 31], z[3, 0] = float("inf"), float("nan"), float("-inf")
    q, s = omni.quantize_rows(z)
    assert not bool(q.any()) and float(s[0]) == 0.0 and bool(torch.isnan(s[1:]).all())


def _int8(g, *shape):
    q = torch.randint(-127, 128, shape, generator=g, device="cuda", dtype=torch.int32)
    return q.to(torch.int8)


def _quantized_ref(xq, xs, Wq, Ws):
    return (xq.double() @ Wq.double().T) * xs.double()[:, None] * Ws.double()


@pytest.mark.parametrize("f32,silu", [(False, False), (True, False), (False, True), (True, True)])
@pytest.mark.parametrize("M,n_in,n_out", [(1, 16, 8), (1, 2048, 8192), (2, 208, 328),
                                          (17, 1040, 1000), (64, 2048, 512), (130, 64, 72),
                                          (300, 512, 1024), (1030, 1040, 264), (5, 65536, 16)])
def test_quantized_linear(M, n_in, n_out, f32, silu):
    g = _gen(9)
    xq, Wq = _int8(g, M, n_in), _int8(g, n_out, n_in)
    xs = torch.rand(M, generator=g, device="cuda") * 0.02 + 1e-4
    Ws = torch.rand(n_out, generator=g, device="cuda") * 0.01 / n_in ** 0.5
    y = omni.quantized_linear(xq, xs, Wq, Ws, silu=silu, out_dtype=F32 if f32 else BF)
    ref = _quantized_ref(xq, xs, Wq, Ws)
    _close(y, ref, 3 * 2.0 ** -24 * ref.abs(), silu)


@pytest.mark.parametrize("listed,gather", [(False, False), (True, True)])
@pytest.mark.parametrize("sizes,n_in,n_out,more", [s for s in SHAPES if s[1] % 16 == 0])
def test_quantized_linear_by_expert(sizes, n_in, n_out, more, listed, gather):
    g = _gen(10)
    kw, off, E, ids = _groups(sizes, listed)
    M = sum(sizes) + more
    T = max(1, M // 3) if gather else M
    rows = _rows(g, M, T, gather)
    xq, Wq = _int8(g, T, n_in), _int8(g, E, n_out, n_in)
    xs = torch.rand(T, generator=g, device="cuda") + 0.5
    Ws = torch.rand((E, n_out), generator=g, device="cuda") + 0.5
    y = torch.full((M, n_out), 7.5, device="cuda")
    counts = omni.new_counts("cuda")
    omni.quantized_linear(xq, xs, Wq, Ws, off, rows=rows, y=y, counts=counts, **kw)
    at = torch.arange(M, device="cuda") if rows is None else rows.long()
    done = torch.zeros(M, dtype=torch.bool, device="cuda")
    for a, b, e in _spans(sizes, ids, listed):
        ref = _quantized_ref(xq[at[a:b]], xs[at[a:b]], Wq[e], Ws[e])
        _close(y[a:b], ref, 3 * 2.0 ** -24 * ref.abs())
        done[a:b] = True
    assert bool((y[~done] == 7.5).all()) and counts.tolist() == [0, 0, 0, 0]


def test_a_row_that_cannot_be_quantised_is_nan():
    g = _gen(11)
    x = _normal(g, 40, 64)
    x[7, 3], x[33, 63] = float("inf"), float("nan")
    Wq, Ws = omni.quantize_rows(_normal(g, 72, 64))
    y = omni.quantized_linear(*omni.quantize_rows(x), Wq, Ws)
    bad = torch.zeros(40, dtype=torch.bool, device="cuda")
    bad[7] = bad[33] = True
    assert bool(torch.isnan(y[bad]).all()) and bool(torch.isfinite(y[~bad]).all())


# ---- as they are used -----------------------------------------------------------

def _layer(T, d, F, K, seed):
    g = _gen(seed)
    D = omni.LayerDims(L=T, d=d, Nr=4, Nc=4, k=4, K=K, B=1)
    p = {"x": _normal(g, T, d), "Wr": _normal(g, 4, d, std=d ** -0.5),
         "Wc": _normal(g, 4, d, std=d ** -0.5), "W1": _normal(g, 16, F, d, std=d ** -0.5),
         "W2": _normal(g, 16, d, F, std=F ** -0.5)}
    return D, p


def _run_experts(D, p, x=None, stream=None):
    """Route, schedule with one expert per group, both products, the gated sum per token."""
    x = p["x"] if x is None else x
    idx, gate, _ = omni.route(D, x, p["Wr"], p["Wc"], stream=stream)
    s = omni.schedule(D, idx, gate, stream=stream)
    by = {"ids": s["uniq"], "n_groups": s["counts"][1:2], "stream": stream}
    h = omni.grouped_linear(x, p["W1"], s["group_off"], rows=s["task_token"], silu=True, **by)
    o = omni.grouped_linear(h, p["W2"], s["group_off"], out_dtype=F32, **by)
    y = torch.zeros((D.L, D.d), device="cuda")
    y.index_add_(0, s["task_token"].long(), o * s["task_gate"][:, None])
    return idx, gate, s, h, o, y


@pytest.mark.parametrize("T,d,F,K", [(1, 64, 128, 4), (33, 200, 328, 2), (500, 512, 256, 4)])
def test_wide_experts_behind_the_router(T, d, F, K):
    """routing -> schedule -> two grouped products -> the gated sum, against the same in 64 bits
    from the routing the GPU chose.  The hidden row h is rounded to bf16 (2^-8 relative), which
    the second product carries on: |dh| <= 2^-8 |h| + (d 2^-23 S), times |W2|."""
    D, p = _layer(T, d, F, K, seed=12)
    idx, gate, s, h, o, y = _run_experts(D, p)
    x = p["x"].double()
    ref, tol = torch.zeros_like(y, dtype=torch.float64), torch.zeros_like(y, dtype=torch.float64)
    for k in range(K):
        w1, w2 = p["W1"][idx[:, k].long()].double(), p["W2"][idx[:, k].long()].double()
        z = torch.einsum("td,tfd->tf", x, w1)
        ez = d * ULP * torch.einsum("td,tfd->tf", x.abs(), w1.abs())
        eh = (1.1 * ez + 8 * 2.0 ** -24 * z.abs()) * (1 + 2.0 ** -8) + 2.0 ** -8 * _silu(z).abs()
        gk = gate[:, k, None].double()
        ref += gk * torch.einsum("tf,tdf->td", _silu(z), w2)
        S = torch.einsum("tf,tdf->td", _silu(z).abs() + eh, w2.abs())
        tol += gk * (torch.einsum("tf,tdf->td", eh, w2.abs()) + (F + 2 * K) * ULP * S)
    assert bool(((y.double() - ref).abs() <= tol).all())
    assert int(s["counts"][2].item()) == 0
    # the hidden layer's gradients of sum(o): the schedule's arrays drive the backward too
    up = torch.ones((D.M, d), dtype=BF, device="cuda")
    b = omni.grouped_linear_backward(h, p["W2"], up, s["group_off"], ids=s["uniq"],
                                     n_groups=s["counts"][1:2])
    e = s["task_expert"].long()
    ref = p["W2"].double().sum(1)[e]
    _close(b["dx"], ref, d * ULP * p["W2"].double().abs().sum(1)[e])
    used = torch.zeros(16, dtype=torch.bool, device="cuda")
    used[e] = True
    assert not bool(b["dW"][~used].any())
    col = torch.zeros((16, F), dtype=torch.float64, device="cuda").index_add_(0, e, h.double())
    mag = torch.zeros_like(col).index_add_(0, e, h.double().abs())
    _close(b["dW"], col[:, None].expand(-1, d, -1), (D.M * ULP * mag)[:, None])


def test_quantised_mlp_next_to_the_shared_mlp():
    """The shared MLP with both matrices in 8 bits, against the same steps in 64 bits on the
    integers the GPU chose for the hidden rows; and within the quantisation's error of the bf16
    MLP (each operand off by at most half a step: |x| max / 254)."""
    g = _gen(13)
    L, d, F = 100, 256, 512
    x = _normal(g, L, d)
    W1, W2 = _normal(g, F, d, std=d ** -0.5), _normal(g, d, F, std=F ** -0.5)
    q1, s1 = omni.quantize_rows(W1)
    q2, s2 = omni.quantize_rows(W2)
    xq, xs = omni.quantize_rows(x)
    h = omni.quantized_linear(xq, xs, q1, s1, silu=True)
    z = _quantized_ref(xq, xs, q1, s1)
    _close(h, z, 3 * 2.0 ** -24 * z.abs(), silu=True)
    hq, hs = omni.quantize_rows(h)
    y = omni.quantized_linear(hq, hs, q2, s2)
    ref = _quantized_ref(hq, hs, q2, s2)
    _close(y, ref, 3 * 2.0 ** -24 * ref.abs())
    D = omni.LayerDims(L=L, d=d, Nr=8, Nc=8, k=2, K=2, B=2)
    full = omni.shared_mlp(D, x, W1, W2).double()
    X, A, B = x.double(), W1.double(), W2.double()
    ez = 0.5 * xs.double()[:, None] * (A.abs().sum(1)) + \
        (X.abs().sum(1, keepdim=True) + 0.5 * d * xs.double()[:, None]) * 0.5 * s1.double()
    H = _silu(X @ A.T)
    eh = 1.1 * ez + 2.0 ** -7 * (H.abs() + ez) + 0.5 * hs.double()[:, None]
    ey = eh @ B.abs().T + (H.abs() + eh).sum(1, keepdim=True) * 0.5 * s2.double()
    assert bool(((y.double() - full).abs() <= ey + 2.0 ** -6 * (full.abs() + ey)).all())


def test_graph_replay_on_new_routing():
    """One capture of routing, schedule, products and gradients, replayed on other tokens: every
    size that depends on the data is read on the device."""
    D, p = _layer(200, 256, 136, 4, seed=14)
    x = p["x"].clone()
    dy = _normal(_gen(15), D.M, D.d)
    stream = torch.cuda.Stream()

    def step():
        idx, gate, s, h, o, y = _run_experts(D, p, x)
        b = omni.grouped_linear_backward(h, p["W2"], dy, s["group_off"], ids=s["uniq"],
                                         n_groups=s["counts"][1:2])
        q, qs = omni.quantize_rows(x)
        return h, o, b["dx"], b["dW"], q, qs

    with torch.cuda.stream(stream):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        out = step()
    for seed in (16, 17):
        x.copy_(_normal(_gen(seed), D.L, D.d))
        for t in out:
            t.fill_(55)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        ref = step()
        torch.cuda.synchronize()
        for a, b in zip(out, ref):
            assert torch.equal(a, b)
    del graph


def test_calls_on_other_streams_are_ordered_and_independent():
    """Each call runs on the stream that is current, or on the one it is given; products on three
    streams at once keep to their own outputs, run after run bit for bit."""
    cases = []
    for i, (T, d, F) in enumerate([(300, 512, 264), (40, 200, 1000), (1000, 256, 256)]):
        D, p = _layer(T, d, F, 4, seed=20 + i)
        cases.append((D, p, [t.clone() for t in _run_experts(D, p)[3:5]], torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(3):
        got = []
        for D, p, _, st in cases:
            with torch.cuda.stream(st):
                got.append(_run_experts(D, p)[3:5])
        torch.cuda.synchronize()
        for (_, _, ref, _), g in zip(cases, got):
            assert torch.equal(g[0], ref[0]) and torch.equal(g[1], ref[1])
    # an explicit stream: ordered behind the work already on it
    D, p, ref, st = cases[0]
    with torch.cuda.stream(st):
        idx, gate, _ = omni.route(D, p["x"], p["Wr"], p["Wc"])
        s = omni.schedule(D, idx, gate)
    h = torch.empty_like(ref[0])
    h.record_stream(st)
    omni.grouped_linear(p["x"], p["W1"], s["group_off"], ids=s["uniq"],
                        n_groups=s["counts"][1:2], rows=s["task_token"], silu=True, y=h,
                        stream=st)
    st.synchronize()
    assert torch.equal(h, ref[0])
