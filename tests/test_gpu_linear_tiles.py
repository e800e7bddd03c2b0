"""Every kernel of the grouped products against 64 bits, at sizes that reach it (linear_cases.py):
tiles of 32, 64 and 128 columns on one CTA and of 256 on a pair, one to a CTA and several, rows
gathered and not, both result types; dW on 128 x 128 and on pairs, with rows to zero.

Tolerances, element by element: a sum of K products in fp32, each addition off by at most a unit
in the last place of the sum of the magnitudes S, K * 2^-23 * S; rounding the result v, 2^-8 |v| to
bf16 and 2^-24 |v| to fp32; SiLU carries on an error at most 1.1-fold and adds 8 * 2^-24 |v|.
Integer sums are exact, their conversion and two scales add 3 * 2^-24 |v|."""
import numpy as np
import pytest
import torch

import atomic_expert_routing_b200 as omni
from linear_cases import GRAD_W, GRAD_W_IDS, ROW_IDS, ROWS

pytestmark = pytest.mark.gpu

BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32
ULP = 2.0 ** -23


@pytest.fixture(autouse=True)
def the_rule_knows_148_sms():
    assert torch.cuda.get_device_properties(0).multi_processor_count == 148


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, *shape, std=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(BF)


def _groups(sizes):
    off = np.concatenate(([0], np.cumsum(sizes)))
    spans = [(int(a), int(b), e) for e, (a, b) in enumerate(zip(off, off[1:])) if b > a]
    return torch.tensor(off, dtype=I32, device="cuda"), spans


def _gather(g, M, on):
    """Rows of x, and the row list: of all of x in another order, some twice."""
    if not on:
        return M, None
    T = max(1, M // 2 + 3)
    return T, torch.randint(0, T, (M,), generator=g, device="cuda", dtype=I32)


def _close(got, ref, err, silu=False):
    v = ref * torch.sigmoid(ref) if silu else ref
    if silu:
        err = 1.1 * err + 8 * 2.0 ** -24 * v.abs()
    half = 2.0 ** -8 if got.dtype == BF else 2.0 ** -24
    tol = err + half * (v.abs() + err) + 1e-37
    off = (got.double() - v).abs()
    assert bool((off <= tol).all()), float((off / tol).max())


@pytest.mark.parametrize("f32", [False, True], ids=["bf16", "f32"])
@pytest.mark.parametrize("gather", [False, True], ids=["in order", "gathered"])
@pytest.mark.parametrize("width,several,sizes,n_out,n_in", ROWS, ids=ROW_IDS)
def test_forward(width, several, sizes, n_out, n_in, gather, f32):
    g = _gen(80)
    off, spans = _groups(sizes)
    M = sum(sizes)
    T, rows = _gather(g, M, gather)
    x, W = _normal(g, T, n_in), _normal(g, len(sizes), n_out, n_in, std=n_in ** -0.5)
    counts = omni.new_counts("cuda")
    kw = dict(rows=rows, out_dtype=F32 if f32 else BF, counts=counts)
    y, ys = (omni.grouped_linear(x, W, off, silu=s, **kw) for s in (False, True))
    xr = (x if rows is None else x[rows.long()]).double()
    for a, b, e in spans:
        w = W[e].double()
        ref, err = xr[a:b] @ w.T, n_in * ULP * (xr[a:b].abs() @ w.abs().T)
        _close(y[a:b], ref, err)
        _close(ys[a:b], ref, err, silu=True)
    assert counts.tolist() == [0, 0, 0, 0]


@pytest.mark.parametrize("f32", [False, True], ids=["bf16", "f32"])
@pytest.mark.parametrize("width,several,sizes,n_in,n_out", ROWS, ids=ROW_IDS)
def test_dx(width, several, sizes, n_in, n_out, f32):
    g = _gen(81)
    off, spans = _groups(sizes)
    M = sum(sizes)
    x = _normal(g, M, n_in)
    W, dy = _normal(g, len(sizes), n_out, n_in, std=n_out ** -0.5), _normal(g, M, n_out)
    counts = omni.new_counts("cuda")
    dx = omni.grouped_linear_backward(x, W, dy, off, need_dW=False, counts=counts,
                                      out_dtype=F32 if f32 else BF)["dx"]
    for a, b, e in spans:
        w, d = W[e].double(), dy[a:b].double()
        _close(dx[a:b], d @ w, n_out * ULP * (d.abs() @ w.abs()))
    assert counts.tolist() == [0, 0, 0, 0]


@pytest.mark.parametrize("f32", [False, True], ids=["bf16", "f32"])
@pytest.mark.parametrize("gather", [False, True], ids=["in order", "gathered"])
@pytest.mark.parametrize("width,several,sizes,n_out,n_in", ROWS, ids=ROW_IDS)
def test_8_bits(width, several, sizes, n_out, n_in, gather, f32):
    g = _gen(82)
    off, spans = _groups(sizes)
    M, E = sum(sizes), len(sizes)
    T, rows = _gather(g, M, gather)

    def ints(*shape):
        return torch.randint(-127, 128, shape, generator=g, device="cuda", dtype=I32).to(torch.int8)

    xq, Wq = ints(T, n_in), ints(E, n_out, n_in)
    xs = torch.rand(T, generator=g, device="cuda") * 0.02 + 1e-4
    Ws = torch.rand((E, n_out), generator=g, device="cuda") * 0.01 / n_in ** 0.5
    counts = omni.new_counts("cuda")
    kw = dict(rows=rows, out_dtype=F32 if f32 else BF, counts=counts)
    y, ys = (omni.quantized_linear(xq, xs, Wq, Ws, off, silu=s, **kw) for s in (False, True))
    at = torch.arange(M, device="cuda") if rows is None else rows.long()
    for a, b, e in spans:
        q = xq[at[a:b]].double() @ Wq[e].double().T
        ref = q * xs[at[a:b]].double()[:, None] * Ws[e].double()
        _close(y[a:b], ref, 3 * 2.0 ** -24 * ref.abs())
        _close(ys[a:b], ref, 3 * 2.0 ** -24 * ref.abs(), silu=True)
    assert counts.tolist() == [0, 0, 0, 0]


@pytest.mark.parametrize("gather", [False, True], ids=["in order", "gathered"])
@pytest.mark.parametrize("pairs,several,sizes,n_in,n_out", GRAD_W, ids=GRAD_W_IDS)
def test_dW(pairs, several, sizes, n_in, n_out, gather):
    g = _gen(83)
    off, spans = _groups(sizes)
    M, E = sum(sizes), len(sizes)
    T, rows = _gather(g, M, gather)
    x, dy = _normal(g, T, n_in), _normal(g, M, n_out)
    W = torch.zeros((E, n_out, n_in), dtype=BF, device="cuda")
    counts = omni.new_counts("cuda")
    base = torch.randn(W.shape, generator=g, device="cuda")
    added, over = base.clone(), base.clone()
    for dW, acc in ((added, True), (over, False)):
        omni.grouped_linear_backward(x, W, dy, off, rows=rows, dW=dW, need_dx=False,
                                     accumulate=acc, counts=counts)
    xr, d = (x if rows is None else x[rows.long()]).double(), dy.double()
    for a, b, e in spans:
        ref, err = d[a:b].T @ xr[a:b], (b - a) * ULP * (d[a:b].abs().T @ xr[a:b].abs())
        _close(over[e], ref, err)
        total = ref + base[e].double()
        _close(added[e], total, err + 2.0 ** -24 * total.abs())
    for e in set(range(E)) - {e for *_, e in spans}:  # a group without rows
        assert not bool(over[e].any()) and torch.equal(added[e], base[e])
    assert counts.tolist() == [0, 0, 0, 0]
