"""fp32 results are sums of pieces of 512 terms, not one running sum on the tensor core, which
cuts every addition towards zero.

With terms of one sign and about one size the partial sums grow evenly.  The tensor core adds 16
products at a time, each addition off by less than a unit in the last place, 2^-23 of its partial
sum: over the 32 of a piece at most (1 + ... + 32) / 32 * 2^-23 = 16.5 * 2^-23 of the piece.  The n
/ 512 pieces are added rounded to nearest, 2^-24 of the partial sum: (n / 512 + 1) / 2 * 2^-24 of
the result.  One running sum would be cut n / 16 times, at about 0.3 * 2^-23 of its partial sum on
average (1.1e-9 of the result per term, measured on the router's logits): five times the bound."""
import pytest
import torch

import atomic_expert_routing_b200 as omni

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
UNEVEN = 1.2  # terms are between 0.25 and 2.25, so the partial sums grow evenly within this


def _ones(g, *shape):
    return (torch.rand(shape, generator=g, device="cuda") + 0.5).to(BF)


def _check(got, ref, n):
    bound = UNEVEN * (16.5 * 2.0 ** -23 + (n / 512 + 1) / 2 * 2.0 ** -24)
    one_sum = 1.1e-9 * n
    assert 3 * bound < one_sum  # the bound tells the two apart
    assert float(((got.double() - ref) / ref).abs().max()) <= bound


@pytest.mark.parametrize("M,n_out", [(40, 64), (150, 4104), (700, 2056), (3001, 1032)])
def test_products(M, n_out):
    g = torch.Generator(device="cuda")
    g.manual_seed(90)
    n = 16384
    off = torch.tensor([0, M], dtype=torch.int32, device="cuda")
    x, W = _ones(g, M, n), _ones(g, 1, n_out, n)
    ref = x.double() @ W[0].double().T
    _check(omni.grouped_linear(x, W, off, out_dtype=F32), ref, n)
    W = W.transpose(1, 2).contiguous()
    r = omni.grouped_linear_backward(_ones(g, M, n_out), W, x, off, need_dW=False, out_dtype=F32)
    _check(r["dx"], ref, n)


@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("n_in,n_out", [(128, 128), (1032, 2056)])
def test_dW(n_in, n_out, gather):
    g = torch.Generator(device="cuda")
    g.manual_seed(91)
    n = 20007
    off = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    rows = torch.randint(0, 5000, (n,), generator=g, device="cuda", dtype=torch.int32) if gather else None
    x, dy = _ones(g, 5000 if gather else n, n_in), _ones(g, n, n_out)
    W = torch.zeros((1, n_out, n_in), dtype=BF, device="cuda")
    r = omni.grouped_linear_backward(x, W, dy, off, rows=rows, need_dx=False)
    xr = x if rows is None else x[rows.long()]
    _check(r["dW"][0], dy.double().T @ xr.double(), n)
