"""Calls without product rows on the GPU: dx alone, and a step whose tokens all went elsewhere."""
import pytest
import torch

import atomic_expert_routing_b200 as omni

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def _i32(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("T,rows", [(0, False), (0, True), (12, True)])
@pytest.mark.parametrize("listed", [False, True])
def test_no_rows(T, rows, listed):
    x, W = torch.ones((T, 64), dtype=BF, device="cuda"), torch.ones((3, 72, 64), dtype=BF, device="cuda")
    dy = torch.ones((0, 72), dtype=BF, device="cuda")
    off = _i32(0, 0, 0, 0)
    kw = {"rows": _i32()} if rows else {}
    if listed:
        kw.update(ids=_i32(0, 1, 2), n_groups=_i32(0))
    counts = omni.new_counts("cuda")
    assert omni.grouped_linear(x, W, off, counts=counts, **kw).shape == (0, 72)
    r = omni.grouped_linear_backward(x, W, dy, off, need_dW=False, counts=counts, **kw)
    assert set(r) == {"dx"} and r["dx"].shape == (0, 64)
    r = omni.grouped_linear_backward(x, W, dy, off, counts=counts, **kw)
    assert not bool(r["dW"].any())
    dW = torch.ones_like(r["dW"])
    omni.grouped_linear_backward(x, W, dy, off, dW=dW, counts=counts, **kw)
    assert bool((dW == 1).all())
    # overwritten: the listed matrices hold zeros, those of no group what they held
    omni.grouped_linear_backward(x, W, dy, off, dW=dW, accumulate=False, counts=counts, **kw)
    assert bool((dW == (1 if listed else 0)).all())
    xq, xs = omni.quantize_rows(x)
    Wq, Ws = omni.quantize_rows(W)
    assert omni.quantized_linear(xq, xs, Wq, Ws, off, counts=counts, **kw).shape == (0, 72)
    assert omni.quantized_linear(xq, xs, Wq[0], Ws[0],
                                 rows=kw.get("rows")).shape == (0, 72)
    assert counts.tolist() == [0, 0, 0, 0]
