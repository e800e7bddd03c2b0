"""Calls without product rows, from the binding through the C ABI's checks (no CUDA call is
reached on these paths).  An empty tensor has no address; the library must not take it for one
that was not given."""
import pytest
import torch

import atomic_expert_routing_b200 as omni
from atomic_expert_routing_b200 import _lib
from atomic_expert_routing_b200 import build as libbuild

BF, F32, I8, I32 = torch.bfloat16, torch.float32, torch.int8, torch.int32


@pytest.fixture
def on_host(monkeypatch):
    libbuild.build()
    monkeypatch.setattr(omni, "_index", lambda t: t.get_device())  # -1: a host tensor's
    monkeypatch.setattr(omni, "_run", lambda fn, index, stream, *a: _lib.check(
        fn, getattr(_lib.load(), fn)(*a, None)))


def _z(*shape, dtype=BF):
    return torch.zeros(shape, dtype=dtype)


# rows of x, and the call's row list: no tokens; tokens none of which came here
EMPTY = [(0, None), (0, _z(0, dtype=I32)), (12, _z(0, dtype=I32))]
GROUPS = [dict(), dict(ids=torch.tensor([0, 2], dtype=I32)),
          dict(ids=torch.tensor([0, 0], dtype=I32), n_groups=_z(1, dtype=I32))]


@pytest.mark.parametrize("groups", range(len(GROUPS)))
@pytest.mark.parametrize("T,rows", EMPTY, ids=["no tokens", "no tokens, no rows", "no rows"])
def test_no_rows(on_host, T, rows, groups):
    x, W, dy, off = _z(T, 64), _z(3, 32, 64), _z(0, 32), _z(3, dtype=I32)
    kw = dict(rows=rows, **GROUPS[groups])
    assert omni.grouped_linear(x, W, off, **kw).shape == (0, 32)
    r = omni.grouped_linear_backward(x, W, dy, off, need_dW=False, **kw)
    assert set(r) == {"dx"} and r["dx"].shape == (0, 64)
    # added to: nothing to add
    dW = torch.ones((3, 32, 64))
    for need_dx in (False, True):
        omni.grouped_linear_backward(x, W, dy, off, dW=dW, need_dx=need_dx, **kw)
    assert bool((dW == 1).all())
    y = omni.quantized_linear(_z(T, 64, dtype=I8), _z(T, dtype=F32), _z(3, 32, 64, dtype=I8),
                              _z(3, 32, dtype=F32), off, **kw)
    assert y.shape == (0, 32)


@pytest.mark.parametrize("T,rows", EMPTY, ids=["no tokens", "no tokens, no rows", "no rows"])
def test_no_rows_of_one_matrix(on_host, T, rows):
    y = omni.quantized_linear(_z(T, 64, dtype=I8), _z(T, dtype=F32), _z(32, 64, dtype=I8),
                              _z(32, dtype=F32), rows=rows)
    assert y.shape == (0, 32)


def test_a_row_list_without_tokens_is_still_refused(on_host):
    with pytest.raises(_lib.OmniError):
        omni.grouped_linear(_z(0, 64), _z(2, 32, 64), _z(3, dtype=I32), rows=_z(5, dtype=I32))
