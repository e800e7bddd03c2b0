"""Arrays of the wide-expert and 8-bit calls whose element count is right and whose layout is not:
refused.  Those that hold the same rows in another shape are taken."""
import pytest
import torch

import atomic_expert_routing_b200 as omni
from atomic_expert_routing_b200 import _lib

BF, F32, I8 = torch.bfloat16, torch.float32, torch.int8
M, IN, OUT, E = 40, 64, 16, 3


def _z(*shape, dtype=BF):
    return torch.zeros(shape, dtype=dtype)


X, W, DY = _z(M, IN), _z(E, OUT, IN), _z(M, OUT)
XQ, WQ, XS, WS = _z(M, IN, dtype=I8), _z(E, OUT, IN, dtype=I8), _z(M, dtype=F32), _z(E, OUT, dtype=F32)
OFF = torch.tensor([0, 3, 8, M], dtype=torch.int32)
CALLS = {
    "dy": lambda t: omni.grouped_linear_backward(X, W, t, OFF),
    "dx": lambda t: omni.grouped_linear_backward(X, W, DY, OFF, dx=t),
    "dW": lambda t: omni.grouped_linear_backward(X, W, DY, OFF, dW=t),
    "y": lambda t: omni.grouped_linear(X, W, OFF, y=t),
    "y of 8 bits": lambda t: omni.quantized_linear(XQ, XS, WQ, WS, OFF, y=t),
    "Ws": lambda t: omni.quantized_linear(XQ, XS, WQ, t, OFF),
    "q": lambda t: omni.quantize_rows(X, q=t),
}
KIND = {"dW": F32, "Ws": F32, "q": I8}
WRONG = [
    ("dy", (OUT, M)), ("dy", (M, OUT // 2, 2)), ("dy", (M * OUT // 8, 8)),
    ("dx", (IN, M)), ("dx", (2, IN, M // 2)),
    ("dW", (E, IN, OUT)), ("dW", (OUT, E, IN)), ("dW", (E * IN, OUT)), ("dW", (IN, OUT, E)),
    ("y", (OUT, M)), ("y of 8 bits", (OUT, M)), ("Ws", (OUT, E)), ("q", (IN, M)),
]
RIGHT = [
    ("dy", (M, OUT)), ("dy", (M * OUT,)), ("dy", (4, M // 4, OUT)), ("dy", (M + 2, OUT)),
    ("dy", (M, OUT, 1)), ("dx", (M * IN + 5,)), ("dx", (1, M, IN)),
    ("dW", (E, OUT, IN)), ("dW", (E * OUT, IN)), ("dW", (E, OUT * IN)), ("dW", (E + 1, OUT, IN)),
    ("dW", (E, 1, OUT, IN)), ("y", (M, OUT)), ("y", (2, M // 2, OUT)), ("y of 8 bits", (M, OUT)),
    ("Ws", (E, OUT)), ("Ws", (E * OUT,)), ("Ws", (E, OUT, 1)), ("q", (M, IN)), ("q", (M * IN,)),
]


@pytest.mark.parametrize("name,shape", WRONG, ids=str)
def test_wrong_layouts_are_refused(name, shape, monkeypatch):
    def no_library(*a, **k):
        raise AssertionError("the library was reached")

    monkeypatch.setattr(_lib, "load", no_library)
    with pytest.raises(ValueError, match=rf"^{name.split()[0]}: shape"):
        CALLS[name](_z(*shape, dtype=KIND.get(name, BF)))


@pytest.mark.parametrize("name,shape", RIGHT, ids=str)
def test_the_same_rows_in_another_shape_are_taken(name, shape, monkeypatch):
    reached = []
    monkeypatch.setattr(omni, "_index", lambda t: t.get_device())
    monkeypatch.setattr(omni, "_run", lambda fn, *a: reached.append(fn))
    CALLS[name](_z(*shape, dtype=KIND.get(name, BF)))
    assert len(reached) == 1
