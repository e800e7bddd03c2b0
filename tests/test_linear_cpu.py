"""Host side of the wide-expert and 8-bit products: the C ABI's checks (no CUDA call is reached
on these paths) and the binding's refusals, without a GPU."""
import ctypes as C

import pytest
import torch

import atomic_expert_routing_b200 as omni
from atomic_expert_routing_b200 import _lib
from atomic_expert_routing_b200 import build as libbuild

OK, BAD, UNS = _lib.OMNI_OK, _lib.OMNI_ERR_INVALID_ARG, _lib.OMNI_ERR_UNSUPPORTED
P, ODD = C.c_void_p(4096), C.c_void_p(4096 + 8)  # aligned and not; never dereferenced here


@pytest.fixture(scope="module")
def lib():
    libbuild.build()
    return _lib.load()


def _dims(**kw):
    base = dict(M=0, T=0, in_=64, out=64, E=4, G=4, out_dtype=_lib.OMNI_BF16, flags=0)
    base.update(kw)
    return _lib.LinearDims(**base)


def _forward(lib, D, x=P, W=P, off=P, ids=None, n=None, rows=None, y=P, counts=None):
    return lib.omni_grouped_linear(C.byref(D), x, W, off, ids, n, rows, y, counts, None)


def _backward(lib, D, x=P, W=P, dy=P, off=P, rows=None, dx=P, dW=P, acc=1):
    return lib.omni_grouped_linear_backward(C.byref(D), x, W, dy, off, None, None, rows, dx, dW,
                                            acc, None, None)


def _quantized(lib, D, x=P, xs=P, W=P, Ws=P, off=P, ids=None, n=None, rows=None, y=P):
    return lib.omni_quantized_linear(C.byref(D), x, xs, W, Ws, off, ids, n, rows, y, None, None)


DIMS = [
    (dict(), OK),
    (dict(M=-1), BAD),
    (dict(T=-1), BAD),
    (dict(M=8, T=0), BAD),
    (dict(in_=0), BAD),
    (dict(out=0), BAD),
    (dict(E=0), BAD),
    (dict(G=0), BAD),
    (dict(G=5), BAD),                       # more groups than matrices
    (dict(out_dtype=2), BAD),
    (dict(flags=2), BAD),
    (dict(T=1), BAD),                       # T != M without rows
    (dict(in_=60), UNS),
    (dict(out=60), UNS),
    (dict(in_=65544), UNS),
    (dict(out=65544), UNS),
    (dict(E=2000, G=1025), UNS),
    (dict(E=1 << 30), UNS),
    (dict(M=1 << 30, T=1 << 30), UNS),
    (dict(in_=60, G=5), BAD),               # both apply: invalid first
]


@pytest.mark.parametrize("bad,code", DIMS, ids=[str(d) for d, _ in DIMS])
def test_dims_checks(lib, bad, code):
    D = _dims(**bad)
    assert _forward(lib, D) == code
    assert _backward(lib, D) == code
    assert _quantized(lib, D) == code


def test_packed_dims_are_the_structure():
    """The binding packs omni_linear_dims itself."""
    v = (5, 7, 64, 72, 9, 3, _lib.OMNI_BF16, _lib.OMNI_LINEAR_SILU)
    assert omni._pack_linear_dims(*v) == bytes(_lib.LinearDims(*v))


def test_null_dims(lib):
    assert lib.omni_grouped_linear(None, *([P] * 9)) == BAD
    assert lib.omni_grouped_linear_backward(None, *([P] * 9), 1, P, None) == BAD
    assert lib.omni_quantized_linear(None, *([P] * 11)) == BAD


def test_pointer_checks(lib):
    D = _dims(M=8, T=8)
    for kw in (dict(x=None), dict(x=ODD), dict(W=None), dict(W=ODD), dict(y=None), dict(y=ODD),
               dict(off=None), dict(off=C.c_void_p(4098)), dict(ids=C.c_void_p(4097)),
               dict(n=C.c_void_p(4097)), dict(rows=C.c_void_p(4097)),
               dict(counts=C.c_void_p(4097))):
        assert _forward(lib, D, **kw) == BAD, kw
    for kw in (dict(dx=None, dW=None), dict(dx=ODD), dict(dW=ODD), dict(dy=None), dict(x=None),
               dict(W=None), dict(off=None)):
        assert _backward(lib, D, **kw) == BAD, kw
    for kw in (dict(x=ODD), dict(xs=None), dict(xs=C.c_void_p(4097)), dict(W=None),
               dict(Ws=None), dict(y=ODD)):
        assert _quantized(lib, D, **kw) == BAD, kw
    # one matrix for every row: E = G = 1 and no group arrays
    assert _quantized(lib, D, off=None) == BAD
    one = _dims(M=8, T=8, E=1, G=1)
    assert _quantized(lib, one, off=None, ids=P) == BAD
    assert _quantized(lib, one, off=None, n=P) == BAD
    # 8-bit rows are whole 16-byte vectors
    assert _quantized(lib, _dims(in_=72)) == UNS
    assert _forward(lib, _dims(in_=72)) == OK


def test_backward_refuses_silu(lib):
    assert _backward(lib, _dims(flags=_lib.OMNI_LINEAR_SILU)) == UNS


def test_quantize_rows_checks(lib):
    def call(n=0, width=64, dtype=_lib.OMNI_BF16, src=P, q=P, scale=P):
        return lib.omni_quantize_rows(n, width, dtype, src, q, scale, None)

    assert call() == OK
    assert call(n=-1) == BAD and call(width=0) == BAD and call(dtype=2) == BAD
    assert call(width=72) == UNS and call(width=65552) == UNS and call(n=1 << 30) == UNS
    assert call(n=1, src=ODD) == BAD and call(n=1, q=ODD) == BAD and call(n=1, scale=None) == BAD


def _z(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype)


I32, I8, F32 = torch.int32, torch.int8, torch.float32
OFF = torch.tensor([0, 3, 8], dtype=I32)


def _binding_calls():
    """Each call with one argument wrong: (call, argument named in the error)."""
    x, W, dy = _z(8, 64), _z(2, 16, 64), _z(8, 16)
    xq, Wq = _z(8, 64, dtype=I8), _z(2, 16, 64, dtype=I8)
    xs, Ws = _z(8, dtype=F32), _z(2, 16, dtype=F32)
    g, b, q = omni.grouped_linear, omni.grouped_linear_backward, omni.quantized_linear
    return [
        ("x", lambda: g(x.float(), W, OFF)),
        ("x", lambda: g(_z(8, 56), W, OFF)),
        ("x", lambda: g(_z(8), W, OFF)),
        ("W", lambda: g(x, W.half(), OFF)),
        ("W", lambda: g(x, W[0], OFF)),
        ("group_off", lambda: g(x, W, OFF.long())),
        ("group_off", lambda: g(x, W, OFF[:1])),
        ("ids", lambda: g(x, W, OFF, ids=_z(1, dtype=I32))),
        ("n_groups", lambda: g(x, W, OFF, n_groups=_z(1, dtype=torch.int64))),
        ("rows", lambda: g(x, W, OFF, rows=_z(8, dtype=torch.int64))),
        ("y", lambda: g(x, W, OFF, y=_z(7, 16))),
        ("y", lambda: g(x, W, OFF, y=_z(8, 16).half())),
        ("y", lambda: g(x, W, OFF, rows=_z(9, dtype=I32), y=_z(8, 16))),
        ("out_dtype", lambda: g(x, W, OFF, out_dtype=torch.float16)),
        ("counts", lambda: g(x, W, OFF, counts=_z(3, dtype=I32))),
        ("dy", lambda: b(x, W, dy[:-1], OFF)),
        ("dy", lambda: b(x, W, dy.float(), OFF)),
        ("dx", lambda: b(x, W, dy, OFF, dx=_z(7, 64))),
        ("dW", lambda: b(x, W, dy, OFF, dW=_z(2, 16, 64))),
        ("dW", lambda: b(x, W, dy, OFF, dW=_z(1, 16, 64, dtype=F32))),
        ("need_dx", lambda: b(x, W, dy, OFF, need_dx=False, need_dW=False)),
        ("xq", lambda: q(x, xs, Wq, Ws, OFF)),
        ("Wq", lambda: q(xq, xs, W, Ws, OFF)),
        ("Wq", lambda: q(xq, xs, Wq, Ws)),
        ("xs", lambda: q(xq, xs[:-1], Wq, Ws, OFF)),
        ("Ws", lambda: q(xq, xs, Wq, Ws[:1], OFF)),
        ("group_off", lambda: q(xq, xs, Wq[0], Ws[0], ids=_z(1, dtype=I32))),
        ("x", lambda: omni.quantize_rows(x.half())),
        ("q", lambda: omni.quantize_rows(x, q=_z(7, 64, dtype=I8))),
        ("scale", lambda: omni.quantize_rows(x, scale=_z(7, dtype=F32))),
    ]


@pytest.mark.parametrize("i", range(len(_binding_calls())))
def test_binding_refuses_before_the_library(i, monkeypatch):
    def no_library(*a, **k):
        raise AssertionError("the library was reached")

    monkeypatch.setattr(_lib, "load", no_library)
    arg, call = _binding_calls()[i]
    with pytest.raises(ValueError, match=rf"^{arg}\b"):
        call()


def test_host_tensors_are_refused():
    x, W = _z(8, 64), _z(2, 16, 64)
    xq, Wq = _z(8, 64, dtype=I8), _z(2, 16, 64, dtype=I8)
    for call in (lambda: omni.grouped_linear(x, W, OFF),
                 lambda: omni.grouped_linear_backward(x, W, _z(8, 16), OFF),
                 lambda: omni.quantize_rows(x),
                 lambda: omni.quantized_linear(xq, _z(8, dtype=F32), Wq, _z(2, 16, dtype=F32),
                                               OFF)):
        with pytest.raises(ValueError, match="CUDA device"):
            call()


def test_register_split_of_the_product_kernels():
    """The kernels move registers between their warps (setmaxnreg): the shares add up to what a
    block of 512 threads starts with only if the compiler gives each thread exactly 128.  With
    fewer, the draining warps would wait for registers that never come."""
    import os
    import re

    src = os.path.join(libbuild.CSRC, "linear_tc.cu")
    libbuild.build()
    if not os.path.exists(libbuild.report(src)):
        libbuild.build(force=True)
    text = open(libbuild.report(src)).read()
    used = re.findall(r"Used (\d+) registers", text)
    assert len(used) > 20 and set(used) == {"128"}
    spills = re.findall(r"(\d+) bytes spill stores, (\d+) bytes spill loads", text)
    assert spills and all(s == ("0", "0") for s in spills)
