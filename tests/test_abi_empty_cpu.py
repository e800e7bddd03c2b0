"""Batches of no tokens: every workspace size is known and the calls that take one are no-ops,
in both storage types (no CUDA call is reached on these paths)."""
import ctypes as C

import pytest

from atomic_expert_routing_b200 import _lib
from atomic_expert_routing_b200 import build as libbuild

P = C.c_void_p(4096)  # never dereferenced


@pytest.fixture(scope="module")
def lib():
    libbuild.build()
    return _lib.load()


@pytest.mark.parametrize("flags", [0, _lib.OMNI_FLAG_ROUTER_SIMT, _lib.OMNI_FLAG_STAGED_SMALL,
                                   _lib.OMNI_FLAG_DENSE_TENSOR_CORES])
@pytest.mark.parametrize("dtype", [_lib.OMNI_F32, _lib.OMNI_BF16], ids=["f32", "bf16"])
def test_no_tokens(lib, dtype, flags):
    D = _lib.Dims(L=0, d=64, Nr=64, Nc=64, k=8, K=8, B=32, dtype=dtype, flags=flags)
    for which in range(5):
        n = C.c_size_t(0)
        assert lib.omni_workspace_size(C.byref(D), which, C.byref(n)) == _lib.OMNI_OK
        assert n.value < 1 << 20
    n = C.c_size_t(0)
    for routed in (0, 1):
        rc = lib.omni_mlp_workspace_size(C.byref(D), 64, routed, C.byref(n))
        assert rc == (_lib.OMNI_OK if dtype == _lib.OMNI_BF16 else _lib.OMNI_ERR_UNSUPPORTED)
    assert lib.omni_route(C.byref(D), P, P, P, None, None, P, P, None, None, P, 1 << 20,
                          None) == _lib.OMNI_OK
