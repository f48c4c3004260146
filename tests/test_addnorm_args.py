"""Refusals of the residual's addition with RMSNorm and of its gradient, through
the C ABI and the binding, without a GPU."""
import ctypes
import math

import pytest
import torch

nts = pytest.importorskip("normalization_token_split_gb300")
from normalization_token_split_gb300 import _lib  # noqa: E402

INVALID, UNSUPPORTED, OK = 1, 2, 0
P = ctypes.c_void_p
A = P(1 << 20)            # aligned, never dereferenced
MIS = P((1 << 20) + 8)
MIS2 = P((1 << 20) + 2)


@pytest.fixture(scope="module")
def lib():
    return _lib.lib()


def fwd(lib, a=A, r=A, g=None, h=A, c=A, s=A, ri=None, type=0, T=3, D=256, eps=1e-6):
    return lib.nts_add_rmsnorm_blockcast(a, r, g, h, c, s, ri, type, T, D, eps, None)


def bwd(lib, a=A, r=A, ri=A, g=A, e=None, h=A, dx=None, dg=A, ws=A, wsb=1 << 30, type=0, T=3, D=256):
    return lib.nts_add_rmsnorm_backward(a, r, ri, g, e, h, dx, dg, ws, wsb, type, T, D, None)


@pytest.mark.parametrize("fn", [fwd, bwd])
def test_shared_refusals(lib, fn):
    for k in ("a", "r", "h"):
        assert fn(lib, **{k: None}) == INVALID and fn(lib, **{k: MIS}) == UNSUPPORTED, k
    assert fn(lib, g=MIS) == UNSUPPORTED and fn(lib, ri=MIS2) == UNSUPPORTED
    assert fn(lib, type=2) == INVALID and fn(lib, type=-1, T=0) == INVALID
    assert fn(lib, T=-1) == INVALID and fn(lib, D=0) == INVALID
    assert fn(lib, D=264) == UNSUPPORTED and fn(lib, D=32784) == UNSUPPORTED
    assert fn(lib, T=1 << 31) == UNSUPPORTED
    assert len(lib.nts_last_error()) > 0
    try:
        assert lib.nts_debug_inject_failure(-1, 1) == OK
        assert fn(lib) == 3 and b"host failure in a launch" in lib.nts_last_error()
    finally:
        assert lib.nts_debug_inject_failure(0, 0) == OK


def test_forward_refusals(lib):
    for k in ("c", "s"):
        assert fwd(lib, **{k: None}) == INVALID and fwd(lib, **{k: MIS2}) == UNSUPPORTED, k
    for eps in (0.0, -1.0, math.nan, math.inf):
        assert fwd(lib, eps=eps) == INVALID
    assert fwd(lib, T=0, a=None, r=None, h=None, c=None, s=None) == OK


def test_backward_refusals(lib):
    assert bwd(lib, ri=None) == INVALID
    assert bwd(lib, e=MIS) == UNSUPPORTED and bwd(lib, dx=MIS, type=1) == UNSUPPORTED
    assert bwd(lib, dx=A) == INVALID                       # a bf16 stream
    assert bwd(lib, g=None) == INVALID                     # dgamma of nothing
    assert bwd(lib, dg=MIS2) == UNSUPPORTED
    need = ctypes.c_int64()
    assert lib.nts_add_rmsnorm_backward_workspace(256, ctypes.byref(need)) == OK
    assert need.value > 0 and bwd(lib, wsb=need.value - 1) == INVALID
    assert bwd(lib, ws=None) == INVALID and bwd(lib, ws=MIS) == UNSUPPORTED
    assert lib.nts_add_rmsnorm_backward_workspace(0, ctypes.byref(need)) == INVALID
    assert lib.nts_add_rmsnorm_backward_workspace(256, None) == INVALID
    assert bwd(lib, T=0, a=None, r=None, h=None, ri=None, g=None, dg=None, ws=None) == OK


def test_binding_refuses_host_tensors():
    x, r = torch.zeros(4, 256, dtype=torch.bfloat16), torch.ones(4)
    with pytest.raises(ValueError, match="CUDA"):
        nts.add_rmsnorm_blockcast(x, x)
    with pytest.raises(ValueError, match="CUDA"):
        nts.add_rmsnorm_backward(x, x, r)
