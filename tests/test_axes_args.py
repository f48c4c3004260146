"""Refusals of the rotation of several axes through the C ABI, and the axes of
pairs, without a GPU."""
import ctypes
import math

import pytest
import torch

nts = pytest.importorskip("normalization_token_split_gb300")
from normalization_token_split_gb300 import _lib  # noqa: E402

INVALID, UNSUPPORTED, OK = 1, 2, 0
P = ctypes.c_void_p
A = P(1 << 20)            # aligned, never dereferenced
MIS = P((1 << 20) + 4)


@pytest.fixture(scope="module")
def lib():
    return _lib.lib()


def pairs(n=64, most=2):
    return ctypes.create_string_buffer(bytes(i % (most + 1) for i in range(n)), n)


def axes(lib, Q=A, ldq=512, gq=A, Yq=A, ldyq=512, K=A, ldk=256, gk=A, Yk=A, ldyk=256, pos=A, st=3,
         sa=1, na=3, pa=..., tab=A, n=64, T=3, hq=4, hk=2, d=128, rot=128, eps=1e-6):
    pa = pairs() if pa is ... else pa
    return lib.nts_qknorm_rope_axes(Q, ldq, gq, Yq, ldyq, None, K, ldk, gk, Yk, ldyk, None, pos, st,
                                    sa, na, pa, tab, n, T, hq, hk, d, rot, 0, eps, None)


def axes_bwd(lib, Q=A, ldq=512, gq=A, K=A, ldk=256, gk=A, pos=A, st=3, sa=1, na=3, pa=..., tab=A,
             n=64, T=3, hq=4, hk=2, d=128, rot=128, eps=1e-6, ws=A, wsb=1 << 30):
    pa = pairs() if pa is ... else pa
    return lib.nts_qknorm_rope_axes_backward(A, 512, A, 256, Q, ldq, gq, K, ldk, gk, pos, st, sa, na,
                                             pa, tab, n, A, 512, A, 256, A, A, ws, wsb, T, hq, hk, d,
                                             rot, 0, eps, None)


@pytest.mark.parametrize("fn", [axes, axes_bwd])
def test_refusals(lib, fn):
    for k in ("Q", "K", "gq", "gk", "pos", "tab"):
        assert fn(lib, **{k: None}) == INVALID, k
        assert fn(lib, **{k: MIS}) == UNSUPPORTED, k
    assert fn(lib, na=0) == INVALID and fn(lib, na=5) == INVALID and fn(lib, na=-1) == INVALID
    assert fn(lib, pa=None) == INVALID
    assert fn(lib, na=2) == INVALID                        # pairs of axis 2
    assert fn(lib, pa=ctypes.create_string_buffer(b"\0" * 63 + b"\xff", 64)) == INVALID
    assert fn(lib, st=-1) == INVALID and fn(lib, sa=-1) == INVALID
    assert fn(lib, st=1 << 58) == UNSUPPORTED and fn(lib, sa=1 << 57) == UNSUPPORTED
    assert fn(lib, n=1 << 24) == UNSUPPORTED               # 2^31 table values
    assert fn(lib, T=-1) == INVALID and fn(lib, n=0) == INVALID
    assert fn(lib, rot=144) == INVALID and fn(lib, rot=24) == UNSUPPORTED
    assert fn(lib, T=1 << 30) == UNSUPPORTED
    for eps in (0.0, math.nan):
        assert fn(lib, eps=eps) == INVALID
    assert len(lib.nts_last_error()) > 0


def test_backward_refusals_and_empty_batches(lib):
    assert axes_bwd(lib, ws=None) == INVALID and axes_bwd(lib, wsb=1024) == INVALID
    assert axes_bwd(lib, eps=2.0 ** -127) == UNSUPPORTED
    none = dict(Q=None, gq=None, Yq=None, K=None, gk=None, Yk=None, pos=None, tab=None)
    assert axes(lib, T=0, **none) == OK
    assert axes(lib, T=0, na=0, **none) == INVALID
    try:
        assert lib.nts_debug_inject_failure(-1, 2) == OK
        for fn in (axes, axes_bwd):
            assert fn(lib) == 3
            assert b"host failure in a launch" in lib.nts_last_error()
    finally:
        assert lib.nts_debug_inject_failure(0, 0) == OK


def test_axes_of_pairs():
    assert nts.rope_axes((2, 3)) == b"\0\0\1\1\1"
    assert nts.rope_axes((4, 2, 1), cyclic=True) == b"\0\1\2\0\1\0\0"
    assert nts.rope_axes((0, 2, 0, 1)) == b"\1\1\3" and nts.rope_axes((3,)) == b"\0\0\0"
    for bad in ((), (1, 1, 1, 1, 1), (2, -1)):
        with pytest.raises(ValueError):
            nts.rope_axes(bad)


def test_binding_refuses_host_tensors():
    x = torch.zeros(4, 256, dtype=torch.bfloat16)
    g, pos = torch.ones(128), torch.zeros(4, 2, dtype=torch.int64)
    a = (x, g, x, g, pos, torch.zeros(8, 128), nts.rope_axes((32, 32)))
    with pytest.raises(ValueError, match="CUDA"):
        nts.qknorm_rope_axes(*a, head_dim=128)
    with pytest.raises(ValueError, match="CUDA"):
        nts.qknorm_rope_axes_backward(x, x, *a, head_dim=128)
