"""Refusals of the operators around a QKV projection, through the C ABI and
the binding, without a GPU; and the rotation table formed on the host."""
import ctypes
import math

import numpy as np
import pytest
import torch

nts = pytest.importorskip("normalization_token_split_gb300")
from normalization_token_split_gb300 import _lib  # noqa: E402

INVALID, UNSUPPORTED, OK = 1, 2, 0
P = ctypes.c_void_p
A = P(1 << 20)            # aligned, never dereferenced
MIS = P((1 << 20) + 4)
MIS2 = P((1 << 20) + 2)


@pytest.fixture(scope="module")
def lib():
    return _lib.lib()


def rope(lib, Q=A, ldq=512, gq=A, Yq=A, ldyq=512, rq=None, K=A, ldk=256, gk=A, Yk=A, ldyk=256,
         rk=None, pos=A, tab=A, n=64, T=3, hq=4, hk=2, d=128, rot=128, il=0, eps=1e-6):
    return lib.nts_qknorm_rope(Q, ldq, gq, Yq, ldyq, rq, K, ldk, gk, Yk, ldyk, rk, pos, tab, n, T,
                               hq, hk, d, rot, il, eps, None)


def rope_bwd(lib, dYq=A, lddyq=512, dYk=A, lddyk=256, Q=A, ldq=512, gq=A, K=A, ldk=256, gk=A,
             pos=A, tab=A, n=64, dQ=A, lddq=512, dK=A, lddk=256, dgq=A, dgk=A, ws=A, wsb=1 << 30,
             T=3, hq=4, hk=2, d=128, rot=128, il=0, eps=1e-6):
    return lib.nts_qknorm_rope_backward(dYq, lddyq, dYk, lddyk, Q, ldq, gq, K, ldk, gk, pos, tab,
                                        n, dQ, lddq, dK, lddk, dgq, dgk, ws, wsb, T, hq, hk, d,
                                        rot, il, eps, None)


@pytest.mark.parametrize("fn", [rope, rope_bwd])
def test_rope_refusals(lib, fn):
    for k in ("Q", "K", "gq", "gk", "pos", "tab"):
        assert fn(lib, **{k: None}) == INVALID, k
        assert fn(lib, **{k: MIS}) == UNSUPPORTED, k
    assert fn(lib, T=-1) == INVALID
    assert fn(lib, n=0) == INVALID
    assert fn(lib, hq=0) == INVALID and fn(lib, hk=-1) == INVALID
    assert fn(lib, d=0) == INVALID
    assert fn(lib, rot=0) == INVALID and fn(lib, rot=144) == INVALID and fn(lib, rot=15) == INVALID
    assert fn(lib, rot=24) == UNSUPPORTED
    assert fn(lib, d=120, rot=16) == UNSUPPORTED
    assert fn(lib, d=528, rot=16, ldq=9999 * 8, ldk=9999 * 8) == UNSUPPORTED
    assert fn(lib, ldq=504) == INVALID          # below the row
    assert fn(lib, ldk=260) == UNSUPPORTED      # rows off 16-byte boundaries
    assert fn(lib, hq=65537, ldq=65537 * 128) == UNSUPPORTED
    assert fn(lib, T=1 << 31) == UNSUPPORTED
    for eps in (0.0, -1.0, math.nan, math.inf):
        assert fn(lib, eps=eps) == INVALID
    assert len(lib.nts_last_error()) > 0


def test_rope_forward_refusals(lib):
    assert rope(lib, Yq=None) == INVALID and rope(lib, Yk=MIS) == UNSUPPORTED
    assert rope(lib, ldyq=256) == INVALID and rope(lib, ldyk=257) == UNSUPPORTED
    assert rope(lib, rq=MIS2) == UNSUPPORTED
    none = dict(Q=None, gq=None, Yq=None, K=None, gk=None, Yk=None, pos=None, tab=None)
    assert rope(lib, T=0, **none) == OK
    assert rope(lib, T=0, n=0, **none) == INVALID


def test_rope_backward_refusals(lib):
    for k in ("dYq", "dYk", "dQ", "dK", "dgq", "dgk"):
        assert rope_bwd(lib, **{k: None}) == INVALID, k
    assert rope_bwd(lib, lddyq=8) == INVALID and rope_bwd(lib, lddk=264 + 4) == UNSUPPORTED
    need = ctypes.c_int64()
    assert lib.nts_qknorm_rope_backward_workspace(128, ctypes.byref(need)) == OK
    assert need.value > 0 and need.value % 4 == 0
    assert rope_bwd(lib, wsb=need.value - 1) == INVALID
    assert rope_bwd(lib, ws=None) == INVALID
    assert rope_bwd(lib, ws=MIS2) == UNSUPPORTED
    assert lib.nts_qknorm_rope_backward_workspace(0, ctypes.byref(need)) == INVALID
    assert lib.nts_qknorm_rope_backward_workspace(128, None) == INVALID


def test_rope_table(lib):
    assert lib.nts_rope_table_host(4, 7, 1e4, A) == INVALID
    assert lib.nts_rope_table_host(4, 0, 1e4, A) == INVALID
    assert lib.nts_rope_table_host(-1, 8, 1e4, A) == INVALID
    assert lib.nts_rope_table_host(4, 8, 0.0, A) == INVALID
    assert lib.nts_rope_table_host(4, 8, math.inf, A) == INVALID
    assert lib.nts_rope_table_host(4, 8, 1e4, None) == INVALID
    assert lib.nts_rope_table_host(0, 8, 1e4, None) == OK
    t = nts.rope_table(3000, 32, base=10000.0, device="cpu").numpy().astype(np.float64)
    ang = np.arange(3000)[:, None] * 10000.0 ** (-2.0 * np.arange(16) / 32)
    assert np.abs(t[:, :16] - np.cos(ang)).max() <= 1.01 * 2.0 ** -25
    assert np.abs(t[:, 16:] - np.sin(ang)).max() <= 1.01 * 2.0 ** -25


def test_cast_refusals(lib):
    def norm(X=A, g=None, c=A, s=A, r=None, T=3, D=256, eps=1e-6):
        return lib.nts_rmsnorm_blockcast(X, g, c, s, r, T, D, eps, None)

    def plain(X=A, c=A, s=A, T=3, D=256, rows=1):
        return lib.nts_blockcast(X, c, s, T, D, rows, None)

    def trans(X=A, c=A, s=A, T=3, D=256):
        return lib.nts_blockcast_t(X, c, s, T, D, None)

    for fn in (norm, plain, trans):
        assert fn(X=None) == INVALID and fn(c=None) == INVALID and fn(s=None) == INVALID
        assert fn(T=-1) == INVALID and fn(D=0) == INVALID
        assert fn(D=264) == UNSUPPORTED and fn(X=MIS) == UNSUPPORTED and fn(c=MIS) == UNSUPPORTED
        assert fn(s=MIS2) == UNSUPPORTED and fn(T=1 << 31) == UNSUPPORTED
        assert fn(T=0, X=None, c=None, s=None) == OK
    assert norm(eps=0.0) == INVALID and norm(D=32784) == UNSUPPORTED
    assert norm(g=MIS) == UNSUPPORTED and norm(r=MIS2) == UNSUPPORTED
    assert plain(rows=64) == INVALID and plain(rows=64, T=0) == INVALID


def test_gemm_refusals(lib):
    def gemm(a=A, sa=A, w=A, sw=A, rows=128, y=A, out=0, M=4, N=256, K=256):
        return lib.nts_gemm_blockscaled(a, sa, w, sw, rows, y, out, M, N, K, None)

    for k in ("a", "sa", "w", "sw", "y"):
        assert gemm(**{k: None}) == INVALID, k
    for k in ("a", "w", "y"):
        assert gemm(**{k: MIS}) == UNSUPPORTED, k
    assert gemm(sa=MIS2) == UNSUPPORTED and gemm(sw=MIS2) == UNSUPPORTED
    assert gemm(rows=64) == INVALID and gemm(out=2) == INVALID
    assert gemm(M=-1) == INVALID and gemm(N=0) == INVALID and gemm(K=0) == INVALID
    assert gemm(K=200) == UNSUPPORTED
    assert gemm(M=1 << 31) == UNSUPPORTED and gemm(N=(1 << 31) - 256) == UNSUPPORTED
    assert gemm(M=0, a=None, sa=None, w=None, sw=None, y=None) == OK
    assert gemm(M=0, K=200) == UNSUPPORTED


def test_binding_refuses_host_tensors():
    x = torch.zeros(4, 256, dtype=torch.bfloat16)
    g = torch.ones(128)
    with pytest.raises(ValueError, match="CUDA"):
        nts.rmsnorm_blockcast(x)
    with pytest.raises(ValueError, match="CUDA"):
        nts.blockcast(x)
    with pytest.raises(ValueError, match="CUDA"):
        nts.blockcast_t(x)
    with pytest.raises(ValueError, match="CUDA"):
        nts.gemm_blockscaled(x.view(torch.uint8), g, x.view(torch.uint8), g)
    with pytest.raises(ValueError, match="CUDA"):
        nts.qknorm_rope(x, g, x, g, torch.zeros(4, dtype=torch.int64), torch.zeros(8, 128),
                        head_dim=128)


def test_a_cpp_exception_ends_as_a_status(lib):
    """Nothing is thrown through the C entries, whose callers cannot catch it."""
    calls = [lambda: rope(lib), lambda: rope_bwd(lib),
             lambda: lib.nts_rmsnorm_blockcast(A, None, A, A, None, 3, 256, 1e-6, None),
             lambda: lib.nts_blockcast(A, A, A, 3, 256, 1, None),
             lambda: lib.nts_blockcast(A, A, A, 3, 256, 128, None),
             lambda: lib.nts_blockcast_t(A, A, A, 3, 256, None),
             lambda: lib.nts_gemm_blockscaled(A, A, A, A, 128, A, 0, 4, 256, 256, None)]
    try:
        for call in calls:
            assert lib.nts_debug_inject_failure(-1, 1) == OK
            assert call() == 3                    # CUDA
            assert b"host failure in a launch" in lib.nts_last_error()
    finally:
        assert lib.nts_debug_inject_failure(0, 0) == OK


@pytest.mark.parametrize("fn", [rope, rope_bwd])
def test_rope_refuses_more_items_than_32_bits_count(lib, fn):
    """4 + 2 heads of 128 are two items a token, of 512 six: 2^31 - 1 items at most."""
    assert fn(lib, T=1 << 30) == UNSUPPORTED
    assert fn(lib, T=(1 << 31) // 6 + 1, d=512, ldq=2048, ldk=1024, **(
        dict(ldyq=2048, ldyk=1024) if fn is rope else
        dict(lddyq=2048, lddyk=1024, lddq=2048, lddk=1024))) == UNSUPPORTED


def test_rope_backward_refuses_an_eps_whose_rinv_squared_overflows(lib):
    assert rope_bwd(lib, eps=2.0 ** -127) == UNSUPPORTED
    assert rope_bwd(lib, eps=2.0 ** -149, T=0) == UNSUPPORTED


def test_cast_refuses_more_blocks_than_a_launch_holds(lib):
    assert lib.nts_blockcast_t(A, A, A, 65535 * 128 + 1, 256, None) == UNSUPPORTED
    assert lib.nts_blockcast(A, A, A, 1 << 30, 256 * 128, 128, None) == UNSUPPORTED   # 2^31
