"""The gradient of the residual's addition with RMSNorm at the ends of fp32: rows of
zeros with a subnormal eps, and rows whose sum of squares is beyond fp32."""
import pytest
import torch

from test_gpu_addnorm import DEV, TYPES, check_backward, make

pytestmark = pytest.mark.gpu

nts = pytest.importorskip("normalization_token_split_gb300")
WIDTHS = [48, 4096, 16400]                        # a warp, a CTA, a cluster to a row


@pytest.mark.parametrize("eps", [2e-39, 1e-40, 1e-45])
@pytest.mark.parametrize("res", TYPES)
@pytest.mark.parametrize("D", WIDTHS)
def test_rows_of_zeros_and_near_them(D, res, eps):
    """Any eps above zero is allowed.  Below 2^-127 rinv^2 of a row of zeros is beyond
    fp32, and rinv u is not.  2^-70 squared lies where fp32 has few digits left, so the
    factor that the formula takes is the forward pass's."""
    T = 7
    c = make(T, D, res, seed=D)
    c["x"][0], c["r"][0] = 0, 0
    c["x"][1], c["r"][1] = 3, -3
    c["r"][2], c["x"][2] = 0, c["x"][2] * 2.0 ** -70
    o = nts.add_rmsnorm_blockcast(c["x"], c["r"], c["gamma"], eps=eps, want_rinv=True)
    assert torch.isfinite(o.rinv).all() and torch.all(o.rinv[:2] > 2.0 ** 63)
    check_backward(c, o.h, o.rinv,
                   nts.add_rmsnorm_backward(c["dy"], o.h, o.rinv, c["gamma"], dres=c["e"]))
    c["e"] = None
    check_backward(c, o.h, o.rinv, nts.add_rmsnorm_backward(c["dy"], o.h, o.rinv, c["gamma"]))
    nts.check_status()


@pytest.mark.parametrize("res", TYPES)
@pytest.mark.parametrize("D", WIDTHS)
def test_rows_beyond_fp32(D, res):
    """Such a row's rinv is 0, so the gradient from behind is all that is left, also where
    the sum of u h is beyond fp32 (row 0), or its parts are and cancel to nothing (row 1)."""
    T = 6
    c = make(T, D, res, seed=D + 1)
    c["x"][:2] = 0
    c["r"][0], c["dy"][0] = 3e38, 2
    c["r"][1] = 3e38 * (1 - 2 * (torch.arange(D, device=DEV) % 2))
    c["dy"][1] = 2
    c["gamma"] = c["gamma"].abs()
    o = nts.add_rmsnorm_blockcast(c["x"], c["r"], c["gamma"], want_rinv=True)
    assert not o.rinv[:2].any() and o.rinv[2:].all()
    got = nts.add_rmsnorm_backward(c["dy"], o.h, o.rinv, c["gamma"], dres=c["e"])
    check_backward(c, o.h, o.rinv, got)
    assert torch.equal(got[0][:2], c["e"][:2])
    c["e"] = None
    got = nts.add_rmsnorm_backward(c["dy"], o.h, o.rinv, c["gamma"])
    check_backward(c, o.h, o.rinv, got)
    assert not got[0][:2].any()
    nts.check_status()
