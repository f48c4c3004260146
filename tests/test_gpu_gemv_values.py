"""Products with 4-bit weights at the ends of what bf16 holds, by passes and by tiles:
the largest group scales.  Bounds are those of test_gpu_gemv.py."""
import pytest
import torch

from test_gpu_gemv import DEV, check, formula

pytestmark = pytest.mark.gpu

nts = pytest.importorskip("normalization_token_split_gb300")
PASSES, TILES = 1, 2


def product(kind, *args, **kw):
    nts.set_tuning(vpt=kind)
    try:
        y = nts.gemv_groupscaled(*args, out_dtype=torch.float32, **kw)
        nts.check_status()
    finally:
        nts.set_tuning()
    return y


@pytest.mark.parametrize("fmt,code", [("e2m1", 0x77), ("e2m1", 0xFF), ("int4", 0x88), ("int4", 0x77)])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("act", ["bf16", "e4m3"])
@pytest.mark.parametrize("M,kind", [(1, PASSES), (9, PASSES), (20, TILES)])
def test_the_largest_group_scales(M, kind, act, group, fmt, code):
    """The largest weights of one sign, and scales of 2^102: on their way in a pass 128
    values below 2^15 each come to less than 2^25, and the scale to 2^127."""
    K, N = 512, 40
    w = torch.full((N, K // 2), code, dtype=torch.uint8, device=DEV)
    s = torch.full((N, K // group), 2.0 ** 102, dtype=torch.bfloat16, device=DEV)
    if act == "bf16":
        a, sa = torch.full((M, K), 1.9921875, dtype=torch.bfloat16, device=DEV), None
    else:
        a = torch.full((M, K), 0x7E, dtype=torch.uint8, device=DEV)      # 448
        sa = torch.full((M, K // 128), 2.0 ** -8, device=DEV)
    want, room = formula(a, sa, w, s, group, fmt)
    y = product(kind, a, w, s, sa, group=group, fmt=fmt)
    assert torch.isfinite(y).all()
    check(y, want, room)
