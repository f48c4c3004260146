"""Products with 4-bit weights at the ends of what bf16 holds, by passes and by tiles:
rows that lie at one magnitude, small values beside a large one that reaches no sum, and
the largest group scales.  Bounds are those of test_gpu_gemv.py: at most 294 roundings or
truncations of a sum's magnitude, and in passes 2^-39 of the largest of 128 neighbours for
a value that is below 2^-31 of it."""
import pytest
import torch

import block_reference as ref
from test_gpu_gemv import DEV, VALUES, check, formula, weights

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


def dense(w, s, group, fmt, K):
    c = torch.stack((w & 15, w >> 4), -1).flatten(1).long()
    v = torch.tensor(VALUES[fmt], device=DEV, dtype=torch.float64)[c]
    return v * s.double().repeat_interleave(group, 1)[:, :K]


@pytest.mark.parametrize("fmt", ["e2m1", "int4"])
@pytest.mark.parametrize("group", [32, 128])
@pytest.mark.parametrize("M,kind", [(6, PASSES), (12, PASSES), (6, TILES), (40, TILES)])
@pytest.mark.parametrize("exponents,up", [((-133, -120, -60), 20), ((-10, 0, 10), 0),
                                          ((60, 100, 118), -20)])
def test_rows_of_one_magnitude(exponents, up, M, kind, group, fmt):
    """Row m at 2^e, e in turn from the smallest bf16 on, and scales that keep the result
    normal: no row and no block of a row hides behind another."""
    K, N = 1056, 70
    g = torch.Generator(device=DEV).manual_seed(M + up + 40)
    w, s = weights(N, K, group, fmt, g)
    s = (s.float() * 2.0 ** up).to(torch.bfloat16)
    if kind == TILES:                             # a group's sum comes before its scale
        exponents = [min(e, 116) for e in exponents]
    unit = torch.tensor([2.0 ** (e - (e > 0)) for e in exponents], device=DEV, dtype=torch.float64)
    a = torch.randint(1, 4, (M, K), generator=g, device=DEV).double()      # exact at 2^-133
    a = a * (torch.randint(0, 2, (M, K), generator=g, device=DEV) * 2 - 1) * unit.repeat(M)[:M, None]
    assert torch.equal(a.to(torch.bfloat16).double(), a)
    a = a.to(torch.bfloat16)
    want, room = formula(a, None, w, s, group, fmt)
    assert torch.equal(room, 294 * ref.U32 * (a.double().abs() @ dense(w, s, group, fmt, K).abs().t()))
    assert torch.all(room > 2.0 ** -123)          # what the output's range adds is little of it
    y = product(kind, a, w, s, group=group, fmt=fmt)
    check(y, want, room)
    assert torch.all((y.double() - want).abs().amax(1) < 0.01 * want.abs().amax(1))


@pytest.mark.parametrize("fmt", ["e2m1", "int4"])
@pytest.mark.parametrize("M,kind", [(3, PASSES), (14, PASSES), (20, TILES)])
@pytest.mark.parametrize("below", [24, 30, 33, 36])
def test_small_values_beside_a_large_one_without_weight(below, M, kind, fmt):
    """Only the small ones reach the sums.  A pass keeps a value down to 2^-31 of the
    largest as it is, and is off by up to 2^-39 of that one beneath; a tile keeps all."""
    K, N, group = 384, 60, 32
    g = torch.Generator(device=DEV).manual_seed(below)
    w, s = weights(N, K, group, fmt, g)
    a = torch.randn(M, K, generator=g, device=DEV).sign() * (1 + torch.rand(M, K, generator=g, device=DEV))
    a = a * 2.0 ** -below
    for block in range(3):
        at = 128 * block + 5 + block
        a[:, at] = 1.0
        byte = w[:, at // 2]
        w[:, at // 2] = byte & (0x0F if at % 2 else 0xF0)
        if fmt == "e2m1":                         # of either sign
            w[::2, at // 2] |= 0x80 if at % 2 else 0x08
    a = a.to(torch.bfloat16)
    W = dense(w, s, group, fmt, K)
    small = torch.where(a.abs() == 1, 0.0, a.double())
    want = small @ W.t()
    room = 294 * ref.U32 * (small.abs() @ W.abs().t())
    if kind == PASSES and below > 31:
        room = room + 2.0 ** -39 * (small != 0).double() @ W.abs().t()
    check(product(kind, a, w, s, group=group, fmt=fmt) * 2.0 ** below, want * 2.0 ** below,
          room * 2.0 ** below)


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
