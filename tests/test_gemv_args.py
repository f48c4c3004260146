"""Refusals of the product with 4-bit weights through the C ABI and the binding,
and the cast of the weights on the host, without a GPU."""
import ctypes

import pytest
import torch

nts = pytest.importorskip("normalization_token_split_gb300")
from normalization_token_split_gb300 import _lib  # noqa: E402

INVALID, UNSUPPORTED, OK = 1, 2, 0
P = ctypes.c_void_p
A = P(1 << 20)            # aligned, never dereferenced
MIS = P((1 << 20) + 8)
VALUES = {"e2m1": [0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6],
          "int4": [0, 1, 2, 3, 4, 5, 6, 7, -8, -7, -6, -5, -4, -3, -2, -1]}


@pytest.fixture(scope="module")
def lib():
    return _lib.lib()


def gemv(lib, a=A, lda=256, sa=None, w=A, s=A, group=32, fmt=0, y=A, out=0, M=4, N=48, K=256):
    return lib.nts_gemv_groupscaled(a, lda, sa, w, s, group, fmt, y, out, M, N, K, None)


def test_refusals(lib):
    for k in ("a", "w", "s", "y"):
        assert gemv(lib, **{k: None}) == INVALID and gemv(lib, **{k: MIS}) == UNSUPPORTED, k
    assert gemv(lib, sa=P((1 << 20) + 2)) == UNSUPPORTED
    assert gemv(lib, group=16) == INVALID and gemv(lib, group=256) == INVALID
    assert gemv(lib, fmt=2) == INVALID and gemv(lib, fmt=-1) == INVALID and gemv(lib, out=2) == INVALID
    assert gemv(lib, M=-1) == INVALID and gemv(lib, N=0) == INVALID and gemv(lib, K=0) == INVALID
    assert gemv(lib, lda=248) == INVALID and gemv(lib, lda=260) == UNSUPPORTED
    assert gemv(lib, lda=264, sa=A) == UNSUPPORTED         # codes: rows on 16 bytes
    assert gemv(lib, K=240, lda=240) == UNSUPPORTED
    assert gemv(lib, K=32800, lda=32800) == UNSUPPORTED
    assert gemv(lib, M=65535 * 16 + 1) == UNSUPPORTED and gemv(lib, N=1 << 31) == UNSUPPORTED
    assert gemv(lib, M=0, a=None, w=None, s=None, y=None) == OK
    assert gemv(lib, M=0, group=16) == INVALID
    try:
        assert lib.nts_debug_inject_failure(-1, 1) == OK
        assert gemv(lib) == 3 and b"host failure in a launch" in lib.nts_last_error()
    finally:
        assert lib.nts_debug_inject_failure(0, 0) == OK


def test_groupcast_refusals(lib):
    one = torch.ones(2, 64, dtype=torch.bfloat16)
    buf = torch.zeros(256, dtype=torch.uint8)
    p, b = P(one.data_ptr()), P(buf.data_ptr())
    assert lib.nts_groupcast_host(None, b, b, 2, 64, 32, 0) == INVALID
    assert lib.nts_groupcast_host(p, None, b, 2, 64, 32, 0) == INVALID
    assert lib.nts_groupcast_host(p, b, None, 2, 64, 32, 0) == INVALID
    assert lib.nts_groupcast_host(p, b, b, 0, 64, 32, 0) == INVALID
    assert lib.nts_groupcast_host(p, b, b, 2, 64, 48, 0) == INVALID
    assert lib.nts_groupcast_host(p, b, b, 2, 64, 32, 7) == INVALID
    assert lib.nts_groupcast_host(p, b, b, 2, 48, 32, 0) == UNSUPPORTED
    for bad in (float("inf"), float("nan")):
        one[1, 3] = bad
        with pytest.raises(nts.NtsError, match="not finite"):
            nts.groupcast(one, device="cpu")
    for w in (one.float(), one[0]):
        with pytest.raises(ValueError):
            nts.groupcast(w, device="cpu")
    with pytest.raises(ValueError):
        nts.groupcast(torch.ones(2, 64, dtype=torch.bfloat16), fmt="e4m3", device="cpu")


@pytest.mark.parametrize("fmt", ["e2m1", "int4"])
@pytest.mark.parametrize("group,K", [(32, 32), (32, 320), (64, 160), (128, 672)])
def test_groupcast_takes_the_nearest_value(fmt, group, K):
    g = torch.Generator().manual_seed(K)
    w = (torch.randn(23, K, generator=g) * 2.0 ** torch.randint(-9, 9, (23, 1), generator=g))
    w[3] = 0
    w[4, 1:] = 0
    w[5] *= 2.0 ** -120                            # below the scale's floor
    w = w.to(torch.bfloat16)
    o = nts.groupcast(w, group=group, fmt=fmt, device="cpu")
    assert o.codes.shape == (23, K // 2) and o.scales.shape == (23, -(-K // group))
    pad = torch.nn.functional.pad(w.float(), (0, -K % group)).reshape(23, -1, group)
    top = 6.0 if fmt == "e2m1" else 7.0
    scales = (pad.abs().amax(-1).clamp_min(2.0 ** -100) / top).to(torch.bfloat16)
    assert torch.equal(o.scales, scales)
    codes = torch.stack((o.codes & 15, o.codes >> 4), -1).flatten(1).long()
    q = (w.float() / scales.float().repeat_interleave(group, 1)[:, :K])
    table = torch.tensor(VALUES[fmt])
    if fmt == "int4":
        assert not (codes == 8).any()              # -8 is never written
        table[8] = 99.0
    far = (q[..., None] - table).abs()
    assert torch.equal((q - table[codes]).abs(), far.amin(-1))
    tie = (far == far.amin(-1, keepdim=True)) & (table != 0)
    tie = tie.sum(-1) > 1
    assert torch.all(codes[tie] % 2 == 0)


def test_groupcast_ties_and_signs():
    row = torch.tensor([6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0] + [-v for v in
                       (6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)] + [0.0] * 16)
    c = nts.groupcast(row[None].to(torch.bfloat16), device="cpu").codes[0]
    c = torch.stack((c & 15, c >> 4), -1).flatten()[:16].tolist()
    assert c == [7, 0, 2, 2, 4, 4, 6, 6, 15, 0, 10, 10, 12, 12, 14, 14]
    row = torch.tensor([7, 0.5, 1.5, 2.5, -0.5, -1.5, -6.5, 6.5] + [0.0] * 24)
    c = nts.groupcast(row[None].to(torch.bfloat16), fmt="int4", device="cpu").codes[0]
    c = torch.stack((c & 15, c >> 4), -1).flatten()[:8].tolist()
    assert c == [7, 0, 2, 2, 0, 14, 10, 6]


def test_binding_refuses_host_tensors():
    x, w = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(8, 32, dtype=torch.uint8)
    with pytest.raises(ValueError, match="CUDA"):
        nts.gemv_groupscaled(x, w, torch.zeros(8, 2, dtype=torch.bfloat16))
