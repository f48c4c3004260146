"""The block-128 E4M3 casts on the GPU: bit for bit against the definition's
fp32 steps, and RMSNorm's factor against fp64."""
import math

import pytest
import torch

import block_reference as ref

pytestmark = pytest.mark.gpu

nts = pytest.importorskip("normalization_token_split_gb300")
DEV = "cuda:0"
EPS = 1e-6

SHAPES = [(1, 16), (1, 4096), (3, 128), (5, 144), (2, 8192), (64, 4096), (7, 2064), (1000, 1040),
          (33, 32768), (300, 5120), (5000, 512), (9, 32752)]


def rows(T, D, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, D, generator=g)
    x[:, torch.rand(D, generator=g) < 0.02] *= 20.0
    return x.to(torch.bfloat16)


@pytest.mark.parametrize("gain", [False, True])
@pytest.mark.parametrize("T,D", SHAPES)
def test_rmsnorm_blockcast(T, D, gain):
    x = rows(T, D, T + D)
    gamma = 1.0 + 0.1 * torch.randn(D, generator=torch.Generator().manual_seed(1)) if gain else None
    o = nts.rmsnorm_blockcast(x.to(DEV), None if gamma is None else gamma.to(DEV), eps=EPS,
                              want_rinv=True)
    nts.check_status()
    rinv = o.rinv.cpu()
    want = (x.double().square().mean(1) + EPS).rsqrt()
    # a sum of D squares, halved by the root, and four roundings
    assert torch.all((rinv.double() - want).abs() <= (D / 2 + 4) * ref.U32 * want)
    w = x.float() if gamma is None else x.float() * gamma
    w = w * rinv[:, None]
    scales = ref.block_scales(w, 1)
    assert torch.equal(o.scales.cpu(), scales)
    assert torch.equal(o.codes.cpu(), ref.block_codes(w, scales, 1))


@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("T,D", SHAPES + [(127, 112), (128, 128), (129, 272), (700, 65536 + 16)])
def test_blockcast(T, D, block_rows):
    x = rows(T, D, T + D + 1)
    o = nts.blockcast(x.to(DEV), block_rows=block_rows)
    nts.check_status()
    scales = ref.block_scales(x.float(), block_rows)
    assert torch.equal(o.scales.cpu(), scales)
    assert torch.equal(o.codes.cpu(), ref.block_codes(x.float(), scales, block_rows))


@pytest.mark.parametrize("T,D", [(1, 16), (15, 64), (16, 80), (17, 48), (127, 128), (128, 4096),
                                 (129, 2064), (1000, 1040), (4099, 272)])
def test_blockcast_t(T, D):
    x = rows(T, D, T + D + 2)
    o = nts.blockcast_t(x.to(DEV))
    nts.check_status()
    Tp = -(-T // 16) * 16
    xt = torch.zeros(D, Tp)
    xt[:, :T] = x.float().t()
    scales = ref.block_scales(xt, 1)
    assert torch.equal(o.scales.cpu(), scales)
    assert torch.equal(o.codes.cpu(), ref.block_codes(xt, scales, 1))


@pytest.mark.parametrize("T,D", SHAPES + [(127, 112), (129, 272), (2, 65536 + 16), (3001, 2048)])
def test_ring_kernel_on_any_shape(T, D):
    """The kernel of large calls, forced: equal to the small calls' bit for bit."""
    x = rows(T, D, T + D + 3).to(DEV)
    gamma = 1.0 + 0.1 * torch.randn(D, generator=torch.Generator().manual_seed(2)).to(DEV)
    try:
        nts.set_tuning(stages=2)
        plain = nts.blockcast(x)
        normed = [nts.rmsnorm_blockcast(x, g, want_rinv=True) for g in (None, gamma)] \
            if D <= 32768 else []
        nts.check_status()
    finally:
        nts.set_tuning()
    scales = ref.block_scales(x.float().cpu(), 1)
    assert torch.equal(plain.scales.cpu(), scales)
    assert torch.equal(plain.codes.cpu(), ref.block_codes(x.float().cpu(), scales, 1))
    for o, g in zip(normed, (None, gamma)):
        rinv = o.rinv.cpu()
        want = (x.cpu().double().square().mean(1) + EPS).rsqrt()
        assert torch.all((rinv.double() - want).abs() <= (D / 2 + 4) * ref.U32 * want)
        w = (x.float() if g is None else x.float() * g).cpu() * rinv[:, None]
        scales = ref.block_scales(w, 1)
        assert torch.equal(o.scales.cpu(), scales)
        assert torch.equal(o.codes.cpu(), ref.block_codes(w, scales, 1))


@pytest.mark.parametrize("D", [2048, 2064, 2304, 2560, 2576, 4096, 4112, 5104, 5120, 5136, 10240,
                               16384, 16400, 20480, 20496])
def test_ring_kernel_at_the_ends_of_its_parts(D):
    """Widths at which a row goes to more warps, and at which a warp's part
    outgrows the gains that it keeps in registers."""
    T = 40
    x = rows(T, D, D).to(DEV)
    gamma = 1.0 + 0.1 * torch.randn(D, generator=torch.Generator().manual_seed(3)).to(DEV)
    try:
        nts.set_tuning(stages=2)
        o = nts.rmsnorm_blockcast(x, gamma, want_rinv=True)
        nts.check_status()
    finally:
        nts.set_tuning()
    rinv = o.rinv.cpu()
    want = (x.cpu().double().square().mean(1) + EPS).rsqrt()
    assert torch.all((rinv.double() - want).abs() <= (D / 2 + 4) * ref.U32 * want)
    w = (x.float() * gamma).cpu() * rinv[:, None]
    scales = ref.block_scales(w, 1)
    assert torch.equal(o.scales.cpu(), scales)
    assert torch.equal(o.codes.cpu(), ref.block_codes(w, scales, 1))


def test_missing_copy_times_out_and_the_context_lives():
    x = rows(700, 5120, 1).to(DEV)
    want = nts.rmsnorm_blockcast(x)
    nts.check_status()
    nts.set_wait_limit_ns(20_000_000)
    nts.set_missing_tx(16)
    nts.set_tuning(stages=2)
    try:
        nts.rmsnorm_blockcast(x)
        with pytest.raises(nts.NtsError, match="TIMEOUT"):
            nts.check_status()
    finally:
        nts.set_tuning()
        nts.set_missing_tx(0)
        nts.set_wait_limit_ns(0)
    assert torch.equal(nts.rmsnorm_blockcast(x).codes, want.codes)
    nts.check_status()


def test_zero_tiny_and_huge_blocks():
    x = torch.zeros(4, 512)
    x[1, 128:256] = 2.0 ** -120              # below the floor of the absmax
    x[1, 300] = -2.0 ** -100
    x[2, :128] = 3.3e38                      # near bf16's largest
    x[3, 5] = -0.0
    x = x.to(torch.bfloat16)
    scales = ref.block_scales(x.float(), 1)
    o = nts.blockcast(x.to(DEV))
    assert torch.equal(o.scales.cpu(), scales) and bool(torch.isfinite(o.scales).all())
    assert torch.equal(o.codes.cpu(), ref.block_codes(x.float(), scales, 1))
    assert not o.codes[0].any()
    z = nts.rmsnorm_blockcast(torch.zeros(3, 256, dtype=torch.bfloat16, device=DEV), want_rinv=True)
    assert not z.codes.any() and torch.all(torch.isfinite(z.scales))
    nts.check_status()


def test_nan_keeps_its_place_and_infinity_marks_its_block():
    x = torch.ones(2, 256, dtype=torch.bfloat16)
    x[0, 7] = float("nan")
    x[1, 200] = float("inf")
    o = nts.blockcast(x.to(DEV))
    v = o.codes.view(torch.float8_e4m3fn).float()
    assert int(torch.isnan(v[0]).sum()) == 1 and bool(torch.isnan(v[0, 7]))
    assert torch.all(v[0, :7] == 448) and torch.all(v[1, :128] == 448)
    assert math.isinf(float(o.scales[1, 1])) and bool(torch.isnan(v[1, 200]))


def test_empty_and_given_outputs():
    e = torch.empty(0, 256, dtype=torch.bfloat16, device=DEV)
    assert nts.blockcast(e).codes.shape == (0, 256)
    assert nts.rmsnorm_blockcast(e, want_rinv=True).rinv.shape == (0,)
    assert nts.blockcast_t(e).codes.shape == (256, 0)
    x = rows(100, 400, 1).to(DEV)
    want = nts.blockcast(x)
    codes = torch.empty(100, 400, dtype=torch.uint8, device=DEV)
    scales = torch.empty(100, 4, device=DEV)
    got = nts.blockcast(x, codes=codes, scales=scales)
    assert got.codes is codes and torch.equal(codes, want.codes) and torch.equal(scales, want.scales)


@pytest.mark.parametrize("T,D", [(1, 16), (37, 1040), (131, 272), (700, 4112)])
def test_canaries(T, D):
    pad = 4096
    x = rows(T, D, 77).to(DEV)

    def padded(shape, dtype):
        n = math.prod(shape) * torch.tensor([], dtype=dtype).element_size()
        buf = torch.full((2 * pad + n,), 0xA5, dtype=torch.uint8, device=DEV)
        return buf, buf[pad:pad + n].view(dtype).view(shape)

    kb, tb = -(-D // 128), -(-T // 128)
    calls = [(nts.rmsnorm_blockcast, {}, (T, D), (T, kb)), (nts.blockcast, {}, (T, D), (T, kb)),
             (nts.blockcast, {"block_rows": 128}, (T, D), (tb, kb)),
             (nts.blockcast_t, {}, (D, -(-T // 16) * 16), (D, tb))]
    for fn, kw, cs, ss in calls:
        (cb, codes), (sb, scales) = padded(cs, torch.uint8), padded(ss, torch.float32)
        fn(x, codes=codes, scales=scales, **kw)
        want = fn(x, **kw)
        nts.check_status()
        for b in (cb, sb):
            assert bool((b[:pad] == 0xA5).all()) and bool((b[-pad:] == 0xA5).all())
        assert torch.equal(codes, want.codes) and torch.equal(scales, want.scales)
