"""Products of few rows with 4-bit weights and group scales, on the GPU against
the fp64 formula."""
import pytest
import torch

import block_reference as ref

pytestmark = pytest.mark.gpu

nts = pytest.importorskip("normalization_token_split_gb300")
DEV = "cuda:0"
VALUES = {"e2m1": [0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6],
          "int4": [0, 1, 2, 3, 4, 5, 6, 7, -8, -7, -6, -5, -4, -3, -2, -1]}


def weights(N, K, group, fmt, g):
    """Every code, scales over a few powers of two."""
    w = torch.randint(0, 256, (N, K // 2), generator=g, device=DEV, dtype=torch.uint8)
    s = torch.rand(N, -(-K // group), generator=g, device=DEV) + 0.5
    s = s * 2.0 ** torch.randint(-6, 3, s.shape, generator=g, device=DEV)
    s = s * (torch.randint(0, 2, s.shape, generator=g, device=DEV) * 2 - 1)
    return w, s.to(torch.bfloat16)


def rows(M, K, act, g, spread=6):
    a = torch.randn(M, K, generator=g, device=DEV)
    a = a * 2.0 ** torch.randint(-spread, spread, (1, K), generator=g, device=DEV)
    if act == "bf16":
        return a.to(torch.bfloat16), None
    o = nts.blockcast(a.to(torch.bfloat16))
    return o.codes, o.scales


def formula(a, sa, w, s, group, fmt):
    """(Y, bound), fp64.  Products of an fp16 and a code are exact in fp32; up to 128 of
    them are added on the tensor cores (counted as truncations: a whole step each), scaled,
    added over 4 groups, 2 blocks, 16 warps and 8 CTAs.  A bf16 value far below its
    neighbours is off by up to 2^-39 of the largest of its 128."""
    K = a.shape[1]
    c = torch.stack((w & 15, w >> 4), -1).flatten(1).long()
    W = torch.tensor(VALUES[fmt], device=DEV, dtype=torch.float64)[c]
    W = W * s.double().repeat_interleave(group, 1)[:, :K]
    lost = 0.0
    if sa is None:
        A = a.double()
        b = torch.nn.functional.pad(A.abs(), (0, -K % 128)).reshape(len(A), -1, 128)
        top = b.amax(-1, keepdim=True)
        lost = torch.where(b < top * 2.0 ** -31, top * 2.0 ** -39, 0.0).flatten(1)[:, :K] @ W.abs().t()
    else:
        A = ref.e4m3(a) * sa.double().repeat_interleave(128, 1)[:, :K]
    room = (2 * 128 + 4 + 2 + 16 + 8 + 8) * ref.U32 * (A.abs() @ W.abs().t()) + lost
    return A @ W.t(), room


def check(y, want, room):
    if y.dtype is torch.bfloat16:
        bound = ref.UBF16 * want.abs() + (1 + ref.UBF16) * room + 2.0 ** -133
    else:
        bound = room + 2.0 ** -126
    assert torch.all((y.double() - want).abs() <= bound)


@pytest.mark.parametrize("fmt", ["e2m1", "int4"])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("act", ["bf16", "e4m3"])
@pytest.mark.parametrize("M", [1, 3, 8, 9, 16, 17, 24, 32, 33, 70])
def test_formats_and_rows(M, act, group, fmt):
    g = torch.Generator(device=DEV).manual_seed(M)
    for N, K in ((200, 1024), (37, 672)):         # 672: the last group of 64 or 128 is short
        a, sa = rows(M, K, act, g)
        w, s = weights(N, K, group, fmt, g)
        want, room = formula(a, sa, w, s, group, fmt)
        for dtype in (torch.bfloat16, torch.float32):
            y = nts.gemv_groupscaled(a, w, s, sa, group=group, fmt=fmt, out_dtype=dtype)
            nts.check_status()
            check(y, want, room)


SIZES = [(1, 1, 32), (1, 16, 32), (2, 17, 64), (5, 15, 96), (1, 5000, 32), (3, 1, 16384), (8, 33, 256),
         (1, 12288, 4096), (1, 4099, 4096), (4, 151, 4128), (7, 1000, 4352), (8, 300, 5120),
         (16, 5120, 8192), (16, 100, 32768), (1, 40, 32768), (30, 77, 2080), (32, 2000, 5120),
         (20, 129, 16384), (40, 64, 20480), (64, 700, 4096), (1, 140000, 96), (25, 70000, 2176)]


@pytest.mark.parametrize("M,N,K", SIZES)
@pytest.mark.parametrize("group", [32, 64, 128])
def test_sizes(M, N, K, group):
    g = torch.Generator(device=DEV).manual_seed(N + K)
    fmt, act = ("e2m1", "bf16") if (N + group // 32) % 2 else ("int4", "e4m3")
    a, sa = rows(M, K, act, g)
    w, s = weights(N, K, group, fmt, g)
    y = nts.gemv_groupscaled(a, w, s, sa, group=group, fmt=fmt, out_dtype=torch.float32)
    nts.check_status()
    check(y, *formula(a, sa, w, s, group, fmt))


@pytest.mark.parametrize("M,N,K", [(1, 33, 64), (9, 100, 4128), (20, 77, 2080)])
def test_bounds_and_strides(M, N, K):
    """Rows of A at a stride, Y between bytes that stay, codes and scales likewise."""
    g = torch.Generator(device=DEV).manual_seed(3)
    a, _ = rows(M, K, "bf16", g)
    w, s = weights(N, K, 32, "e2m1", g)
    wide = torch.full((M, K + 72), float("nan"), dtype=torch.bfloat16, device=DEV)
    wide[:, 8:8 + K] = a
    want = nts.gemv_groupscaled(a, w, s)
    for dtype in (torch.bfloat16, torch.float32):
        n = M * N * (2 if dtype is torch.bfloat16 else 4)
        buf = torch.full((n + 4096,), 0xA5, dtype=torch.uint8, device=DEV)
        out = buf[2048:2048 + n].view(dtype).view(M, N)
        y = nts.gemv_groupscaled(wide[:, 8:8 + K], w, s, out=out)
        assert y.data_ptr() == out.data_ptr()
        assert bool((buf[:2048] == 0xA5).all()) and bool((buf[2048 + n:] == 0xA5).all())
        assert torch.equal(y.to(torch.bfloat16), want)
    # neighbours of codes and scales are not read into the sums
    big = torch.full((N * K // 2 + 64,), 0x77, dtype=torch.uint8, device=DEV)
    big[32:32 + N * K // 2] = w.flatten()
    bs = torch.full((s.numel() + 16,), float("nan"), dtype=torch.bfloat16, device=DEV)
    bs[8:8 + s.numel()] = s.flatten()
    y = nts.gemv_groupscaled(a, big[32:32 + N * K // 2].view(N, K // 2),
                             bs[8:8 + s.numel()].view(s.shape))
    assert torch.equal(y, want)
    nts.check_status()


@pytest.mark.parametrize("M", [1, 10, 30])
@pytest.mark.parametrize("fmt", ["e2m1", "int4"])
def test_far_apart_values(M, fmt):
    """bf16 rows over the whole range of the type, zeros and subnormals among them."""
    K, N, group = 1024, 50, 64
    g = torch.Generator(device=DEV).manual_seed(5)
    w, s = weights(N, K, group, fmt, g)
    a = torch.randn(M, K, generator=g, device=DEV)
    a = a * 2.0 ** torch.randint(-60, 60, (M, K), generator=g, device=DEV).double()
    a[:, 128:256] = 0
    a[:, 256:384] *= 2.0 ** -60
    a[:, 384:512] *= 2.0 ** -75
    a[0, 512:640] = 2.0 ** -133                   # the smallest bf16
    a[0, 640:768] = 2.0 ** 118
    a = a.to(torch.bfloat16)
    y = nts.gemv_groupscaled(a, w, s, group=group, fmt=fmt, out_dtype=torch.float32)
    nts.check_status()
    check(y, *formula(a, None, w, s, group, fmt))


def test_infinities_and_nan_stay_in_their_row():
    K, N, M = 4096, 70, 12
    g = torch.Generator(device=DEV).manual_seed(6)
    a, _ = rows(M, K, "bf16", g, spread=1)
    w, s = weights(N, K, 32, "e2m1", g)
    want = nts.gemv_groupscaled(a, w, s, out_dtype=torch.float32)
    b = a.clone()
    b[3, 100], b[7, 4000] = float("nan"), float("inf")
    t = s.clone()
    t[5, 2] = float("nan")
    y = nts.gemv_groupscaled(b, w, t, out_dtype=torch.float32)
    assert torch.all(y[3].isnan()) and not y[7].isfinite().any() and torch.all(y[:, 5].isnan())
    keep_m = [i for i in range(M) if i not in (3, 7)]
    keep_n = [i for i in range(N) if i != 5]
    assert torch.equal(y[keep_m][:, keep_n], want[keep_m][:, keep_n])
    nts.check_status()


def test_equal_calls_give_equal_bits():
    g = torch.Generator(device=DEV).manual_seed(7)
    for M, N, K in ((1, 4096, 4096), (8, 1000, 16384), (32, 3001, 5120), (64, 512, 2048)):
        a, sa = rows(M, K, "e4m3", g)
        w, s = weights(N, K, 64, "int4", g)
        y = nts.gemv_groupscaled(a, w, s, sa, group=64, fmt="int4")
        for _ in range(10):
            assert torch.equal(nts.gemv_groupscaled(a, w, s, sa, group=64, fmt="int4"), y)
    nts.check_status()


def test_beyond_32_bit_offsets():
    M, N, K = 3, 300000, 32768                    # 4.9e9 bytes of codes
    g = torch.Generator(device=DEV).manual_seed(8)
    a, _ = rows(M, K, "bf16", g)
    w = torch.randint(0, 256, (1000, K // 2), generator=g, device=DEV, dtype=torch.uint8).repeat(300, 1)
    w[-50:] = 255 - w[-50:]
    s = torch.rand(N, K // 128, generator=g, device=DEV).to(torch.bfloat16)
    y = nts.gemv_groupscaled(a, w, s, group=128)
    nts.check_status()
    check(y[:, -60:], *formula(a, None, w[-60:], s[-60:], 128, "e2m1"))
    far = torch.empty(2, 1 << 32, dtype=torch.bfloat16, device=DEV)[:, :K]
    far.copy_(a[:2])
    w, s = w[-60:].contiguous(), s[-60:].contiguous()
    assert torch.equal(nts.gemv_groupscaled(far, w, s, group=128),
                       nts.gemv_groupscaled(a[:2].contiguous(), w, s, group=128))
    y = nts.gemv_groupscaled(a[:1].expand(70000, K)[:, :32].contiguous(),
                             w[:, :16].repeat(600, 1), s[:, :1].repeat(600, 1), group=128)
    assert torch.equal(y[-1], y[0]) and y.numel() > 1 << 31   # passes, offsets of Y
    nts.check_status()


@pytest.mark.parametrize("fmt", ["e2m1", "int4"])
def test_with_the_cast_of_the_weights_and_the_norm(fmt):
    """As a decode step uses it: the error is the weights' and the activations' roundings."""
    g = torch.Generator(device=DEV).manual_seed(9)
    M, N, K = 4, 512, 1024
    x = torch.randn(M, K, generator=g, device=DEV).to(torch.bfloat16)
    w = (torch.randn(N, K, generator=g, device=DEV) * K ** -0.5).to(torch.bfloat16)
    W = nts.groupcast(w, group=32, fmt=fmt)
    X = nts.rmsnorm_blockcast(x)
    y = nts.gemv_groupscaled(X.codes, W.codes, W.scales, a_scales=X.scales, fmt=fmt)
    nts.check_status()
    check(y, *formula(X.codes, X.scales, W.codes, W.scales, 32, fmt))


def test_empty_batch_and_refusals():
    g = torch.Generator(device=DEV).manual_seed(10)
    a, _ = rows(4, 256, "bf16", g)
    w, s = weights(40, 256, 32, "e2m1", g)
    assert nts.gemv_groupscaled(a[:0], w, s).shape == (0, 40)
    o = nts.blockcast(a)
    for args, kw, match in (
            ((a.float(), w, s), {}, "a must be torch.bfloat16"),
            ((a, w.t(), s), {}, "w_codes must be contiguous"),
            ((a, w[:, :64].contiguous(), s), {}, "K/2 bytes"),
            ((a, w, s.float()), {}, "w_scales must be torch.bfloat16"),
            ((a, w, s), dict(group=64), "w_scales must have shape"),
            ((a, w, s), dict(group=48), "group must be 32, 64 or 128"),
            ((a, w, s), dict(fmt="nf4"), "'e2m1' or 'int4'"),
            ((a, w, s), dict(a_scales=o.scales), "a must be torch.uint8"),
            ((o.codes, w, s), dict(a_scales=o.scales[:3]), "a_scales must have shape"),
            ((a, w, s), dict(out=torch.zeros(40, 4, device=DEV)), "out has the wrong shape"),
            ((a, w, s), dict(out_dtype=torch.float16), "bfloat16 or float32"),
            ((a.t(), w, s), {}, "contiguous rows"),
            ((a, w.cpu(), s), {}, "w_codes must be a CUDA tensor")):
        with pytest.raises(ValueError, match=match):
            nts.gemv_groupscaled(*args, **kw)
    long = torch.zeros(1, 32768 + 32, dtype=torch.bfloat16, device=DEV)
    for bad in (lambda: nts.gemv_groupscaled(long, *weights(4, 32768 + 32, 32, "e2m1", g)),
                lambda: nts.gemv_groupscaled(torch.zeros(2, 260, dtype=torch.bfloat16,
                                                         device=DEV)[:, 4:], w, s)):
        with pytest.raises(nts.NtsError, match="UNSUPPORTED"):
            bad()
    nts.check_status()
