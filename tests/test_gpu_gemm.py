"""The block-scaled E4M3 product on the GPU against fp64, and the run from
the normalized cast through the projection to the rotated heads and back."""
import pytest
import torch

import block_reference as ref

pytestmark = pytest.mark.gpu

nts = pytest.importorskip("normalization_token_split_gb300")
DEV = "cuda:0"


def operands(M, N, K, rows, seed):
    """Codes over all finite E4M3 values, scales over six binades."""
    g = torch.Generator(device=DEV).manual_seed(seed)

    def codes(n):
        c = torch.randint(0, 254, (n, K), generator=g, device=DEV)     # 0..0x7E, 0x80..0xFE
        return (c + (c >= 127)).to(torch.uint8)

    def scales(n):
        return torch.exp2(6 * torch.rand(n, -(-K // 128), generator=g, device=DEV) - 9)

    return codes(M), scales(M), codes(N), scales(-(-N // rows))


def check(y, a, sa, w, sw, rows):
    want, mag = ref.gemm(a, sa, w, sw, rows)
    bound = ref.gemm_bound(want, mag, a.shape[1], y.dtype == torch.float32)
    bad = (y.double() - want).abs() > bound
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} outside the bound"


SHAPES = [(1, 1, 16), (1, 128, 128), (1, 4096, 4096), (3, 130, 144), (16, 256, 1024),
          (17, 1000, 2064), (33, 200, 400), (64, 384, 512), (65, 129, 272), (128, 640, 2048),
          (129, 127, 128), (130, 257, 1040), (300, 1000, 528), (333, 5120, 1280), (513, 2304, 640),
          (2048, 5120, 256), (1025, 4999, 400), (200, 33, 16), (4100, 1280, 1152)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows", [128, 1])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_product(M, N, K, rows, dtype):
    a, sa, w, sw = operands(M, N, K, rows, seed=M + N + K)
    y = nts.gemm_blockscaled(a, sa, w, sw, out_dtype=dtype)
    nts.check_status()
    assert y.shape == (M, N) and y.dtype == dtype
    check(y, a, sa, w, sw, rows)


@pytest.mark.parametrize("kernel", [1, 2, 3])
@pytest.mark.parametrize("rows", [128, 1])
@pytest.mark.parametrize("M,N,K", [(1, 1, 16), (3, 130, 144), (64, 384, 512), (130, 257, 1040),
                                   (300, 1000, 528), (513, 2305, 640), (700, 1537, 2192)])
def test_every_kernel_on_any_shape(M, N, K, rows, kernel):
    """The kernels of few rows, of single CTAs and of pairs, forced."""
    a, sa, w, sw = operands(M, N, K, rows, seed=M + N + K + 1)
    for dtype in (torch.bfloat16, torch.float32):
        try:
            nts.set_tuning(vpt=kernel)
            y = nts.gemm_blockscaled(a, sa, w, sw, out_dtype=dtype)
            nts.check_status()
        finally:
            nts.set_tuning()
        check(y, a, sa, w, sw, rows)


@pytest.mark.parametrize("kernel", [2, 3])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows", [128, 1])
@pytest.mark.parametrize("M,N,K", [(2100, 5120, 1168), (2100, 5001, 2192), (4100, 3000, 1040)])
def test_tiles_of_many_blocks_one_after_another(M, N, K, rows, dtype, kernel):
    """A CTA or pair takes several tiles, whose K blocks (10, 18 and 9) end a tile in
    the middle of a turn of the stages, of the accumulators' ring, or of the pieces
    of scales."""
    a, sa, w, sw = operands(M, N, K, rows, seed=M + N + K + 2)
    try:
        nts.set_tuning(vpt=kernel)
        y = nts.gemm_blockscaled(a, sa, w, sw, out_dtype=dtype)
        nts.check_status()
    finally:
        nts.set_tuning()
    check(y, a, sa, w, sw, rows)


def test_whole_numbers_are_exact():
    """Small whole numbers: every sum is exact in fp32."""
    g = torch.Generator(device=DEV).manual_seed(3)
    for M, N, K in ((5, 300, 640), (260, 520, 640)):
        a = torch.randint(-4, 5, (M, K), generator=g, device=DEV).float()
        w = torch.randint(-4, 5, (N, K), generator=g, device=DEV).float()
        sa = 2.0 ** torch.randint(-2, 3, (M, 5), generator=g, device=DEV)
        sw = 2.0 ** torch.randint(-2, 3, (-(-N // 128), 5), generator=g, device=DEV)
        y = nts.gemm_blockscaled(a.to(torch.float8_e4m3fn), sa, w.to(torch.float8_e4m3fn), sw,
                                 out_dtype=torch.float32)
        want = (a * ref.spread(sa, 1, M, K)).double() @ (w * ref.spread(sw, 128, N, K)).double().t()
        assert torch.equal(y.double(), want)


@pytest.mark.parametrize("M", [4, 200])
def test_nan_code_stays_in_its_row_and_column(M):
    N, K = 300, 384
    a, sa, w, sw = operands(M, N, K, 128, seed=9)
    clean = nts.gemm_blockscaled(a, sa, w, sw)
    a[2, 100] = 0x7F
    w[131, 300] = 0xFF
    y = nts.gemm_blockscaled(a, sa, w, sw)
    nan = torch.isnan(y)
    assert nan[2].all() and nan[:, 131].all() and int(nan.sum()) == M + N - 1
    assert torch.equal(y[~nan], clean[~nan])


def test_zero_scales_and_empty():
    a, sa, w, sw = operands(40, 200, 256, 128, seed=2)
    sa[3] = 0
    y = nts.gemm_blockscaled(a, sa, w, sw)
    assert not y[3].any()
    assert nts.gemm_blockscaled(a[:0], sa[:0], w, sw).shape == (0, 200)
    nts.check_status()


@pytest.mark.parametrize("M,N,K", [(1, 130, 144), (70, 515, 272), (131, 257, 400), (1100, 4999, 144)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_canaries(M, N, K, dtype):
    pad = 4096
    a, sa, w, sw = operands(M, N, K, 128, seed=4)
    n = M * N * torch.tensor([], dtype=dtype).element_size()
    buf = torch.full((2 * pad + n,), 0xA5, dtype=torch.uint8, device=DEV)
    out = buf[pad:pad + n].view(dtype).view(M, N)
    assert nts.gemm_blockscaled(a, sa, w, sw, out=out) is out
    nts.check_status()
    assert bool((buf[:pad] == 0xA5).all()) and bool((buf[-pad:] == 0xA5).all())
    assert torch.equal(out, nts.gemm_blockscaled(a, sa, w, sw, out_dtype=dtype))


@pytest.mark.parametrize("M", [1, 64, 333, 2048])
def test_equal_bits_on_streams_and_in_graphs(M):
    N, K = 2560, 1280
    a, sa, w, sw = operands(M, N, K, 128, seed=M)
    want = nts.gemm_blockscaled(a, sa, w, sw)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    outs = [torch.empty_like(want) for _ in streams]
    for _ in range(5):
        for s, o in zip(streams, outs):     # calls that may run at once
            nts.gemm_blockscaled(a, sa, w, sw, out=o, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cap = nts.gemm_blockscaled(a, sa, w, sw)
        cap2 = nts.gemm_blockscaled(a, sa, w, sw)
    for _ in range(3):
        cap.zero_()
        cap2.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(cap, want) and torch.equal(cap2, want)
    nts.check_status()


@pytest.mark.parametrize("M", [4, 300])
def test_missing_copy_times_out_and_the_context_lives(M):
    a, sa, w, sw = operands(M, 512, 512, 128, seed=1)
    want = nts.gemm_blockscaled(a, sa, w, sw)
    nts.check_status()
    nts.set_wait_limit_ns(20_000_000)
    nts.set_missing_tx(16)
    try:
        nts.gemm_blockscaled(a, sa, w, sw)
        with pytest.raises(nts.NtsError, match="TIMEOUT"):
            nts.check_status()
    finally:
        nts.set_missing_tx(0)
        nts.set_wait_limit_ns(0)
    assert torch.equal(nts.gemm_blockscaled(a, sa, w, sw), want)
    nts.check_status()


@pytest.mark.parametrize("T,hq,hk,d", [(1, 8, 2, 128), (77, 4, 4, 64), (300, 8, 2, 128)])
def test_projection_run_forward_and_backward(T, hq, hk, d):
    """x -> normalized cast -> QKV product -> rotated heads, and the gradients
    back through the rotation to the weights and the normalized input, each
    stage against fp64 on the stage's own inputs."""
    D, width = 640, (hq + 2 * hk) * d
    g = torch.Generator(device=DEV).manual_seed(T)
    x = torch.randn(T, D, generator=g, device=DEV).to(torch.bfloat16)
    w = (torch.randn(width, D, generator=g, device=DEV) * D ** -0.5).to(torch.bfloat16)
    gamma = 1.0 + 0.1 * torch.randn(D, generator=g, device=DEV)
    gq = 1.0 + 0.1 * torch.randn(d, generator=g, device=DEV)
    gk = 1.0 + 0.1 * torch.randn(d, generator=g, device=DEV)
    pos = torch.arange(T, device=DEV)
    table = nts.rope_table(T, d)

    W = nts.blockcast(w, block_rows=128)
    X = nts.rmsnorm_blockcast(x, gamma)
    qkv = nts.gemm_blockscaled(X.codes, X.scales, W.codes, W.scales)
    check(qkv, X.codes, X.scales, W.codes, W.scales, 128)
    q, k = qkv[:, :hq * d], qkv[:, hq * d:(hq + hk) * d]
    yq, yk, _, _ = nts.qknorm_rope(q, gq, k, gk, pos, table, head_dim=d)
    nts.check_status()
    for y, h, gm in ((yq, q, gq), (yk, k, gk)):
        want, _, bound = ref.rope_forward(h.cpu(), gm.cpu(), pos.cpu(), table.cpu(), d, 1e-6, False)
        assert torch.all((y.cpu().double() - want).abs() <= bound)
    # end to end against the unquantized product: E4M3 operands are off by at
    # most 2^-4 relative (2^-10/448 of their block's largest below the normal
    # range), both factors, so each sum by 2 * 2^-4 (1 + 2^-5) of its
    # magnitudes and a little for the subnormal codes
    xn = x.double() * (x.double().square().mean(1, keepdim=True) + 1e-6).rsqrt() * gamma.double()
    full, mag = xn @ w.double().t(), xn.abs() @ w.double().abs().t()
    tiny = 2.0 ** -10 / 448 * (xn.abs().amax() * w.double().abs().sum(1)[None, :]
                               + xn.abs().sum(1)[:, None] * w.double().abs().amax())
    assert torch.all((qkv.double() - full).abs()
                     <= (2.0 ** -3 * (1 + 2.0 ** -5) + 2.0 ** -7) * mag + 1.1 * tiny)

    dqkv = torch.randn(T, width, generator=g, device=DEV).to(torch.bfloat16)
    dyq, dyk = dqkv[:, :hq * d], dqkv[:, hq * d:(hq + hk) * d]
    want_q = ref.rope_backward(dyq.cpu(), q.cpu(), gq.cpu(), pos.cpu(), table.cpu(), d, 1e-6, False)
    nts.qknorm_rope_backward(dyq, dyk, q, gq, k, gk, pos, table, head_dim=d, out_dq=dyq,
                             out_dk=dyk)
    assert torch.all((dyq.cpu().double() - want_q[0]).abs() <= want_q[2])
    # gradient of the normalized input: the same product with the weights transposed
    dY = nts.blockcast(dqkv)
    Wt = (W.codes.t().contiguous(), W.scales.t().contiguous())
    dX = nts.gemm_blockscaled(dY.codes, dY.scales, *Wt)
    check(dX, dY.codes, dY.scales, *Wt, 128)
    # gradient of the weights: sums over the tokens of transposed operands
    xn16 = xn.to(torch.bfloat16)
    dYt, Xt = nts.blockcast_t(dqkv), nts.blockcast_t(xn16)
    dW = nts.gemm_blockscaled(dYt.codes, dYt.scales, Xt.codes, Xt.scales, out_dtype=torch.float32)
    check(dW, dYt.codes, dYt.scales, Xt.codes, Xt.scales, 1)
    assert dW.shape == w.shape
    nts.check_status()


@pytest.mark.parametrize("kernel,M,N,K", [(1, 600, 2000, 2192), (2, 2500, 2600, 1168),
                                          (3, 2100, 5120, 1168), (3, 600, 520, 4112)])
@pytest.mark.parametrize("rows", [128, 1])
def test_a_wait_that_expires_ends_every_tile(kernel, M, N, K, rows):
    """Several tiles for a CTA, or several pieces of scales for a tile: all roles
    leave their loops, by whole warps, and the next product is right."""
    a, sa, w, sw = operands(M, N, K, rows, seed=M)
    try:
        nts.set_tuning(vpt=kernel)
        want = nts.gemm_blockscaled(a, sa, w, sw)
        nts.check_status()
        check(want, a, sa, w, sw, rows)
        nts.set_wait_limit_ns(20_000_000)
        nts.set_missing_tx(16)
        for _ in range(3):
            nts.gemm_blockscaled(a, sa, w, sw)
            with pytest.raises(nts.NtsError, match="TIMEOUT"):
                nts.check_status()
        nts.set_missing_tx(0)
        nts.set_wait_limit_ns(0)
        assert torch.equal(nts.gemm_blockscaled(a, sa, w, sw), want)
        nts.check_status()
    finally:
        nts.set_missing_tx(0)
        nts.set_wait_limit_ns(0)
        nts.set_tuning()
