"""Products of more than 16 rows with 4-bit weights by tiles on the tensor cores: the
same formula and bounds as of the passes (a group's products are exact in fp32 and at
most 128; a team adds at most four groups of each of at most 17 K blocks at these sizes,
then two teams and 8 CTAs are added, fewer roundings than the passes' bound counts)."""
import threading

import pytest
import torch

from test_gpu_gemv import DEV, check, formula, rows, weights

pytestmark = pytest.mark.gpu

nts = pytest.importorskip("normalization_token_split_gb300")


@pytest.fixture
def tiles():
    nts.set_tuning(vpt=2)
    yield
    nts.set_tuning()


@pytest.mark.parametrize("fmt", ["e2m1", "int4"])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("act", ["bf16", "e4m3"])
@pytest.mark.parametrize("M", [1, 17, 31, 32, 33, 70])
def test_formats_and_rows(tiles, M, act, group, fmt):
    g = torch.Generator(device=DEV).manual_seed(M)
    for N, K in ((200, 1024), (37, 672), (1, 32), (128, 160)):
        a, sa = rows(M, K, act, g)
        w, s = weights(N, K, group, fmt, g)
        want, room = formula(a, sa, w, s, group, fmt)
        for dtype in (torch.bfloat16, torch.float32):
            y = nts.gemv_groupscaled(a, w, s, sa, group=group, fmt=fmt, out_dtype=dtype)
            nts.check_status()
            check(y, want, room)


@pytest.mark.parametrize("M,N,K", [(20, 4001, 4224), (32, 20000, 4096), (24, 129, 32768),
                                   (40, 640, 2080), (100, 1300, 96), (17, 30000, 608)])
@pytest.mark.parametrize("group", [32, 64, 128])
def test_sizes(tiles, M, N, K, group):
    """Clusters of every size, one CTA with many K blocks, more tiles than SMs."""
    g = torch.Generator(device=DEV).manual_seed(N)
    for fmt, act in (("e2m1", "bf16"), ("int4", "e4m3")):
        a, sa = rows(M, K, act, g)
        w, s = weights(N, K, group, fmt, g)
        y = nts.gemv_groupscaled(a, w, s, sa, group=group, fmt=fmt, out_dtype=torch.float32)
        nts.check_status()
        check(y, *formula(a, sa, w, s, group, fmt))


@pytest.mark.parametrize("M,N,K", [(17, 4128, 4096), (32, 5000, 3584)])
def test_chosen_by_size(M, N, K):
    """Without a choice by hand: more than 16 rows and more than 4096 x 4096 weights."""
    g = torch.Generator(device=DEV).manual_seed(1)
    a, _ = rows(M, K, "bf16", g)
    w, s = weights(N, K, 64, "int4", g)
    auto = nts.gemv_groupscaled(a, w, s, group=64, fmt="int4", out_dtype=torch.float32)
    nts.set_tuning(vpt=2)
    try:
        byhand = nts.gemv_groupscaled(a, w, s, group=64, fmt="int4", out_dtype=torch.float32)
    finally:
        nts.set_tuning()
    nts.check_status()
    assert torch.equal(auto, byhand)
    check(auto, *formula(a, None, w, s, 64, "int4"))


@pytest.mark.parametrize("act", ["bf16", "e4m3"])
@pytest.mark.parametrize("M,N,K", [(20, 77, 2080), (33, 130, 160)])
def test_bounds_and_strides(tiles, M, N, K, act):
    """bf16 rows at a stride with NaN between them, Y between bytes that stay."""
    g = torch.Generator(device=DEV).manual_seed(3)
    a, sa = rows(M, K, act, g)
    w, s = weights(N, K, 32, "e2m1", g)
    x = a
    if act == "bf16":                             # codes have no row stride
        x = torch.full((M, K + 32), float("nan"), dtype=torch.bfloat16, device=DEV)[:, 16:16 + K]
        x.copy_(a)
    want = nts.gemv_groupscaled(a, w, s, sa)
    for dtype in (torch.bfloat16, torch.float32):
        n = M * N * (2 if dtype is torch.bfloat16 else 4)
        buf = torch.full((n + 4096,), 0xA5, dtype=torch.uint8, device=DEV)
        out = buf[2048:2048 + n].view(dtype).view(M, N)
        nts.gemv_groupscaled(x, w, s, sa, out=out)
        assert bool((buf[:2048] == 0xA5).all()) and bool((buf[2048 + n:] == 0xA5).all())
        assert torch.equal(out.to(torch.bfloat16), want)
    big = torch.full((N * K // 2 + 64,), 0x77, dtype=torch.uint8, device=DEV)
    big[32:32 + N * K // 2] = w.flatten()
    bs = torch.full((s.numel() + 16,), float("nan"), dtype=torch.bfloat16, device=DEV)
    bs[8:8 + s.numel()] = s.flatten()
    y = nts.gemv_groupscaled(a, big[32:32 + N * K // 2].view(N, K // 2),
                             bs[8:8 + s.numel()].view(s.shape), sa)
    assert torch.equal(y, want)
    nts.check_status()


def test_infinities_and_nan_stay_in_their_row(tiles):
    K, N, M = 4096, 300, 37
    g = torch.Generator(device=DEV).manual_seed(6)
    a, _ = rows(M, K, "bf16", g, spread=1)
    w, s = weights(N, K, 32, "e2m1", g)
    want = nts.gemv_groupscaled(a, w, s, out_dtype=torch.float32)
    b = a.clone()
    b[3, 100], b[34, 4000] = float("nan"), float("inf")
    t = s.clone()
    t[5, 2] = float("nan")
    y = nts.gemv_groupscaled(b, w, t, out_dtype=torch.float32)
    assert torch.all(y[3].isnan()) and not y[34].isfinite().any() and torch.all(y[:, 5].isnan())
    keep_m = [i for i in range(M) if i not in (3, 34)]
    keep_n = [i for i in range(N) if i != 5]
    assert torch.equal(y[keep_m][:, keep_n], want[keep_m][:, keep_n])
    nts.check_status()


@pytest.mark.parametrize("fmt", ["e2m1", "int4"])
def test_far_apart_values(tiles, fmt):
    """bf16 rows over most of the type's range: they enter the products as they are."""
    M, K, N, group = 30, 1024, 50, 64
    g = torch.Generator(device=DEV).manual_seed(5)
    w, s = weights(N, K, group, fmt, g)
    a = torch.randn(M, K, generator=g, device=DEV)
    a = a * 2.0 ** torch.randint(-60, 60, (M, K), generator=g, device=DEV).double()
    a[:, 128:256] = 0
    a[:, 256:384] *= 2.0 ** -60
    a[0, 512:640] = 2.0 ** -133
    a[0, 640:768] = 2.0 ** 116
    a = a.to(torch.bfloat16)
    y = nts.gemv_groupscaled(a, w, s, group=group, fmt=fmt, out_dtype=torch.float32)
    nts.check_status()
    check(y, *formula(a, None, w, s, group, fmt))


def test_equal_calls_streams_and_graphs(tiles):
    """Beside each other on streams and threads, with the other product that holds tensor
    memory between them, and captured: always the same bits."""
    g = torch.Generator(device=DEV).manual_seed(7)
    calls = []
    for M, N, K, group, act in ((32, 3001, 5120, 32, "bf16"), (20, 640, 2048, 64, "e4m3"),
                                (64, 2000, 4096, 32, "e4m3"), (17, 128, 16384, 128, "bf16")):
        a, sa = rows(M, K, act, g)
        w, s = weights(N, K, group, "int4", g)
        calls.append(lambda a=a, w=w, s=s, sa=sa, group=group: nts.gemv_groupscaled(
            a, w, s, sa, group=group, fmt="int4"))
    x = torch.randn(16, 4096, generator=g, device=DEV).to(torch.bfloat16)
    o = nts.blockcast(x)
    W = nts.blockcast(torch.randn(2048, 4096, generator=g, device=DEV).to(torch.bfloat16))
    calls.append(lambda: nts.gemm_blockscaled(o.codes, o.scales, W.codes, W.scales))
    want = [c() for c in calls]
    torch.cuda.synchronize()
    bad = []

    def run(k):
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            for i in range(60):
                j = (i + k) % len(calls)
                if not torch.equal(calls[j](), want[j]):
                    bad.append((k, i))
        stream.synchronize()

    threads = [threading.Thread(target=run, args=(k,)) for k in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = [c() for c in calls * 5]
    for _ in range(20):
        for y in got:
            y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(y, want[i % len(calls)]) for i, y in enumerate(got))
    nts.check_status()


def test_missing_copy_times_out_and_the_context_lives(tiles):
    g = torch.Generator(device=DEV).manual_seed(8)
    a, _ = rows(32, 1024, "bf16", g)
    w, s = weights(512, 1024, 32, "e2m1", g)
    want = nts.gemv_groupscaled(a, w, s)
    nts.check_status()
    nts.set_wait_limit_ns(20_000_000)
    nts.set_missing_tx(16)
    try:
        nts.gemv_groupscaled(a, w, s)
        with pytest.raises(nts.NtsError, match="TIMEOUT"):
            nts.check_status()
    finally:
        nts.set_missing_tx(0)
        nts.set_wait_limit_ns(0)
    assert torch.equal(nts.gemv_groupscaled(a, w, s), want)
    nts.check_status()
