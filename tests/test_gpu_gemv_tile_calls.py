"""Products by tiles right behind launches that write their operands, and with offsets
beyond 32 bits."""
import pytest
import torch

from test_gpu_gemv import DEV, check, formula, rows, weights
from test_gpu_layer_calls import cast_into, gen, product_into, randn, same

pytestmark = pytest.mark.gpu

nts = pytest.importorskip("normalization_token_split_gb300")


def by_tiles(a, w, s, sa=None):
    nts.set_tuning(vpt=2)                         # not of the launch that writes an operand
    try:
        return [nts.gemv_groupscaled(a, w, s, a_scales=sa, out_dtype=torch.float32)]
    finally:
        nts.set_tuning()


def pair(M, N, K, written):
    """(a launch that writes one operand, the product that reads it)."""
    g = gen(30)
    w = torch.randint(0, 256, (N, K // 2), generator=g, device=DEV, dtype=torch.uint8)
    s = torch.rand(N, K // 32, generator=g, device=DEV).to(torch.bfloat16)
    a = randn(g, M, K).to(torch.bfloat16)
    o = nts.blockcast(a)
    if written == "a":
        return product_into(a, 31), lambda: by_tiles(a, w, s)
    if written == "scales of w":
        return product_into(s, 32), lambda: by_tiles(a, w, s)
    if written == "codes of w":
        return cast_into(w, torch.empty(N, K // 256, device=DEV), 33, (N, K // 2)), \
            lambda: by_tiles(a, w, s)
    if written == "codes of a":
        return cast_into(o.codes, o.scales, 35, (M, K)), lambda: by_tiles(o.codes, w, s, o.scales)
    return product_into(o.scales, 36), lambda: by_tiles(o.codes, w, s, o.scales)


# One CTA to a tile where tiles fill the GPU, a cluster where they do not.
@pytest.mark.parametrize("N,K", [(20000, 256), (1000, 2048)])
@pytest.mark.parametrize("M", [17, 40])
@pytest.mark.parametrize("written", ["a", "codes of a", "scales of a", "scales of w", "codes of w"])
def test_a_tile_reads_what_the_launch_before_it_wrote(written, M, N, K):
    make, use = pair(M, N, K, written)
    want = []
    try:
        nts.set_pdl(False)
        for which in range(2):
            make(which)
            torch.cuda.synchronize()
            want.append([t.clone() for t in use()])
        torch.cuda.synchronize()
    finally:
        nts.set_pdl(True)
    nts.check_status()
    assert not torch.equal(want[0][0], want[1][0]) and torch.isfinite(want[0][0]).all()
    got = []
    for i in range(12):
        make(i % 2)
        got.append(use())
    torch.cuda.synchronize()
    for i, g in enumerate(got):
        assert same(g, want[i % 2])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = []
        for i in range(6):
            make(i % 2)
            got.append(use())
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    for i, g in enumerate(got):
        assert same(g, want[i % 2])
    nts.check_status()


@pytest.mark.parametrize("act", ["bf16", "e4m3"])
def test_more_than_4_gb_of_codes(act):
    M, N, K = 17, 270000, 32768                   # 4.4e9 bytes, by tiles for their number
    g = torch.Generator(device=DEV).manual_seed(8)
    a, sa = rows(M, K, act, g)
    w = torch.randint(0, 256, (1000, K // 2), generator=g, device=DEV, dtype=torch.uint8).repeat(270, 1)
    w[-50:] = 255 - w[-50:]
    s = torch.rand(N, K // 128, generator=g, device=DEV).to(torch.bfloat16)
    y = nts.gemv_groupscaled(a, w, s, sa, group=128, out_dtype=torch.float32)
    nts.check_status()
    check(y[:, -60:], *formula(a, sa, w[-60:], s[-60:], 128, "e2m1"))


def test_more_than_2_31_outputs_and_rows_far_apart():
    M, N, K = 17, 134_500_000, 32                 # 2.29e9 outputs
    g = torch.Generator(device=DEV).manual_seed(9)
    a, _ = rows(M, K, "bf16", g)
    w, s = weights(1000, K, 32, "int4", g)
    y = nts.gemv_groupscaled(a, w.repeat(N // 1000, 1), s.repeat(N // 1000, 1), fmt="int4")
    nts.check_status()
    assert y.numel() > 1 << 31
    check(y[:, :1000], *formula(a, None, w, s, 32, "int4"))
    assert torch.all(y.view(M, -1, 1000) == y[:, None, :1000])
    del y
    M, K = 24, 4096
    a, _ = rows(M, K, "bf16", g)
    w, s = weights(4200, K, 32, "int4", g)
    far = torch.empty((M - 1) * (1 << 27) + K, dtype=torch.bfloat16, device=DEV)   # 6 GB
    far = far.as_strided((M, K), (1 << 27, 1))
    far.copy_(a)
    assert torch.equal(nts.gemv_groupscaled(far, w, s, fmt="int4"),
                       nts.gemv_groupscaled(a, w, s, fmt="int4"))
    nts.check_status()
