"""Programmatic dependent launches of the operators around a projection: what a
kernel reads -- gains, tables, positions, codes and scales as much as rows -- may
have been written by the launch just before it, which may still run when it
starts.  Each producer below writes one of two values into the same memory, in
turn, late in a launch of a few microseconds; a consumer that read too early
would show the other value."""
import pytest
import torch

pytestmark = pytest.mark.gpu

nts = pytest.importorskip("normalization_token_split_gb300")
DEV = "cuda:0"


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def product_into(out, seed, K=8192):
    """A launch that writes one of two matrices into out (fp32)."""
    g = gen(seed)
    M, N = out.shape
    a = torch.randint(0x20, 0x40, (M, K), generator=g, device=DEV).to(torch.uint8)
    w = torch.randint(0x20, 0x40, (N, K), generator=g, device=DEV).to(torch.uint8)
    sw = torch.rand(-(-N // 128), K // 128, generator=g, device=DEV)
    sa = [(i + 1) * torch.rand(M, K // 128, generator=g, device=DEV) / K for i in range(2)]
    return lambda which: nts.gemm_blockscaled(a, sa[which], w, sw, out=out)


def cast_into(codes, scales, xs, **kw):
    return lambda which: nts.blockcast(xs[which], codes=codes, scales=scales, **kw)


def bf16(seed, *shape):
    return torch.randn(*shape, generator=gen(seed), device=DEV).to(torch.bfloat16)


def norm_gain(T):
    D = 4096
    gain, x = torch.empty(1, D, device=DEV), bf16(1, T, D)
    return product_into(gain, 2), lambda: nts.rmsnorm_blockcast(x, gain.view(D), want_rinv=True)


def positions_into(pos):
    """Positions are codes of the cast: each int64's first byte one of 0 .. 126, the
    others zero, and in each block of 16 positions the code of 448, so that the
    block's scale is 1 and the cast gives back the codes."""
    T = pos.numel()
    xs = []
    for which in range(2):
        c = torch.zeros(T, 8, dtype=torch.uint8, device=DEV)
        c[:, 0] = ((7 * torch.arange(T, device=DEV) + which) % 100).to(torch.uint8)
        c[15::16, 0] = 0x7E
        xs.append(c.view(-1, 128).view(torch.float8_e4m3fn).to(torch.bfloat16))
    codes = pos.view(torch.uint8).view(-1, 128)
    return cast_into(codes, torch.empty(len(codes), 1, device=DEV), xs)


def rope(T, written, backward):
    """A rotation or its gradient; `written`: the gains, the table or the positions."""
    d, hq, hk, P = 128, 8, 2, 128
    q, k, dq, dk = (bf16(i, T, h * d) for i, h in enumerate((hq, hk, hq, hk)))
    gain, table = torch.rand(1, d, device=DEV, generator=gen(5)), nts.rope_table(P, d)
    pos = torch.arange(T, device=DEV) % P
    ws = torch.empty(nts.rope_backward_workspace(d), dtype=torch.uint8, device=DEV)
    make = {"gains": lambda: product_into(gain, 6), "table": lambda: product_into(table, 7),
            "positions": lambda: positions_into(pos)}[written]()
    g = gain.view(d)
    if backward:
        return make, lambda: nts.qknorm_rope_backward(dq, dk, q, g, k, g, pos, table, d, workspace=ws)
    return make, lambda: nts.qknorm_rope(q, g, k, g, pos, table, d, want_rinv=True)


def product_operand(M, which):
    """The product's A or W, codes and scales, written by the cast before it."""
    N, K = 1024, 2048
    rows = 1 if which == "A" else 128
    n = M if which == "A" else N
    xs = [bf16(30 + i, n, K) * (i + 1) for i in range(2)]
    codes = torch.zeros(n, K, dtype=torch.uint8, device=DEV)
    scales = torch.zeros(-(-n // rows), K // 128, device=DEV)
    other = nts.blockcast(bf16(33, N if which == "A" else M, K), block_rows=129 - rows)
    a, w = ((codes, scales), other[:2]) if which == "A" else (other[:2], (codes, scales))
    return cast_into(codes, scales, xs, block_rows=rows), \
        lambda: [nts.gemm_blockscaled(*a, *w), nts.gemm_blockscaled(*a, *w, out_dtype=torch.float32)]


PAIRS = {f"norm gain T={T}": (lambda T=T: norm_gain(T)) for T in (4, 2000)}
PAIRS.update({f"rotation {w} T={T} backward={b}": (lambda T=T, w=w, b=b: rope(T, w, b))
              for T in (16, 3008) for w in ("gains", "table", "positions") for b in (False, True)})
PAIRS.update({f"product {w} M={M}": (lambda M=M, w=w: product_operand(M, w))
              for M in (3, 60, 300, 4000) for w in ("A", "W")})


def tensors(r):
    return [t for t in (r if isinstance(r, (list, tuple)) else [r]) if t is not None]


@pytest.mark.parametrize("name", PAIRS)
def test_a_launch_reads_what_the_launch_before_it_wrote(name):
    make, use = PAIRS[name]()
    want = []
    try:
        nts.set_pdl(False)
        for which in range(2):
            make(which)
            torch.cuda.synchronize()
            want.append([t.clone() for t in tensors(use())])
        torch.cuda.synchronize()
    finally:
        nts.set_pdl(True)
    nts.check_status()
    assert not all(torch.equal(a, b) for a, b in zip(*want))
    got = []
    for i in range(12):
        make(i % 2)
        got.append(tensors(use()))
    torch.cuda.synchronize()
    for i, g in enumerate(got):
        assert all(torch.equal(a, b) for a, b in zip(g, want[i % 2]))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = []
        for i in range(6):
            make(i % 2)
            got.append(tensors(use()))
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    for i, g in enumerate(got):
        assert all(torch.equal(a, b) for a, b in zip(g, want[i % 2]))
    nts.check_status()
