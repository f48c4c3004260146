"""The operators beside the projection's, run together as a layer uses them --
a decode step on 4-bit weights, a training step on 8-bit products -- and called
from several threads, on other streams than the current one, in graphs, and right
behind launches that write what they read."""
import threading

import pytest
import torch

import block_reference as ref

pytestmark = pytest.mark.gpu

nts = pytest.importorskip("normalization_token_split_gb300")
DEV = "cuda:0"
EPS = 1e-6
D, HQ, HK, HD, FF = 1024, 8, 2, 128, 2048
AXES = nts.rope_axes((16, 24, 24))


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV)


def grid_positions(T):
    i = torch.arange(T, device=DEV)
    return torch.stack((i // 16, i // 4 % 4, i % 4), -1)


def close(got, want, room):
    if got.dtype is torch.bfloat16:
        room = ref.UBF16 * want.abs() + (1 + ref.UBF16) * room + 2.0 ** -133
    assert torch.all((got.double() - want).abs() <= room + 2.0 ** -126)


def check_addnorm(x, r, gamma, o):
    h = (x.float() + r.float()).to(r.dtype)
    assert torch.equal(o.h, h)
    rinv = (h.double().square().mean(1) + EPS).rsqrt()
    assert torch.all((o.rinv.double() - rinv).abs() <= (h.shape[1] / 2 + 4) * ref.U32 * rinv)
    w = (h.float() * gamma * o.rinv[:, None]).cpu()
    scales = ref.block_scales(w, 1)
    assert torch.equal(o.scales.cpu(), scales)
    assert torch.equal(o.codes.cpu(), ref.block_codes(w, scales, 1))


E2M1 = [0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6]


def four_bit(W, group):
    c = torch.stack((W.codes & 15, W.codes >> 4), -1).flatten(1).long()
    v = torch.tensor(E2M1, device=DEV, dtype=torch.float64)[c]
    return v * W.scales.double().repeat_interleave(group, 1)[:, :v.shape[1]]


def check_gemv(y, a, sa, W, group):
    A = a.double() if sa is None else ref.e4m3(a) * sa.double().repeat_interleave(128, 1)[:, :a.shape[1]]
    w = four_bit(W, group)
    # sums as counted in the operator's own tests; the inputs lie within 2^31 of each other
    close(y, A @ w.t(), 300 * ref.U32 * (A.abs() @ w.abs().t()))


def check_axes(y, x, gamma, pos, table):
    c = torch.tensor(list(AXES))
    p = pos.cpu()
    keep = (p >= 0).all(1)
    i = torch.arange(len(c))
    rows = p.clamp_min(0)[:, c]
    t = table.cpu()
    tab = torch.cat((t[rows, i], t[rows, len(c) + i]), 1)
    want, _, bound = ref.rope_forward(x.cpu(), gamma.cpu(), torch.where(keep, torch.arange(len(p)), -1),
                                      tab, HD, EPS, False)
    assert torch.all((y.cpu().double() - want).abs() <= bound)


@pytest.mark.parametrize("T", [1, 5, 24])
@pytest.mark.parametrize("res", [torch.bfloat16, torch.float32])
def test_decode_steps_of_a_layer(T, res):
    g = gen(T)
    qkv_n = (HQ + 2 * HK) * HD
    W = {n: nts.groupcast((randn(g, *s) * s[1] ** -0.5).to(torch.bfloat16), group=gr)
         for n, s, gr in (("qkv", (qkv_n, D), 32), ("o", (D, HQ * HD), 64), ("up", (FF, D), 128),
                          ("down", (D, FF), 32))}
    gain = {n: 1 + 0.1 * randn(g, D) for n in ("a", "f")}
    gq, gk = 1 + 0.1 * randn(g, HD), 1 + 0.1 * randn(g, HD)
    table, pos = nts.rope_table(64, HD), grid_positions(T)
    pos[T // 2] = -1 if T > 1 else pos[0]
    x, r = randn(g, T, D).to(torch.bfloat16), randn(g, T, D).to(res)
    for _ in range(3):
        before = r.clone()
        n = nts.add_rmsnorm_blockcast(x, r, gain["a"], out=r, want_rinv=True)
        qkv = nts.gemv_groupscaled(n.codes, *W["qkv"], a_scales=n.scales)
        q, k = qkv[:, :HQ * HD], qkv[:, HQ * HD:(HQ + HK) * HD]
        yq, yk, _, _ = nts.qknorm_rope_axes(q, gq, k, gk, pos, table, AXES, head_dim=HD)
        o = nts.gemv_groupscaled(yq, *W["o"], group=64)       # stands for what attends
        m = nts.add_rmsnorm_blockcast(o, r, gain["f"], want_rinv=True)
        up = nts.gemv_groupscaled(m.codes, *W["up"], a_scales=m.scales, group=128)
        down = nts.gemv_groupscaled(up, *W["down"])
        nts.check_status()
        check_addnorm(x, before, gain["a"], n)
        check_gemv(qkv, n.codes, n.scales, W["qkv"], 32)
        check_axes(yq, q, gq, pos, table)
        check_axes(yk, k, gk, pos, table)
        check_gemv(o, yq, None, W["o"], 64)
        check_addnorm(o, r, gain["f"], m)
        check_gemv(up, m.codes, m.scales, W["up"], 128)
        check_gemv(down, up, None, W["down"], 32)
        x, r = down, m.h


@pytest.mark.parametrize("res", [torch.bfloat16, torch.float32])
def test_training_step_of_a_layer(res):
    """Residual, norm and cast, 8-bit projection, rotation, and all of it back."""
    T = 200
    g = gen(3)
    N = (HQ + HK) * HD
    w = (randn(g, N, D) * D ** -0.5).to(torch.bfloat16)
    W, Wt = nts.blockcast(w, block_rows=128), nts.blockcast(w.t().contiguous(), block_rows=128)
    gain, gq, gk = 1 + 0.1 * randn(g, D), 1 + 0.1 * randn(g, HD), 1 + 0.1 * randn(g, HD)
    table, pos = nts.rope_table(64, HD), grid_positions(T)
    pos[T - 9:] = -1
    x, r = randn(g, T, D).to(torch.bfloat16), randn(g, T, D).to(res)
    n = nts.add_rmsnorm_blockcast(x, r, gain, want_rinv=True)
    y = nts.gemm_blockscaled(n.codes, n.scales, W.codes, W.scales)
    q, k = y[:, :HQ * HD], y[:, HQ * HD:]
    yq, yk, _, _ = nts.qknorm_rope_axes(q, gq, k, gk, pos, table, AXES, head_dim=HD)
    dyq, dyk = randn(g, T, HQ * HD).to(torch.bfloat16), randn(g, T, HK * HD).to(torch.bfloat16)
    dy = torch.empty_like(y)
    _, _, dgq, dgk = nts.qknorm_rope_axes_backward(
        dyq, dyk, q, gq, k, gk, pos, table, AXES, head_dim=HD, out_dq=dy[:, :HQ * HD],
        out_dk=dy[:, HQ * HD:])
    dY = nts.blockcast(dy)
    dn = nts.gemm_blockscaled(dY.codes, dY.scales, Wt.codes, Wt.scales)
    behind = randn(g, T, D).to(res)
    dres, dx, dgain = nts.add_rmsnorm_backward(dn, n.h, n.rinv, gain, dres=behind)
    nts.check_status()
    check_addnorm(x, r, gain, n)
    check_axes(yq, q, gq, pos, table)
    # the whole chain in fp64 from the products' outputs on: the gradient along a direction
    # of the stream, against differences, is off by the 8-bit casts' roundings alone
    u = torch.randn(T, D, generator=gen(4), device=DEV, dtype=torch.float64)

    def value(s):
        h = n.h.double() + s * u
        v = h * (h.square().mean(1, keepdim=True) + EPS).rsqrt() * gain.double()
        return (v * dn.double()).sum() + (h * behind.double()).sum()

    step = 1e-5
    want = (value(step) - value(-step)) / (2 * step)
    got = dres if dx is None else dx
    mag = (got.double() * u).abs().sum()
    assert abs((got.double() * u).sum() - want) <= (2.0 ** -8 + (D + 32) * ref.U32) * mag + 1e-6 * mag
    for dg, dyv, xv, gm in ((dgq, dyq, q, gq), (dgk, dyk, k, gk)):
        c = torch.tensor(list(AXES))
        keep = (pos >= 0).all(1).cpu()
        rows, i, t = pos.cpu().clamp_min(0)[:, c], torch.arange(len(c)), table.cpu()
        tab = torch.cat((t[rows, i], t[rows, len(c) + i]), 1)
        _, wg, _, bg = ref.rope_backward(dyv.cpu(), xv.cpu(), gm.cpu(),
                                         torch.where(keep, torch.arange(T), -1), tab, HD, EPS, False)
        assert torch.all((dg.cpu().double() - wg).abs() <= bg)
    assert torch.isfinite(dgain).all()


def everything(seed, stream=None):
    """One run of all the operators; its tensors."""
    g = gen(seed)
    t, dim, hd = 90 + 70 * seed, 512 + 16 * seed, 64
    x, r = randn(g, t, dim).to(torch.bfloat16), randn(g, t, dim).to((torch.float32, torch.bfloat16)[seed % 2])
    gamma, gq = 1 + 0.1 * randn(g, dim), 1 + 0.1 * randn(g, hd)
    w = torch.randint(0, 256, (8 * hd, 256), generator=g, device=DEV, dtype=torch.uint8)
    s = torch.rand(8 * hd, 16, generator=g, device=DEV).to(torch.bfloat16)
    a = randn(g, 3 + 5 * seed, 512).to(torch.bfloat16)
    q, k = randn(g, t, 6 * hd).to(torch.bfloat16), randn(g, t, 2 * hd).to(torch.bfloat16)
    axes, pos, table = nts.rope_axes((8, 12, 12), cyclic=True), grid_positions(t), nts.rope_table(64, hd)
    torch.cuda.current_stream().synchronize()

    def run():
        n = nts.add_rmsnorm_blockcast(x, r, gamma, want_rinv=True, stream=stream)
        b = nts.add_rmsnorm_backward(x, n.h, n.rinv, gamma, dres=n.h, stream=stream)
        y = nts.gemv_groupscaled(a, w, s, fmt=("e2m1", "int4")[seed % 2], stream=stream)
        rot = nts.qknorm_rope_axes(q, gq, k, gq, pos, table, axes, head_dim=hd, stream=stream)
        back = nts.qknorm_rope_axes_backward(rot[0], rot[1], q, gq, k, gq, pos, table, axes, head_dim=hd,
                                             stream=stream)
        return [v for v in (*n, *b, y, *rot, *back) if v is not None]
    return run


def same(a, b):
    return len(a) == len(b) and all(torch.equal(x, y) for x, y in zip(a, b))


def test_threads_on_streams_of_their_own():
    want = [everything(i)() for i in range(4)]
    torch.cuda.synchronize()
    errors = []

    def work(i):
        try:
            s = torch.cuda.Stream()
            with torch.cuda.stream(s):
                run = everything(i)
                for _ in range(30):
                    got = run()
                s.synchronize()
                assert same(got, want[i])
        except BaseException as e:   # reported by the main thread
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors[0]
    nts.check_status()


def test_what_a_call_makes_belongs_to_its_stream():
    s = torch.cuda.Stream()
    run, here = everything(1, stream=s), everything(1)
    want = here()
    torch.cuda.synchronize()
    for _ in range(20):
        got = run()
        del got
        junk = [torch.full((1 << 18,), 255, dtype=torch.uint8, device=DEV) for _ in range(8)]
        got = run()
        del junk
    s.synchronize()
    assert same(got, want)
    nts.check_status()


def test_two_graphs_replayed_at_once_beside_eager_calls():
    runs = [everything(i) for i in range(3)]
    want = [r() for r in runs]
    graphs, caps = [], []
    for r in runs[:2]:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            caps.append(r())
        graphs.append(graph)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(20):
        for graph, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                graph.replay()
        eager = runs[2]()
    torch.cuda.synchronize()
    for got, w in zip(caps + [eager], want):
        assert same(got, w)
    nts.check_status()


class Handle:
    def __init__(self, handle):
        self.cuda_stream = handle


def test_the_per_thread_stream():
    """It has no pool of torch's: the workspace is the caller's, and beside a side stream
    the outputs too."""
    g = gen(5)
    x, r, gm = randn(g, 40, 256).to(torch.bfloat16), randn(g, 40, 256), 1 + 0.1 * randn(g, 256)
    want = nts.add_rmsnorm_blockcast(x, r, gm, want_rinv=True)
    back = nts.add_rmsnorm_backward(x, want.h, want.rinv, gm)
    w = torch.randint(0, 256, (48, 128), generator=g, device=DEV, dtype=torch.uint8)
    s = torch.ones(48, 8, dtype=torch.bfloat16, device=DEV)
    y = nts.gemv_groupscaled(x[:3].contiguous(), w, s)
    torch.cuda.synchronize()
    per_thread = Handle(2)
    with pytest.raises(ValueError, match="workspace is needed"):
        nts.add_rmsnorm_backward(x, want.h, want.rinv, gm, stream=per_thread)
    ws = torch.empty(nts.add_rmsnorm_backward_workspace(256), dtype=torch.uint8, device=DEV)
    got = nts.add_rmsnorm_backward(x, want.h, want.rinv, gm, workspace=ws, stream=per_thread)
    other = nts.add_rmsnorm_blockcast(x, r, gm, want_rinv=True, stream=per_thread)
    z = nts.gemv_groupscaled(x[:3].contiguous(), w, s, stream=per_thread)
    torch.cuda.synchronize()
    assert same(got, back) and same(other, want) and torch.equal(z, y)
    with torch.cuda.stream(torch.cuda.Stream()):
        for name, fn in (("out", lambda: nts.add_rmsnorm_blockcast(x, r, gm, stream=per_thread)),
                         ("out", lambda: nts.gemv_groupscaled(x, w, s, stream=per_thread)),
                         ("out_x", lambda: nts.add_rmsnorm_backward(
                             x, want.h, want.rinv, gm, out=torch.empty_like(r), workspace=ws,
                             stream=per_thread))):
            with pytest.raises(ValueError, match=f"{name} is needed on the per-thread stream"):
                fn()
    torch.cuda.synchronize()
    nts.check_status()


# ------------------------------------------------ what the launch before wrote

def product_into(out, seed, K=8192):
    """A launch that writes one of two matrices into out (fp32 or bf16)."""
    g = gen(seed)
    M, N = out.shape
    a = torch.randint(0x20, 0x40, (M, K), generator=g, device=DEV).to(torch.uint8)
    w = torch.randint(0x20, 0x40, (N, K), generator=g, device=DEV).to(torch.uint8)
    sw = torch.rand(-(-N // 128), K // 128, generator=g, device=DEV)
    sa = [(i + 1) * torch.rand(M, K // 128, generator=g, device=DEV) / K for i in range(2)]
    return lambda which: nts.gemm_blockscaled(a, sa[which], w, sw, out=out)


def cast_into(codes, scales, seed, shape):
    xs = [randn(gen(seed + i), *shape).to(torch.bfloat16) for i in range(2)]
    return lambda which: nts.blockcast(xs[which], codes=codes, scales=scales)


def addnorm_pair(T, written, backward):
    g = gen(20)
    dim = 1024
    t = dict(x=randn(g, T, dim).to(torch.bfloat16), r=randn(g, T, dim), gamma=torch.rand(1, dim, device=DEV),
             e=randn(g, T, dim), rinv=torch.rand(1, T, generator=g, device=DEV))
    make = product_into(t[written], 21)
    if backward:
        ws = torch.empty(nts.add_rmsnorm_backward_workspace(dim), dtype=torch.uint8, device=DEV)
        return make, lambda: nts.add_rmsnorm_backward(t["x"], t["r"], t["rinv"].view(T), t["gamma"].view(dim),
                                                      dres=t["e"], workspace=ws)
    return make, lambda: nts.add_rmsnorm_blockcast(t["x"], t["r"], t["gamma"].view(dim), want_rinv=True)


def gemv_pair(M, written):
    g = gen(30)
    N, K = 1000, 2048
    w = torch.randint(0, 256, (N, K // 2), generator=g, device=DEV, dtype=torch.uint8)
    s = torch.rand(N, K // 32, generator=g, device=DEV).to(torch.bfloat16)
    a = randn(g, M, K).to(torch.bfloat16)
    o = nts.blockcast(a)
    if written == "a":
        return product_into(a, 31), lambda: [nts.gemv_groupscaled(a, w, s)]
    if written == "scales of w":
        return product_into(s, 32), lambda: [nts.gemv_groupscaled(a, w, s)]
    if written == "codes of w":
        return cast_into(w, torch.empty(N, K // 256, device=DEV), 33, (N, K // 2)), \
            lambda: [nts.gemv_groupscaled(a, w, s)]
    return cast_into(o.codes, o.scales, 35, (M, K)), \
        lambda: [nts.gemv_groupscaled(o.codes, w, s, a_scales=o.scales)]


def axes_pair(T, backward):
    """Positions, each first byte a code of the cast (a block's scale is 1)."""
    g = gen(40)
    hd, P = 128, 128
    q, k = randn(g, T, 4 * hd).to(torch.bfloat16), randn(g, T, 2 * hd).to(torch.bfloat16)
    gain, table, axes = torch.ones(hd, device=DEV), nts.rope_table(P, hd), nts.rope_axes((32, 32))
    pos = torch.zeros(T, 2, dtype=torch.int64, device=DEV)
    xs = []
    for which in range(2):
        c = torch.zeros(2 * T, 8, dtype=torch.uint8, device=DEV)
        c[:, 0] = ((7 * torch.arange(2 * T, device=DEV) + which) % 100).to(torch.uint8)
        c[15::16, 0] = 0x7E
        xs.append(c.view(-1, 128).view(torch.float8_e4m3fn).to(torch.bfloat16))
    codes = pos.view(torch.uint8).view(-1, 128)
    scales = torch.empty(len(codes), 1, device=DEV)
    make = lambda which: nts.blockcast(xs[which], codes=codes, scales=scales)  # noqa: E731
    if backward:
        ws = torch.empty(nts.rope_backward_workspace(hd), dtype=torch.uint8, device=DEV)
        return make, lambda: nts.qknorm_rope_axes_backward(q, k, q, gain, k, gain, pos, table, axes, hd,
                                                           workspace=ws)
    return make, lambda: nts.qknorm_rope_axes(q, gain, k, gain, pos, table, axes, hd)


PAIRS = {f"addition {w} T={T} backward={b}": (lambda T=T, w=w, b=b: addnorm_pair(T, w, b))
         for T in (4, 3000) for b, ws in ((False, ("x", "r", "gamma")),
                                          (True, ("x", "r", "gamma", "e", "rinv"))) for w in ws}
PAIRS.update({f"product {w} M={M}": (lambda M=M, w=w: gemv_pair(M, w))
              for M in (1, 12, 40) for w in ("a", "codes of a", "scales of w", "codes of w")})
PAIRS.update({f"axes T={T} backward={b}": (lambda T=T, b=b: axes_pair(T, b))
              for T in (16, 3008) for b in (False, True)})


def tensors(r):
    return [t for t in r if t is not None]


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
        assert same(g, want[i % 2])
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
        assert same(g, want[i % 2])
    nts.check_status()
