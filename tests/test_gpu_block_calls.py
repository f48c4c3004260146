"""How the operators around a projection may be called: what the binding
refuses on CUDA tensors, calls from several threads and streams, memory on
other streams than the current one, offsets beyond 32 bits, outputs of odd
widths with a scale per weight row."""
import os
import re
import subprocess
import sys
import threading

import pytest
import torch

import block_reference as ref

pytestmark = pytest.mark.gpu

nts = pytest.importorskip("normalization_token_split_gb300")
DEV = "cuda:0"
T, HQ, HK, D = 6, 4, 2, 64


def rope_args(**changed):
    g = torch.Generator(device=DEV).manual_seed(1)
    a = dict(dyq=torch.randn(T, HQ * D, generator=g, device=DEV).to(torch.bfloat16),
             dyk=torch.randn(T, HK * D, generator=g, device=DEV).to(torch.bfloat16),
             q=torch.randn(T, HQ * D, generator=g, device=DEV).to(torch.bfloat16),
             gamma_q=torch.ones(D, device=DEV),
             k=torch.randn(T, HK * D, generator=g, device=DEV).to(torch.bfloat16),
             gamma_k=torch.ones(D, device=DEV), positions=torch.arange(T, device=DEV),
             table=nts.rope_table(16, D), head_dim=D)
    a.update(changed)
    return a


def forward(**changed):
    a = rope_args(**changed)
    a.pop("dyq"), a.pop("dyk")
    return nts.qknorm_rope(**a)


def backward(**changed):
    return nts.qknorm_rope_backward(**rope_args(**changed))


def bf16(*shape):
    return torch.zeros(*shape, dtype=torch.bfloat16, device=DEV)


def f32(*shape):
    return torch.zeros(*shape, device=DEV)


@pytest.mark.parametrize("fn", [forward, backward])
def test_rope_refusals(fn):
    for changed, match in (
            (dict(q=f32(T, HQ * D)), "q must be torch.bfloat16"),
            (dict(q=bf16(T, HQ, D)), "q must be a matrix"),
            (dict(q=bf16(HQ * D, T).t()), "q must have contiguous rows"),
            (dict(q=bf16(T, HQ * D - 16)), "whole heads"),
            (dict(k=bf16(T + 1, HK * D)), "same number of tokens"),
            (dict(k=bf16(T, HK * D).cpu()), "k must be a CUDA tensor"),
            (dict(gamma_q=f32(D + 16)), "gamma_q must hold head_dim values"),
            (dict(gamma_k=bf16(D)), "gamma_k must be torch.float32"),
            (dict(gamma_k=f32(2 * D)[::2]), "gamma_k must be contiguous"),
            (dict(positions=torch.arange(T, device=DEV, dtype=torch.int32)), "must be torch.int64"),
            (dict(positions=torch.arange(T + 1, device=DEV)), "one position per token"),
            (dict(table=f32(16 * D)), "table must be a matrix"),
            (dict(table=f32(16, 2 * D)[:, :D]), "table must be contiguous"),
            (dict(head_dim=0), "whole heads")):
        with pytest.raises(ValueError, match=match):
            fn(**changed)
    with pytest.raises(nts.NtsError, match="INVALID_ARG"):
        fn(table=f32(16, D + 16))                 # turns more than a head holds
    with pytest.raises(nts.NtsError, match="UNSUPPORTED"):
        fn(table=f32(16, 24))
    with pytest.raises(nts.NtsError, match="INVALID_ARG"):
        fn(eps=-1.0)
    with pytest.raises(nts.NtsError, match="UNSUPPORTED"):
        fn(q=bf16(T, HQ * D + 4)[:, 4:])          # rows off 16 bytes
    with pytest.raises(TypeError):
        fn(head_dim="64")


def test_rope_output_refusals():
    for changed, match in ((dict(out_q=bf16(T, HQ * D + 16)), "out_q has the wrong shape"),
                           (dict(out_k=f32(T, HK * D)), "out_k must be torch.bfloat16"),
                           (dict(rinv_q=f32(T, HK)), "rinv_q has the wrong shape"),
                           (dict(rinv_k=f32(HK, T).t()), "rinv_k must be contiguous")):
        with pytest.raises(ValueError, match=match):
            forward(**changed)
    for changed, match in ((dict(dyq=bf16(T, HK * D)), "dyq has the wrong shape"),
                           (dict(out_dk=bf16(T + 1, HK * D)), "out_dk has the wrong shape"),
                           (dict(dgamma_q=f32(2 * D)), "dgamma_q has the wrong shape"),
                           (dict(workspace=f32(1 << 16)), "workspace must be torch.uint8")):
        with pytest.raises(ValueError, match=match):
            backward(**changed)
    with pytest.raises(nts.NtsError, match="INVALID_ARG.*workspace"):
        backward(workspace=torch.zeros(64, dtype=torch.uint8, device=DEV))


def test_cast_and_product_refusals():
    x = bf16(32, 256)
    u8 = torch.zeros(32, 256, dtype=torch.uint8, device=DEV)
    for fn in (nts.rmsnorm_blockcast, nts.blockcast, nts.blockcast_t):
        for bad, match in ((x.float(), "x must be torch.bfloat16"), (x.t(), "x must be contiguous"),
                           (x[0], "x must be a matrix"), (x.cpu(), "x must be a CUDA tensor")):
            with pytest.raises(ValueError, match=match):
                fn(bad)
        with pytest.raises(ValueError, match="codes has the wrong shape"):
            fn(x, codes=u8[:, :128].contiguous())
        with pytest.raises(ValueError, match="scales must be torch.float32"):
            fn(x, scales=u8)
        with pytest.raises(nts.NtsError, match="UNSUPPORTED"):
            fn(bf16(4, 24))
    with pytest.raises(ValueError, match="block_rows must be 1 or 128"):
        nts.blockcast(x, block_rows=64)
    with pytest.raises(ValueError, match="gamma must hold D values"):
        nts.rmsnorm_blockcast(x, f32(128))
    with pytest.raises(nts.NtsError, match="UNSUPPORTED"):
        nts.rmsnorm_blockcast(bf16(1, 32768 + 16))

    a, sa, w, sw = u8, f32(32, 2), torch.zeros(300, 256, dtype=torch.uint8, device=DEV), f32(3, 2)
    for args, match in (((a.float(), sa, w, sw), "a_codes must be torch.uint8"),
                        ((a, sa[:, :1].contiguous(), w, sw), "a_scales must have shape"),
                        ((a, sa, w[:, :128].contiguous(), sw), "same K"),
                        ((a, sa, w[:, :128], sw), "w_codes must be contiguous"),
                        ((a, sa, w, f32(2, 2)), "w_scales must have shape"),
                        ((a, sa, w, sw.cpu()), "w_scales must be a CUDA tensor")):
        with pytest.raises(ValueError, match=match):
            nts.gemm_blockscaled(*args)
    with pytest.raises(ValueError, match="out must be bfloat16 or float32"):
        nts.gemm_blockscaled(a, sa, w, sw, out=torch.zeros(32, 300, dtype=torch.float16, device=DEV))
    with pytest.raises(ValueError, match="out has the wrong shape"):
        nts.gemm_blockscaled(a, sa, w, sw, out=bf16(300, 32))
    with pytest.raises(ValueError):
        nts.gemm_blockscaled(a, sa, w, sw, out_dtype=torch.float16)
    with pytest.raises(nts.NtsError, match="UNSUPPORTED"):
        nts.gemm_blockscaled(a[:, :24].contiguous(), f32(32, 1), w[:, :24].contiguous(), f32(3, 1))


def everything(seed, stream=None):
    """One run of all the operators; its tensors."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    t, dim, hq, hk, d = 150 + 40 * seed, 512, 6, 2, 64
    x = torch.randn(t, dim, generator=g, device=DEV).to(torch.bfloat16)
    w = torch.randn((hq + 2 * hk) * d, dim, generator=g, device=DEV).to(torch.bfloat16)
    gq, gk = torch.rand(d, generator=g, device=DEV), torch.rand(d, generator=g, device=DEV)
    pos, table = torch.arange(t, device=DEV), nts.rope_table(t, d)
    torch.cuda.current_stream().synchronize()

    def run():
        X = nts.rmsnorm_blockcast(x, None, want_rinv=True, stream=stream)
        W = nts.blockcast(w, block_rows=128, stream=stream)
        y = nts.gemm_blockscaled(X.codes, X.scales, W.codes, W.scales, stream=stream)
        q, k = y[:, :hq * d], y[:, hq * d:(hq + hk) * d]
        yq, yk, _, _ = nts.qknorm_rope(q, gq, k, gk, pos, table, head_dim=d, stream=stream)
        back = nts.qknorm_rope_backward(yq, yk, q, gq, k, gk, pos, table, head_dim=d,
                                        stream=stream)
        Xt = nts.blockcast_t(x, stream=stream)
        return [*X, W.codes, W.scales, y, yq, yk, *back, Xt.codes, Xt.scales]
    return run


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
                assert all(torch.equal(a, b) for a, b in zip(got, want[i]))
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
    """Calls on another stream than the current one, their outputs dropped at
    once while the current stream allocates and writes."""
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
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    back = torch.cuda.current_stream()
    back.wait_stream(s)
    total = sum(t.float().nan_to_num().sum() for t in got)
    del got
    assert torch.isfinite(total)
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
        assert all(torch.equal(a, b) for a, b in zip(got, w))
    nts.check_status()


class Handle:
    def __init__(self, handle):
        self.cuda_stream = handle


def test_streams_that_torch_does_not_know():
    want = backward()
    torch.cuda.synchronize()
    per_thread = Handle(2)                        # the driver's name of that stream
    with pytest.raises(ValueError, match="workspace is needed"):
        backward(stream=per_thread)
    ws = torch.empty(nts.rope_backward_workspace(D), dtype=torch.uint8, device=DEV)
    got = backward(stream=per_thread, workspace=ws)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    got = backward(stream=Handle(0))              # the default stream
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    with pytest.raises(AttributeError):
        backward(stream=2)
    nts.check_status()


@pytest.mark.parametrize("ring", [False, True])
def test_rope_rows_beyond_32_bit_offsets(ring):
    n, ld = 20, 1 << 27                           # 20 rows 256 MB apart
    pos, table = torch.arange(n, device=DEV), nts.rope_table(n, D)
    ones = torch.ones(D, device=DEV)

    def far(width):
        buf = torch.empty((n - 1) * ld + width, dtype=torch.bfloat16, device=DEV)
        return buf.as_strided((n, width), (ld, 1))

    q, k, dyq, dyk = far(HQ * D), far(HK * D), far(HQ * D), far(HK * D)
    g = torch.Generator(device=DEV).manual_seed(5)
    near = [torch.randn(n, t.shape[1], generator=g, device=DEV).to(torch.bfloat16)
            for t in (q, k, dyq, dyk)]
    for t, v in zip((q, k, dyq, dyk), near):
        t.copy_(v)
    a = (pos, table, D)
    y = nts.qknorm_rope(near[0], ones, near[1], ones, *a)
    b = nts.qknorm_rope_backward(near[2], near[3], near[0], ones, near[1], ones, *a)
    try:
        if ring:
            nts.set_tuning(rows=1, stages=2)
        nts.qknorm_rope_backward(dyq, dyk, q, ones, k, ones, *a, out_dq=dyq, out_dk=dyk)
        nts.qknorm_rope(q, ones, k, ones, *a, out_q=q, out_k=k)
        nts.check_status()
    finally:
        nts.set_tuning()
    for t, v in zip((q, k, dyq, dyk), (y[0], y[1], b[0], b[1])):
        assert torch.equal(t, v)


def test_casts_beyond_32_bit_offsets():
    n, dim = 66000, 32768                         # 2.2e9 values
    g = torch.Generator(device=DEV).manual_seed(6)
    x = torch.randn(1000, dim, generator=g, device=DEV).to(torch.bfloat16).repeat(66, 1)
    x[-1] *= 3
    o, tail = nts.blockcast(x), nts.blockcast(x[-100:].contiguous())
    assert torch.equal(o.codes[-100:], tail.codes) and torch.equal(o.scales[-100:], tail.scales)
    del o
    # calls of other lengths may sum a row in another order: by the formula, from rinv on
    o = nts.rmsnorm_blockcast(x, want_rinv=True)
    last, rinv = x[-100:].cpu(), o.rinv[-100:].cpu()
    want = (last.double().square().mean(1) + 1e-6).rsqrt()
    assert torch.all((rinv.double() - want).abs() <= (dim / 2 + 4) * ref.U32 * want)
    w = last.float() * rinv[:, None]
    scales = ref.block_scales(w, 1)
    assert torch.equal(o.scales[-100:].cpu(), scales)
    assert torch.equal(o.codes[-100:].cpu(), ref.block_codes(w, scales, 1))
    del o
    o, tail = nts.blockcast(x, block_rows=128), nts.blockcast(x[-80:].contiguous(), block_rows=128)
    assert n % 128 == 80
    assert torch.equal(o.codes[-80:], tail.codes) and torch.equal(o.scales[-1:], tail.scales)
    del o
    o, tail = nts.blockcast_t(x), nts.blockcast_t(x[:, -16:].contiguous())
    assert torch.equal(o.codes[-16:], tail.codes) and torch.equal(o.scales[-16:], tail.scales)
    nts.check_status()


@pytest.mark.parametrize("rows", [128, 1])
def test_product_beyond_32_bit_offsets(rows):
    M, N, K = 66000, 33001, 16                    # 2.2e9 outputs, rows off 32 bytes
    g = torch.Generator(device=DEV).manual_seed(7)
    a = torch.randint(0, 127, (M, K), generator=g, device=DEV).to(torch.uint8)
    w = torch.randint(0, 127, (N, K), generator=g, device=DEV).to(torch.uint8)
    sa = torch.rand(M, 1, generator=g, device=DEV)
    sw = torch.rand(-(-N // rows), 1, generator=g, device=DEV)
    y = nts.gemm_blockscaled(a, sa, w, sw)
    nts.check_status()
    want, mag = ref.gemm(a[-40:], sa[-40:], w, sw, rows)
    assert torch.all((y[-40:].double() - want).abs() <= ref.gemm_bound(want, mag, K, False))


@pytest.mark.parametrize("M,N,K", [(1, 130, 144), (70, 515, 272), (131, 257, 400), (300, 264, 272),
                                   (1100, 4999, 144), (1100, 5000, 144)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("kernel", [0, 1, 2, 3])
def test_outputs_with_a_scale_per_weight_row_stay_in_bounds(M, N, K, dtype, kernel):
    pad = 4096
    g = torch.Generator(device=DEV).manual_seed(M + N)
    a = torch.randint(0, 127, (M, K), generator=g, device=DEV).to(torch.uint8)
    w = torch.randint(0, 127, (N, K), generator=g, device=DEV).to(torch.uint8)
    sa = torch.rand(M, -(-K // 128), generator=g, device=DEV)
    sw = torch.rand(N, -(-K // 128), generator=g, device=DEV)
    n = M * N * torch.tensor([], dtype=dtype).element_size()
    buf = torch.full((2 * pad + n,), 0xA5, dtype=torch.uint8, device=DEV)
    out = buf[pad:pad + n].view(dtype).view(M, N)
    try:
        nts.set_tuning(vpt=kernel)
        nts.gemm_blockscaled(a, sa, w, sw, out=out)
        nts.check_status()
    finally:
        nts.set_tuning()
    assert bool((buf[:pad] == 0xA5).all()) and bool((buf[-pad:] == 0xA5).all())
    want, mag = ref.gemm(a, sa, w, sw, 1)
    assert torch.all((out.double() - want).abs()
                     <= ref.gemm_bound(want, mag, K, dtype == torch.float32))


def test_far_positions_at_the_ends_of_their_type():
    """Padding is any negative position; any other one beyond the table is reported."""
    low, high = -(1 << 63), (1 << 63) - 1
    pos = torch.tensor([0, low, -1, 3, 15, 2], device=DEV)
    y, k, rq, _ = forward(positions=pos, want_rinv=True)
    nts.check_status()
    assert not y[1:3].any() and not k[1:3].any() and not rq[1:3].any()
    pos[3] = high
    y, _, _, _ = forward(positions=pos)
    with pytest.raises(nts.NtsError, match="rotation table"):
        nts.check_status()
    assert not y[3].any() and y[4].any()


@pytest.mark.parametrize("kernel", [1, 2, 3])
@pytest.mark.parametrize("rows", [128, 1])
def test_a_copy_that_never_lands_ends_a_long_product(kernel, rows):
    """More K blocks than the ring has stages: what gave up issues nothing more."""
    g = torch.Generator(device=DEV).manual_seed(8)
    M, N, K = 600, 520, 2048
    a = torch.randint(0, 127, (M, K), generator=g, device=DEV).to(torch.uint8)
    w = torch.randint(0, 127, (N, K), generator=g, device=DEV).to(torch.uint8)
    sa = torch.rand(M, K // 128, generator=g, device=DEV)
    sw = torch.rand(-(-N // rows), K // 128, generator=g, device=DEV)
    try:
        nts.set_tuning(vpt=kernel)
        want = nts.gemm_blockscaled(a, sa, w, sw)
        nts.check_status()
        nts.set_wait_limit_ns(20_000_000)
        nts.set_missing_tx(16)
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


def test_outputs_on_the_per_thread_stream_beside_a_side_stream():
    """A side stream does not wait for the per-thread stream, nor that one for it:
    memory of the side stream's pool is not the call's to write."""
    x = bf16(4, 256)
    u8, s = torch.zeros(4, 256, dtype=torch.uint8, device=DEV), f32(4, 2)
    ws = torch.empty(nts.rope_backward_workspace(D), dtype=torch.uint8, device=DEV)
    want = [t.clone() for t in backward()]
    outs = dict(out_dq=bf16(T, HQ * D), out_dk=bf16(T, HK * D), dgamma_q=f32(D), dgamma_k=f32(D))
    a = rope_args()
    torch.cuda.synchronize()
    per_thread = Handle(2)
    calls = {"out_q": lambda **k: forward(stream=per_thread, **k),
             "codes": lambda **k: nts.blockcast(x, stream=per_thread, **k),
             "out": lambda **k: nts.gemm_blockscaled(u8, s, u8, s[:1], stream=per_thread, **k)}
    for fn in (nts.rmsnorm_blockcast, nts.blockcast_t):
        with torch.cuda.stream(torch.cuda.Stream()), pytest.raises(ValueError, match="codes is needed"):
            fn(x, stream=per_thread)
    for name, fn in calls.items():
        fn()                                      # the default stream waits for it, and it for that
        with torch.cuda.stream(torch.cuda.Stream()), \
                pytest.raises(ValueError, match=f"{name} is needed on the per-thread stream"):
            fn()
    with torch.cuda.stream(torch.cuda.Stream()):
        for name in outs:
            some = {k: v for k, v in outs.items() if k != name}
            with pytest.raises(ValueError, match=f"{name} is needed on the per-thread stream"):
                nts.qknorm_rope_backward(**a, workspace=ws, stream=per_thread, **some)
        got = nts.qknorm_rope_backward(**a, workspace=ws, stream=per_thread, **outs)
    torch.cuda.synchronize()
    assert all(torch.equal(g, w) for g, w in zip(got, want))
    nts.check_status()


def test_the_legacy_handle_is_the_default_stream():
    """What a call on it makes comes from the default stream's pool, a workspace too."""
    want = [t.clone() for t in backward()]
    a = rope_args()
    torch.cuda.synchronize()
    legacy = Handle(1)
    got = nts.qknorm_rope_backward(**a, stream=legacy)
    torch.cuda.synchronize()
    assert all(torch.equal(g, w) for g, w in zip(got, want))
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = nts.qknorm_rope_backward(**a, stream=legacy)
        held = {b["address"] for seg in torch.cuda.memory_snapshot()
                if seg["stream"] == side.cuda_stream for b in seg["blocks"]
                if b["state"] == "active_allocated"}
        assert not held & {t.data_ptr() for t in got}
    torch.cuda.synchronize()
    assert all(torch.equal(g, w) for g, w in zip(got, want))
    nts.check_status()


STATUS_RUN = """
import torch
import normalization_token_split_gb300 as nts
x = torch.ones(4, 256, dtype=torch.bfloat16, device="cuda")
g, pos = torch.ones(64, device="cuda"), torch.arange(4, device="cuda")
table = nts.rope_table(4, 64)
nts.rmsnorm_mxcast(x)
nts.check_status()                                # 0
o = nts.blockcast(x)
nts.check_status()                                # 1
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    nts.qknorm_rope(x, g, x, g, pos, table, 64)
pos.fill_(9)
graph.replay()
try:
    nts.check_status()                            # 2: a captured launch counts
except nts.NtsError as e:
    assert "rotation table" in str(e)
else:
    raise SystemExit("the position went unseen")
nts.gemm_blockscaled(o.codes, o.scales, o.codes, o.scales)
nts.check_status()                                # 3
"""


def test_check_status_reads_the_words_of_what_ran():
    """Users of the other operators do not wait for copies of these ones' words."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", STATUS_RUN], cwd=root, capture_output=True, text=True,
                       env={**os.environ, "NTS_LOG": "1"}, timeout=300)
    assert r.returncode == 0, r.stderr
    assert re.findall(r"words of (\d+) operators", r.stderr) == ["0", "1", "2", "3"]
