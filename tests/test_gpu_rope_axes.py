"""Headwise QK-RMSNorm with a rotation of several position axes, and its
gradient, on the GPU against the fp64 formulas, against differences, and against
the one-axis operator where the two must agree bit for bit."""
import pytest
import torch

import block_reference as ref

pytestmark = pytest.mark.gpu

nts = pytest.importorskip("normalization_token_split_gb300")
DEV = "cuda:0"
EPS = 1e-6


def pair_axes(kind, half, A, g):
    if kind == "random":
        return bytes(torch.randint(0, A, (half,), generator=g).tolist())
    rest = half // (A + 1)
    return nts.rope_axes([half - (A - 1) * rest] + [rest] * (A - 1), cyclic=kind == "cyclic")


def make(T, hq, hk, d, rot, A, kind, seed, P=500, packed=False, pad=0):
    """CPU tensors; q and k are columns of one buffer when packed, with a gap behind."""
    g = torch.Generator().manual_seed(seed)
    out = {}
    for names in (("q", "k"), ("dyq", "dyk")):
        if packed:
            buf = torch.randn(T, (hq + 2 * hk) * d + 8, generator=g).to(torch.bfloat16)
            out[names[0]], out[names[1]] = buf[:, :hq * d], buf[:, hq * d:(hq + hk) * d]
        else:
            out[names[0]] = torch.randn(T, hq * d, generator=g).to(torch.bfloat16)
            out[names[1]] = torch.randn(T, hk * d, generator=g).to(torch.bfloat16)
    out["gq"] = 1.0 + 0.1 * torch.randn(d, generator=g)
    out["gk"] = 1.0 + 0.1 * torch.randn(d, generator=g)
    out["pos"] = torch.randint(0, P, (T, A), generator=g)
    for i in range(pad):      # one axis is enough to make a padding row
        out["pos"][T - 1 - i, i % A] = -1 - i
    out["table"] = nts.rope_table(P, rot, device="cpu")
    out["axes"] = pair_axes(kind, rot // 2, A, g)
    return out


def one_axis(c):
    """Positions and a table of one axis that give the same angles: row t of the table
    holds token t's own."""
    pos, axis = c["pos"], torch.tensor(list(c["axes"]))
    half = len(axis)
    P = c["table"].shape[0]
    keep = ((pos >= 0) & (pos < P)).all(1)
    rows = pos.clamp(0, P - 1)[:, axis]
    i = torch.arange(half)
    table = torch.cat((c["table"][rows, i], c["table"][rows, half + i]), 1)
    return torch.where(keep, torch.arange(len(pos)), -1), table


def to_dev(t):
    """A copy on the device that keeps the row stride."""
    if isinstance(t, bytes):
        return t
    if t.dim() == 2 and t.shape[0] > 1 and t.stride(0) != t.shape[1]:
        buf = torch.zeros(t.shape[0], t.stride(0), dtype=t.dtype, device=DEV)
        view = buf[:, :t.shape[1]]
        view.copy_(t)
        return view
    return t.to(DEV)


def forward(c, d, il, **kw):
    D = {k: to_dev(v) for k, v in c.items()}
    return nts.qknorm_rope_axes(D["q"], D["gq"], D["k"], D["gk"], D["pos"], D["table"], D["axes"],
                                head_dim=d, eps=EPS, interleaved=il, **kw)


def backward(c, d, il, **kw):
    D = {k: to_dev(v) for k, v in c.items()}
    return nts.qknorm_rope_axes_backward(D["dyq"], D["dyk"], D["q"], D["gq"], D["k"], D["gk"],
                                         D["pos"], D["table"], D["axes"], head_dim=d, eps=EPS,
                                         interleaved=il, **kw)


SHAPES = [  # T, hq, hk, d, rot, axes, order, packed, padded rows
    (1, 1, 1, 16, 16, 2, "sections", False, 0),
    (1, 32, 32, 128, 128, 3, "sections", True, 0),
    (2, 3, 1, 32, 16, 3, "cyclic", False, 1),
    (5, 7, 7, 48, 48, 4, "random", True, 4),
    (64, 32, 8, 128, 128, 3, "cyclic", True, 3),
    (33, 20, 4, 96, 64, 2, "random", True, 8),
    (17, 5, 3, 80, 32, 1, "sections", False, 0),
    (13, 6, 2, 256, 128, 3, "random", True, 0),
    (7, 4, 4, 512, 512, 4, "sections", False, 1),
    (11, 65, 13, 160, 112, 3, "sections", True, 0),
    (700, 16, 4, 128, 64, 3, "sections", True, 100),
    (300, 40, 40, 112, 112, 3, "cyclic", False, 0),
]


def check_forward(c, d, il, got):
    pos, table = one_axis(c)
    yq, yk, rq, rk = got
    for y, r, x, g in ((yq, rq, c["q"], c["gq"]), (yk, rk, c["k"], c["gk"])):
        want, rinv, bound = ref.rope_forward(x, g, pos, table, d, EPS, il)
        assert torch.all((y.cpu().double() - want).abs() <= bound)
        if r is not None:
            assert torch.all((r.cpu().double() - rinv).abs() <= (d / 2 + 8) * ref.U32 * rinv)


def check_backward(c, d, il, got):
    pos, table = one_axis(c)
    dq, dk, dgq, dgk = got
    for dx, dg, dy, x, g in ((dq, dgq, c["dyq"], c["q"], c["gq"]),
                             (dk, dgk, c["dyk"], c["k"], c["gk"])):
        wx, wg, bx, bg = ref.rope_backward(dy, x, g, pos, table, d, EPS, il)
        assert torch.all((dx.cpu().double() - wx).abs() <= bx)
        assert torch.all((dg.cpu().double() - wg).abs() <= bg)


@pytest.mark.parametrize("il", [False, True])
@pytest.mark.parametrize("T,hq,hk,d,rot,A,kind,packed,pad", SHAPES)
def test_formulas(T, hq, hk, d, rot, A, kind, packed, pad, il):
    c = make(T, hq, hk, d, rot, A, kind, seed=T + d, packed=packed, pad=pad)
    fwd, bwd = forward(c, d, il, want_rinv=True), backward(c, d, il)
    nts.check_status()
    check_forward(c, d, il, fwd)
    check_backward(c, d, il, bwd)


@pytest.mark.parametrize("rows,stages", [(1, 2), (2, 3), (5, 1)])
@pytest.mark.parametrize("T,hq,hk,d,rot,A,kind,packed,pad", SHAPES)
def test_ring_kernels_on_any_shape(T, hq, hk, d, rot, A, kind, packed, pad, rows, stages):
    c = make(T, hq, hk, d, rot, A, kind, seed=3 * T + d, packed=packed, pad=pad)
    il = (T + d) % 2 == 0
    try:
        nts.set_tuning(rows=rows, stages=stages)
        fwd, bwd = forward(c, d, il), backward(c, d, il)
        nts.check_status()
    finally:
        nts.set_tuning()
    check_forward(c, d, il, fwd)
    check_backward(c, d, il, bwd)


@pytest.mark.parametrize("T", [3, 900])
@pytest.mark.parametrize("il", [False, True])
def test_alike_positions_are_one_axis(T, il):
    """Positions alike on all axes (text): the bits of the one-axis operator."""
    c = make(T, 16, 4, 128, 96, 3, "cyclic", seed=T, packed=True, pad=0)
    c["pos"] = c["pos"][:, :1].repeat(1, 3)
    c["pos"][T // 2] = -1
    D = {k: to_dev(v) for k, v in c.items()}
    a = (D["q"], D["gq"], D["k"], D["gk"], D["pos"][:, 0].contiguous(), D["table"])
    want = nts.qknorm_rope(*a, head_dim=128, eps=EPS, interleaved=il, want_rinv=True)
    for got, w in zip(forward(c, 128, il, want_rinv=True), want):
        assert torch.equal(got, w)
    want = nts.qknorm_rope_backward(D["dyq"], D["dyk"], *a, head_dim=128, eps=EPS, interleaved=il)
    for got, w in zip(backward(c, 128, il), want):
        assert torch.equal(got, w)


@pytest.mark.parametrize("T", [5, 800])
def test_positions_of_any_strides(T):
    c = make(T, 8, 2, 64, 64, 3, "sections", seed=T)
    D = {k: to_dev(v) for k, v in c.items()}
    a = (D["q"], D["gq"], D["k"], D["gk"])
    b = (D["table"], D["axes"])
    pos = D["pos"]
    want = nts.qknorm_rope_axes(*a, pos, *b, head_dim=64)[:2]
    wide = torch.full((T, 7), 1 << 40, device=DEV)
    wide[:, 1::2] = pos
    far = torch.full((3, 2 * T), -5, device=DEV)
    far[:, ::2] = pos.t()
    for p in (pos.t().contiguous().t(), wide[:, 1::2], far[:, ::2].t()):
        got = nts.qknorm_rope_axes(*a, p, *b, head_dim=64)[:2]
        assert all(torch.equal(x, y) for x, y in zip(got, want))
    same = pos[:, :1].expand(T, 3)                # stride 0 along the axes
    got = nts.qknorm_rope_axes(*a, same, *b, head_dim=64)[:2]
    want = nts.qknorm_rope_axes(*a, same.contiguous(), *b, head_dim=64)[:2]
    assert all(torch.equal(x, y) for x, y in zip(got, want))
    nts.check_status()


@pytest.mark.parametrize("ring", [False, True])
def test_positions_outside_the_table(ring):
    """Zeros, and a report unless another axis makes the token a padding row."""
    c = make(9, 4, 2, 64, 64, 3, "sections", seed=1, P=50)
    low, high = -(1 << 63), (1 << 63) - 1
    c["pos"][1, 2] = low
    c["pos"][2] = torch.tensor([high, 3, -1])
    try:
        if ring:
            nts.set_tuning(rows=1, stages=2)
        y = forward(c, 64, False, want_rinv=True)
        g = backward(c, 64, False)
        nts.check_status()
        for t in (*y, *g[:2]):
            assert not t[1:3].any() and t[3].any()
        for axis in range(3):
            bad = dict(c, pos=c["pos"].clone())
            bad["pos"][4, axis] = 50 if axis else high
            y = forward(bad, 64, False)
            with pytest.raises(nts.NtsError, match="rotation table"):
                nts.check_status()
            assert not y[0][4].any() and y[0][3].any()
            g = backward(bad, 64, False)
            with pytest.raises(nts.NtsError, match="rotation table"):
                nts.check_status()
            assert not g[0][4].any()
            check_backward(bad, 64, False, g)
    finally:
        nts.set_tuning()


def test_padding_rows_may_hold_anything():
    c = make(40, 4, 2, 64, 48, 2, "cyclic", seed=2, pad=7)
    for k in ("q", "k", "dyq", "dyk"):
        c[k][33:] = float("nan")
    c["table"][0] = float("inf")                  # not read for them either
    c["pos"][:33] = c["pos"][:33].clamp_min(1)
    fwd, bwd = forward(c, 64, True, want_rinv=True), backward(c, 64, True)
    nts.check_status()
    for t in (*fwd, *bwd[:2]):
        assert not t[33:].any()
    clean = {k: (torch.nan_to_num(v) if k in ("q", "k", "dyq", "dyk") else v) for k, v in c.items()}
    check_forward(clean, 64, True, fwd)
    check_backward(clean, 64, True, bwd)


def test_gradient_against_differences():
    """The kernel's dq along a direction against differences of the fp64 formula."""
    d, rot = 64, 64
    c = make(6, 3, 1, d, rot, 3, "random", seed=4)
    pos, table = one_axis(c)
    dq, _, dgq, _ = backward(c, d, False)
    g = torch.Generator().manual_seed(9)
    u = torch.randn(c["q"].shape, generator=g, dtype=torch.float64)
    v = torch.randn(d, generator=g, dtype=torch.float64)
    step = 1e-5

    def value(s):
        y, _, _ = ref.rope_forward(c["q"].double() + s * u, c["gq"].double() + s * v, pos, table, d,
                                   EPS, False)
        return (y * c["dyq"].double()).sum()

    want = (value(step) - value(-step)) / (2 * step)
    got = (dq.cpu().double() * u).sum() + (dgq.cpu().double() * v).sum()
    # bf16 roundings of dq; the differences' own error is of the order of step^2
    room = ref.UBF16 * (dq.cpu().double() * u).abs().sum() + 1e-6 * abs(want) + 1e-6
    assert abs(got - want) <= room


def test_in_place_and_untouched_gaps():
    c = make(50, 8, 2, 64, 64, 3, "sections", seed=6, packed=True, pad=5)
    D = {k: to_dev(v) for k, v in c.items()}
    a = (D["gq"], D["k"], D["gk"], D["pos"], D["table"], D["axes"])
    want = nts.qknorm_rope_axes(D["q"], *a, head_dim=64)
    qkv = D["q"]._base.clone()
    q, k = qkv[:, :512], qkv[:, 512:640]
    k.copy_(D["k"])
    gap = qkv[:, 640:].clone()
    got = nts.qknorm_rope_axes(q, D["gq"], k, *a[2:], head_dim=64, out_q=q, out_k=k)
    assert got[0].data_ptr() == q.data_ptr()
    assert torch.equal(q, want[0]) and torch.equal(k, want[1]) and torch.equal(qkv[:, 640:], gap)
    nts.check_status()


def test_empty_batch():
    c = make(1, 4, 2, 64, 64, 2, "sections", seed=7)
    for k in ("q", "k", "dyq", "dyk", "pos"):
        c[k] = c[k][:0]
    y = forward(c, 64, False)
    g = backward(c, 64, False)
    assert y[0].shape == (0, 256) and not g[2].any() and not g[3].any()
    nts.check_status()


def test_refusals():
    c = make(6, 4, 2, 64, 64, 3, "sections", seed=8)
    for changed, match in (
            (dict(axes=c["axes"][:-1]), "an axis for each pair"),
            (dict(axes=list(c["axes"])), "axes must be bytes"),
            (dict(axes=None), "axes must be bytes"),
            (dict(pos=c["pos"][:, 0]), "positions must be a matrix"),
            (dict(pos=c["pos"][:5]), "1 to 4 positions"),
            (dict(pos=c["pos"][:, :0]), "1 to 4 positions"),
            (dict(pos=torch.zeros(6, 5, dtype=torch.int64)), "1 to 4 positions"),
            (dict(pos=c["pos"].int()), "must be torch.int64"),
            (dict(q=c["q"][:5]), "same number of tokens")):
        for fn in (forward, backward):
            b = dict(c, **changed)
            D = {k: (v if not torch.is_tensor(v) else to_dev(v)) for k, v in b.items()}
            with pytest.raises(ValueError, match=match):
                if fn is forward:
                    nts.qknorm_rope_axes(D["q"], D["gq"], D["k"], D["gk"], D["pos"], D["table"],
                                         D["axes"], head_dim=64)
                else:
                    nts.qknorm_rope_axes_backward(D["dyq"][:len(b["q"])], D["dyk"], D["q"], D["gq"],
                                                  D["k"], D["gk"], D["pos"], D["table"], D["axes"],
                                                  head_dim=64)
    for fn in (forward, backward):
        with pytest.raises(nts.NtsError, match="INVALID_ARG.*axis 3 of 3"):
            fn(dict(c, axes=c["axes"][:-1] + b"\x03"), 64, False)
    nts.check_status()
