"""Headwise QK-RMSNorm with the rotary position embedding, and its gradient,
on the GPU against the fp64 formulas and against differences."""
import math

import pytest
import torch

import block_reference as ref

pytestmark = pytest.mark.gpu

nts = pytest.importorskip("normalization_token_split_gb300")
DEV = "cuda:0"
EPS = 1e-6


def make(T, hq, hk, d, rot, seed, P=4096, packed=False, pad=0, spare=0):
    """CPU tensors; q and k are columns of one buffer when packed."""
    g = torch.Generator().manual_seed(seed)
    width = (hq + 2 * hk) * d + spare if packed else None
    out = {}
    for names in (("q", "k"), ("dyq", "dyk")):
        if packed:
            buf = torch.randn(T, width, generator=g).to(torch.bfloat16)
            out[names[0]], out[names[1]] = buf[:, :hq * d], buf[:, hq * d:(hq + hk) * d]
        else:
            out[names[0]] = torch.randn(T, hq * d, generator=g).to(torch.bfloat16)
            out[names[1]] = torch.randn(T, hk * d, generator=g).to(torch.bfloat16)
    out["gq"] = 1.0 + 0.1 * torch.randn(d, generator=g)
    out["gk"] = 1.0 + 0.1 * torch.randn(d, generator=g)
    out["pos"] = torch.randint(0, P, (T,), generator=g)
    if pad:
        out["pos"][T - pad:] = -1
    out["table"] = nts.rope_table(P, rot, device="cpu")
    return out


def to_dev(t):
    """A copy on the device that keeps the row stride."""
    if t.dim() == 2 and t.shape[0] > 1 and t.stride(0) != t.shape[1]:
        buf = torch.zeros(t.shape[0], t.stride(0), dtype=t.dtype, device=DEV)
        view = buf[:, :t.shape[1]]
        view.copy_(t)
        return view
    return t.to(DEV)


def forward(c, d, il, **kw):
    D = {k: to_dev(v) for k, v in c.items()}
    return nts.qknorm_rope(D["q"], D["gq"], D["k"], D["gk"], D["pos"], D["table"], head_dim=d,
                           eps=EPS, interleaved=il, **kw)


def backward(c, d, il, **kw):
    D = {k: to_dev(v) for k, v in c.items()}
    return nts.qknorm_rope_backward(D["dyq"], D["dyk"], D["q"], D["gq"], D["k"], D["gk"],
                                    D["pos"], D["table"], head_dim=d, eps=EPS, interleaved=il, **kw)


SHAPES = [  # T, hq, hk, d, rot, packed, padded rows
    (1, 1, 1, 16, 16, False, 0),
    (1, 32, 32, 128, 128, True, 0),
    (2, 3, 1, 32, 16, False, 1),
    (5, 7, 7, 48, 48, True, 0),
    (64, 32, 8, 128, 128, True, 3),
    (33, 20, 4, 96, 64, True, 8),
    (17, 5, 3, 80, 32, False, 0),
    (19, 9, 9, 64, 64, False, 2),
    (13, 6, 2, 256, 128, True, 0),
    (7, 4, 4, 512, 512, False, 1),
    (11, 65, 13, 160, 112, True, 0),
    (700, 16, 4, 128, 64, True, 100),
    (300, 40, 40, 112, 112, False, 0),
]


@pytest.mark.parametrize("il", [False, True])
@pytest.mark.parametrize("T,hq,hk,d,rot,packed,pad", SHAPES)
def test_forward(T, hq, hk, d, rot, packed, pad, il):
    c = make(T, hq, hk, d, rot, seed=T + d, packed=packed, pad=pad)
    yq, yk, rq, rk = forward(c, d, il, want_rinv=True)
    nts.check_status()
    for y, r, x, g in ((yq, rq, c["q"], c["gq"]), (yk, rk, c["k"], c["gk"])):
        want, rinv, bound = ref.rope_forward(x, g, c["pos"], c["table"], d, EPS, il)
        assert torch.all((y.cpu().double() - want).abs() <= bound)
        assert torch.all((r.cpu().double() - rinv).abs() <= (d / 2 + 8) * ref.U32 * rinv)


@pytest.mark.parametrize("il", [False, True])
@pytest.mark.parametrize("T,hq,hk,d,rot,packed,pad", SHAPES)
def test_backward(T, hq, hk, d, rot, packed, pad, il):
    c = make(T, hq, hk, d, rot, seed=2 * T + d, packed=packed, pad=pad)
    dq, dk, dgq, dgk = backward(c, d, il)
    nts.check_status()
    for dx, dg, dy, x, g in ((dq, dgq, c["dyq"], c["q"], c["gq"]),
                             (dk, dgk, c["dyk"], c["k"], c["gk"])):
        wx, wg, bx, bg = ref.rope_backward(dy, x, g, c["pos"], c["table"], d, EPS, il)
        assert torch.all((dx.cpu().double() - wx).abs() <= bx)
        assert torch.all((dg.cpu().double() - wg).abs() <= bg)


@pytest.mark.parametrize("rows,stages", [(1, 2), (2, 3), (5, 1)])
@pytest.mark.parametrize("T,hq,hk,d,rot,packed,pad", SHAPES)
def test_ring_kernels_on_any_shape(T, hq, hk, d, rot, packed, pad, rows, stages):
    """The kernels of large calls, forced with other rings."""
    c = make(T, hq, hk, d, rot, seed=3 * T + d, packed=packed, pad=pad)
    il = (T + d) % 2 == 0
    try:
        nts.set_tuning(rows=rows, stages=stages)
        yq, yk, _, _ = forward(c, d, il)
        dq, dk, dgq, dgk = backward(c, d, il)
        nts.check_status()
    finally:
        nts.set_tuning()
    for y, dx, dg, dy, x, g in ((yq, dq, dgq, c["dyq"], c["q"], c["gq"]),
                                (yk, dk, dgk, c["dyk"], c["k"], c["gk"])):
        want, _, bound = ref.rope_forward(x, g, c["pos"], c["table"], d, EPS, il)
        assert torch.all((y.cpu().double() - want).abs() <= bound)
        wx, wg, bx, bg = ref.rope_backward(dy, x, g, c["pos"], c["table"], d, EPS, il)
        assert torch.all((dx.cpu().double() - wx).abs() <= bx)
        assert torch.all((dg.cpu().double() - wg).abs() <= bg)


def test_missing_copy_times_out_and_the_context_lives():
    c = make(50, 8, 2, 128, 128, seed=2)
    want = forward(c, 128, False)
    for fn in (forward, backward):
        nts.set_wait_limit_ns(20_000_000)
        nts.set_missing_tx(16)
        nts.set_tuning(rows=1, stages=2)
        try:
            fn(c, 128, False)
            with pytest.raises(nts.NtsError, match="TIMEOUT"):
                nts.check_status()
        finally:
            nts.set_tuning()
            nts.set_missing_tx(0)
            nts.set_wait_limit_ns(0)
    assert torch.equal(forward(c, 128, False)[0], want[0])
    nts.check_status()


def test_backward_against_differences():
    """Central differences of the fp64 forward formula, in every input value."""
    T, hq, hk, d, rot, il = 3, 2, 1, 32, 16, True
    c = make(T, hq, hk, d, rot, seed=5, pad=1)
    dq, _, dgq, _ = backward(c, d, il)
    h = 1e-6

    def loss(x, g):
        y, _, _ = ref.rope_forward(x, g, c["pos"], c["table"], d, EPS, il)
        return (y * torch.where((c["pos"] >= 0)[:, None], c["dyq"].double(), 0.0)).sum()

    x, g = c["q"].double(), c["gq"].double()
    _, _, bx, bg = ref.rope_backward(c["dyq"], c["q"], c["gq"], c["pos"], c["table"], d, EPS, il)
    # fp64 differences: the loss (below 1e3) is rounded at 2^-53, so a
    # quotient by 2h is off by less than 1e-6; the third derivative's term
    # h^2/6 lies far below that
    for t in range(T):
        for j in range(hq * d):
            up, dn = x.clone(), x.clone()
            up[t, j] += h
            dn[t, j] -= h
            num = (loss(up, g) - loss(dn, g)) / (2 * h)
            assert abs(float(dq[t, j]) - float(num)) <= float(bx[t, j]) + 1e-6
    for j in range(d):
        up, dn = g.clone(), g.clone()
        up[j] += h
        dn[j] -= h
        num = (loss(x, up) - loss(x, dn)) / (2 * h)
        assert abs(float(dgq[j]) - float(num)) <= float(bg[j]) + 1e-6


def test_matches_headwise_norm_without_turning():
    """Position 0 turns nothing: the result is the headwise norm's."""
    c = make(37, 8, 4, 128, 128, seed=3)
    c["pos"].zero_()
    yq, yk, _, _ = forward(c, 128, False)
    for y, x, g in ((yq, c["q"], c["gq"]), (yk, c["k"], c["gk"])):
        want, _ = nts.qknorm_rms_heads(x.to(DEV), g.to(DEV), 128, eps=EPS)
        # the sums of squares may be added in another order
        assert torch.all((y.float() - want.float()).abs() <= 2 * ref.UBF16 * want.float().abs())


def test_far_positions_keep_their_angle():
    P, rot = 1 << 17, 64
    t = nts.rope_table(P, rot, base=500000.0, device="cpu")
    pos = torch.tensor([0, 1, 99999, P - 1], dtype=torch.float64)
    i = torch.arange(rot // 2, dtype=torch.float64)
    ang = pos[:, None] * 500000.0 ** (-2 * i / rot)
    got = t[pos.long()].double()
    # an angle near 1e5 is rounded at 2^-37 in fp64, the value at 2^-24
    assert torch.all((got[:, :rot // 2] - ang.cos()).abs() <= 1.1 * ref.U32)
    assert torch.all((got[:, rot // 2:] - ang.sin()).abs() <= 1.1 * ref.U32)


def test_padding_rows_may_hold_anything_and_come_back_zero():
    c = make(9, 4, 2, 64, 64, seed=8, pad=4)
    for n in ("q", "k", "dyq", "dyk"):
        c[n][5:7] = float("nan")
        c[n][7:] = float("inf")
    yq, yk, rq, rk = forward(c, 64, False, want_rinv=True)
    dq, dk, dgq, dgk = backward(c, 64, False)
    nts.check_status()
    for t in (yq, yk, rq, rk, dq, dk):
        assert torch.all(t[5:] == 0) and torch.all(torch.isfinite(t))
    assert torch.all(torch.isfinite(dgq)) and torch.all(torch.isfinite(dgk))
    for dg, dy, x, g in ((dgq, c["dyq"], c["q"], c["gq"]), (dgk, c["dyk"], c["k"], c["gk"])):
        _, wg, _, bg = ref.rope_backward(dy, x, g, c["pos"], c["table"], 64, EPS, False)
        assert torch.all((dg.cpu().double() - wg).abs() <= bg)


def test_all_rows_padded_and_no_rows():
    c = make(6, 2, 2, 32, 32, seed=9, pad=6)
    dq, _, dgq, dgk = backward(c, 32, False)
    assert not dq.any() and not dgq.any() and not dgk.any()
    e = make(0, 2, 2, 32, 32, seed=9)
    yq, yk, _, _ = forward(e, 32, False)
    assert yq.shape == (0, 64) and yk.shape == (0, 64)
    _, _, dgq, dgk = backward(e, 32, False, dgamma_q=torch.full((32,), 7.0, device=DEV))
    assert not dgq.any() and not dgk.any()
    nts.check_status()


def test_position_outside_the_table_is_reported_and_gives_zeros():
    c = make(5, 2, 1, 64, 64, seed=4, P=100)
    good = forward(c, 64, False)
    c["pos"][2] = 100
    yq, yk, _, _ = forward(c, 64, False)
    with pytest.raises(nts.NtsError, match="INVALID_ARG.*rotation table"):
        nts.check_status()
    nts.check_status()   # cleared
    rows = [0, 1, 3, 4]
    assert not yq[2].any() and not yk[2].any()
    assert torch.equal(yq[rows], good[0][rows]) and torch.equal(yk[rows], good[1][rows])
    dq, _, _, _ = backward(c, 64, False)
    with pytest.raises(nts.NtsError, match="rotation table"):
        nts.check_status()
    assert not dq[2].any() and dq[1].any()


@pytest.mark.parametrize("spare", [0, 8])
def test_in_place_on_a_packed_buffer_leaves_the_rest(spare):
    T, hq, hk, d = 70, 6, 2, 128
    g = torch.Generator().manual_seed(1)
    buf = torch.randn(T, (hq + 2 * hk) * d + spare, generator=g).to(torch.bfloat16).to(DEV)
    keep = buf.clone()
    gq, gk = torch.ones(d, device=DEV), torch.full((d,), 0.5, device=DEV)
    pos = torch.arange(T, device=DEV)
    tab = nts.rope_table(T, d)
    q, k = buf[:, :hq * d], buf[:, hq * d:(hq + hk) * d]
    want = nts.qknorm_rope(q, gq, k, gk, pos, tab, head_dim=d)
    got = nts.qknorm_rope(q, gq, k, gk, pos, tab, head_dim=d, out_q=q, out_k=k)
    assert got[0].data_ptr() == q.data_ptr()
    assert torch.equal(q, want[0]) and torch.equal(k, want[1])
    assert torch.equal(buf[:, (hq + hk) * d:], keep[:, (hq + hk) * d:])
    # the gradient in place of the incoming gradient, in a packed buffer too
    dbuf = torch.randn(T, buf.shape[1], generator=g).to(torch.bfloat16).to(DEV)
    dkeep = dbuf.clone()
    dyq, dyk = dbuf[:, :hq * d], dbuf[:, hq * d:(hq + hk) * d]
    x = keep[:, :hq * d], keep[:, hq * d:(hq + hk) * d]
    w = nts.qknorm_rope_backward(dyq, dyk, x[0], gq, x[1], gk, pos, tab, head_dim=d)
    nts.qknorm_rope_backward(dyq, dyk, x[0], gq, x[1], gk, pos, tab, head_dim=d, out_dq=dyq,
                             out_dk=dyk)
    assert torch.equal(dyq, w[0]) and torch.equal(dyk, w[1])
    assert torch.equal(dbuf[:, (hq + hk) * d:], dkeep[:, (hq + hk) * d:])
    nts.check_status()


def test_infinite_and_nan_values_stay_in_their_head():
    c = make(4, 3, 2, 64, 32, seed=6)
    clean = forward(c, 64, True)
    c["q"][1, 64 + 5] = float("nan")    # token 1, head 1
    c["k"][2, 40] = float("inf")        # token 2, head 0, beyond rot
    yq, yk, _, _ = forward(c, 64, True)
    assert torch.isnan(yq[1, 64:128]).all()
    mask = torch.ones_like(yq, dtype=torch.bool)
    mask[1, 64:128] = False
    assert torch.equal(yq[mask], clean[0][mask])
    # an infinite sum of squares: rinv = 0, the infinite value NaN, the others 0
    row = yk[2, :64]
    assert torch.isnan(row[40]) and int(torch.isnan(row).sum()) == 1
    assert not torch.nan_to_num(row).any()
    assert torch.equal(yk[2, 64:], clean[1][2, 64:])


def test_equal_calls_give_equal_bits_on_streams_and_in_graphs():
    c = make(257, 12, 4, 128, 128, seed=12, packed=True, pad=5)
    D = {k: to_dev(v) for k, v in c.items()}

    def both(**kw):
        y = nts.qknorm_rope(D["q"], D["gq"], D["k"], D["gk"], D["pos"], D["table"], head_dim=128,
                            **kw)
        g = nts.qknorm_rope_backward(D["dyq"], D["dyk"], D["q"], D["gq"], D["k"], D["gk"],
                                     D["pos"], D["table"], head_dim=128, **kw)
        return list(y[:2]) + list(g)

    want = both()
    assert all(torch.equal(a, b) for a, b in zip(want, both()))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    other = both(stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, other))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cap = both()
    for _ in range(3):
        for t in cap:
            t.fill_(9)
        graph.replay()
        both()                     # an eager call between the replays
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, cap))
    nts.check_status()


@pytest.mark.parametrize("T,d", [(1, 16), (9, 16), (300, 48), (2000, 64), (257, 128), (40, 512)])
def test_the_gains_gradients_have_one_order_however_they_are_summed(T, d):
    """The last CTA's sum, a launch of its own in a graph, and a workspace that
    starts off a vector boundary."""
    c = make(T, 5, 2, d, d, seed=41)
    want = backward(c, d, False)
    ws = torch.empty(nts.rope_backward_workspace(d) + 4, dtype=torch.uint8, device=DEV)
    odd = backward(c, d, False, workspace=ws[4:])
    D = {k: to_dev(v) for k, v in c.items()}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cap = nts.qknorm_rope_backward(D["dyq"], D["dyk"], D["q"], D["gq"], D["k"], D["gk"],
                                       D["pos"], D["table"], head_dim=d, eps=EPS)
    graph.replay()
    torch.cuda.synchronize()
    for a, b, g in zip(want, odd, cap):
        assert torch.equal(a, b) and torch.equal(a, g)
    nts.check_status()


def test_canaries():
    T, hq, hk, d = 41, 5, 2, 96
    c = make(T, hq, hk, d, 64, seed=31, packed=True, pad=2)
    pad = 4096

    def padded(shape, dtype):
        n = math.prod(shape) * torch.tensor([], dtype=dtype).element_size()
        buf = torch.full((2 * pad + n,), 0xA5, dtype=torch.uint8, device=DEV)
        return buf, buf[pad:pad + n].view(dtype).view(shape)

    bufs = {n: padded(s, t) for n, s, t in (
        ("out_q", (T, hq * d), torch.bfloat16), ("out_k", (T, hk * d), torch.bfloat16),
        ("rinv_q", (T, hq), torch.float32), ("rinv_k", (T, hk), torch.float32))}
    forward(c, d, False, **{n: t for n, (_, t) in bufs.items()})
    grads = {n: padded(s, t) for n, s, t in (
        ("out_dq", (T, hq * d), torch.bfloat16), ("out_dk", (T, hk * d), torch.bfloat16),
        ("dgamma_q", (d,), torch.float32), ("dgamma_k", (d,), torch.float32),
        ("workspace", (nts.rope_backward_workspace(d),), torch.uint8))}
    backward(c, d, False, **{n: t for n, (_, t) in grads.items()})
    nts.check_status()
    for n, (buf, _) in {**bufs, **grads}.items():
        assert bool((buf[:pad] == 0xA5).all()) and bool((buf[-pad:] == 0xA5).all()), n


@pytest.mark.parametrize("ring", [False, True])
@pytest.mark.parametrize("bad", ["gain", "row 0"])
@pytest.mark.parametrize("value", [math.inf, math.nan])
def test_padding_rows_are_zeros_whatever_the_gain_and_the_table_hold(value, bad, ring):
    """Zeros out, and nothing added to the gains' gradients, in rows that no value of
    theirs decides: by choice, not by products with zero."""
    T, hq, hk, d, rot = 21, 6, 2, 64, 48
    c = make(T, hq, hk, d, rot, seed=11, pad=4)
    c["pos"][:T - 4] = torch.arange(1, T - 3)     # row 0 belongs to no token
    c["pos"][3] = c["table"].shape[0] + 5         # nor does a row beyond the table
    wants = [ref.rope_backward(dy, x, g, c["pos"], c["table"], d, EPS, False)
             for dy, x, g in ((c["dyq"], c["q"], c["gq"]), (c["dyk"], c["k"], c["gk"]))]
    if bad == "gain":
        c["gq"][5] = c["gk"][60] = value
    else:
        c["table"][0] = value
    try:
        if ring:
            nts.set_tuning(rows=1, stages=2)
        y = forward(c, d, False, want_rinv=True)
        dq, dk, dgq, dgk = backward(c, d, False)
        with pytest.raises(nts.NtsError, match="rotation table"):
            nts.check_status()
    finally:
        nts.set_tuning()
    empty = [3] + list(range(T - 4, T))
    for t in (*y, dq, dk):
        assert not t[empty].any()                 # a NaN counts as something
    for dx, dg, (wx, wg, bx, bg) in ((dq, dgq, wants[0]), (dk, dgk, wants[1])):
        assert torch.all((dg.cpu().double() - wg).abs() <= bg)   # no gain is part of it
        if bad == "row 0":
            assert torch.all((dx.cpu().double() - wx).abs() <= bx)


def test_gradient_of_zero_rows_at_the_smallest_eps():
    T, hq, hk, d, rot, eps = 5, 2, 1, 32, 32, 2.0 ** -126
    c = make(T, hq, hk, d, rot, seed=12)
    c["q"][1] = 0
    c["k"][2] = 0
    c["dyq"] *= 2.0 ** -40                        # rinv is 2^63 there
    c["dyk"] *= 2.0 ** -40
    D = {k: to_dev(v) for k, v in c.items()}
    got = nts.qknorm_rope_backward(D["dyq"], D["dyk"], D["q"], D["gq"], D["k"], D["gk"], D["pos"],
                                   D["table"], head_dim=d, eps=eps)
    nts.check_status()
    for dx, dg, dy, x, g in ((got[0], got[2], c["dyq"], c["q"], c["gq"]),
                             (got[1], got[3], c["dyk"], c["k"], c["gk"])):
        wx, wg, bx, bg = ref.rope_backward(dy, x, g, c["pos"], c["table"], d, eps, False)
        assert wx.abs().max() > 2.0 ** 20 and bool(torch.isfinite(dx).all())
        assert torch.all((dx.cpu().double() - wx).abs() <= bx)
        assert torch.all((dg.cpu().double() - wg).abs() <= bg)
    with pytest.raises(nts.NtsError, match="UNSUPPORTED"):
        nts.qknorm_rope_backward(D["dyq"], D["dyk"], D["q"], D["gq"], D["k"], D["gk"], D["pos"],
                                 D["table"], head_dim=d, eps=2.0 ** -130)
