"""The residual's addition with RMSNorm and the block-128 cast, and its gradient,
on the GPU against the fp64 formulas, fp32 steps and differences."""
import pytest
import torch

import block_reference as ref

pytestmark = pytest.mark.gpu

nts = pytest.importorskip("normalization_token_split_gb300")
DEV = "cuda:0"
EPS = 1e-6
TYPES = [torch.bfloat16, torch.float32]

SHAPES = [  # T, D
    (1, 16), (3, 48), (70, 128), (33, 144), (1, 4096), (130, 496), (2500, 512), (9, 528), (700, 1024),
    (5, 2064), (64, 4096), (999, 4096), (6, 5120), (1237, 5120), (4, 8192), (3, 8208), (40, 16384),
    (7, 16400), (600, 16384), (2, 32768), (333, 32768), (70000, 32),
]


def make(T, D, res, seed, gain=True, behind=True):
    g = torch.Generator(device=DEV).manual_seed(seed)

    def randn(*shape):
        return torch.randn(*shape, generator=g, device=DEV)

    return dict(x=randn(T, D).to(torch.bfloat16), r=(2 * randn(T, D)).to(res),
                gamma=1 + 0.1 * randn(D) if gain else None, dy=randn(T, D).to(torch.bfloat16),
                e=randn(T, D).to(res) if behind else None)


def check_forward(c, o, eps=EPS):
    h = (c["x"].float() + c["r"].float()).to(c["r"].dtype)
    assert torch.equal(o.h, h)
    D = h.shape[1]
    want = (h.double().square().mean(1) + eps).rsqrt()
    # a sum of D squares, halved by the root, and a few roundings
    assert torch.all((o.rinv.double() - want).abs() <= (D / 2 + 4) * ref.U32 * want)
    # from the kernel's factor on, step by step in fp32
    w = h.float() if c["gamma"] is None else h.float() * c["gamma"]
    w = (w * o.rinv[:, None]).cpu()
    scales = ref.block_scales(w, 1)
    assert torch.equal(o.scales.cpu(), scales)
    assert torch.equal(o.codes.cpu(), ref.block_codes(w, scales, 1))


def gradient(c, h, rinv):
    """(dres, dgamma, bounds), fp64.  dres: the sum of D products, then about a dozen
    roundings of each of its three terms; dgamma: the sum over the rows."""
    T, D = h.shape
    v, dy, r = h.double(), c["dy"].double(), rinv.double()[:, None]
    u = dy if c["gamma"] is None else dy * c["gamma"].double()
    e = torch.zeros_like(v) if c["e"] is None else c["e"].double()
    dh = r * u - v * r ** 3 * (u * v).mean(1, keepdim=True) + e
    mag = r * u.abs() + v.abs() * r ** 3 * (u * v).abs().mean(1, keepdim=True) + e.abs()
    n = dy * v * r
    room = (D + 16) * ref.U32 * mag
    return dh, n.sum(0), room, (T + 4) * ref.U32 * n.abs().sum(0) + 2.0 ** -126


def check_backward(c, h, rinv, got):
    dres, dx, dg = got
    want, wg, room, bg = gradient(c, h, rinv)
    rounded = ref.UBF16 * want.abs() + (1 + ref.UBF16) * room + 2.0 ** -133
    for t in (dres, dx):
        if t is not None:
            bound = rounded if t.dtype is torch.bfloat16 else room + 2.0 ** -149
            assert torch.all((t.double() - want).abs() <= bound)
    assert (dx is None) == (h.dtype is torch.bfloat16)
    if dx is not None:
        assert torch.equal(dx, dres.to(torch.bfloat16))
    assert (dg is None) == (c["gamma"] is None)
    if dg is not None:
        assert torch.all((dg.double() - wg).abs() <= bg)


@pytest.mark.parametrize("res", TYPES)
@pytest.mark.parametrize("T,D", SHAPES)
def test_formulas(T, D, res):
    c = make(T, D, res, seed=T + D)
    o = nts.add_rmsnorm_blockcast(c["x"], c["r"], c["gamma"], eps=EPS, want_rinv=True)
    nts.check_status()
    check_forward(c, o)
    got = nts.add_rmsnorm_backward(c["dy"], o.h, o.rinv, c["gamma"], dres=c["e"])
    nts.check_status()
    check_backward(c, o.h, o.rinv, got)


@pytest.mark.parametrize("res", TYPES)
@pytest.mark.parametrize("T,D", [(5, 96), (300, 4096), (3, 16384)])
def test_without_a_gain_or_a_gradient_from_behind(T, D, res):
    c = make(T, D, res, seed=T, gain=False, behind=False)
    o = nts.add_rmsnorm_blockcast(c["x"], c["r"], eps=EPS, want_rinv=True)
    check_forward(c, o)
    assert nts.add_rmsnorm_blockcast(c["x"], c["r"], eps=EPS).rinv is None
    check_backward(c, o.h, o.rinv, nts.add_rmsnorm_backward(c["dy"], o.h, o.rinv))
    c["gamma"] = torch.rand(D, device=DEV)
    check_backward(c, o.h, o.rinv, nts.add_rmsnorm_backward(c["dy"], o.h, o.rinv, c["gamma"]))
    nts.check_status()


@pytest.mark.parametrize("res", TYPES)
def test_rows_that_are_the_norm_alone(res):
    """A residual of zeros: what rmsnorm_blockcast gives, but for the order of a sum."""
    c = make(50, 4096, torch.bfloat16, seed=3)
    o = nts.add_rmsnorm_blockcast(c["x"], torch.zeros(50, 4096, dtype=res, device=DEV), c["gamma"],
                                  want_rinv=True)
    want = nts.rmsnorm_blockcast(c["x"], c["gamma"], want_rinv=True)
    assert torch.all((o.rinv / want.rinv - 1).abs() <= 4096 * ref.U32)
    assert (o.codes != want.codes).float().mean() < 1e-3
    nts.check_status()


@pytest.mark.parametrize("res", TYPES)
def test_odd_rows(res):
    """Zeros, tiny and huge sums, infinities and NaN stay in their rows."""
    T, D = 12, 640
    c = make(T, D, res, seed=5)
    c["x"][0] = 0
    c["r"][0] = 0
    c["x"][1], c["r"][1] = 1, -1                  # a sum of zero
    c["x"][2], c["r"][2] = 2.0 ** -120, 0
    c["r"][3, 5] = float("inf")
    c["x"][4, 7] = float("nan")
    c["x"][5, 9] = 3e38
    c["r"][5, 9] = 3e38                           # the sum overflows
    c["x"][6], c["r"][6] = 1e18, -2e17
    o = nts.add_rmsnorm_blockcast(c["x"], c["r"], c["gamma"], eps=EPS, want_rinv=True)
    nts.check_status()
    h = (c["x"].float() + c["r"].float()).to(res)
    assert torch.equal(o.h.nan_to_num(7.0, 8.0, 9.0), h.nan_to_num(7.0, 8.0, 9.0))
    fine = [i for i in range(T) if i not in (3, 4, 5, 6)]
    sub = {k: (v if k == "gamma" else v[fine]) for k, v in c.items()}
    check_forward(sub, nts.AddNormOut(*(t[fine] for t in o)))
    assert not o.codes[:2].any() and o.rinv[0] == torch.tensor(EPS).rsqrt()
    # an infinite row: its finite values vanish, the infinite one has no value
    for row, at in ((3, 5), (5, 9)):
        assert o.rinv[row] == 0 and o.codes[row, at] & 127 == 127
    # 640 squares of 8e17 are 4.1e38, beyond fp32: the row counts as infinitely large
    assert o.rinv[6] == 0 and not o.codes[6].any()
    assert o.rinv[4].isnan() and torch.all(o.codes[4] & 127 == 127)
    got = nts.add_rmsnorm_backward(c["dy"], o.h, o.rinv, None, dres=c["e"])
    check_backward(dict(sub, gamma=None), o.h[fine], o.rinv[fine],
                   (got[0][fine], None if got[1] is None else got[1][fine], None))


@pytest.mark.parametrize("res", TYPES)
@pytest.mark.parametrize("T,D", [(1, 80), (37, 528), (300, 4096), (5, 16400)])
def test_bounds_and_alignment(T, D, res):
    """Buffers on 16-byte but not 32-byte boundaries, with bytes around them that stay."""
    c = make(T, D, res, seed=T + D)

    def odd(t):
        n, size = t.numel(), t.element_size()
        buf = torch.full((n * size + 4096 + 16,), 0xA5, dtype=torch.uint8, device=DEV)
        start = (-buf.data_ptr()) % 32 + 16
        v = buf[start:start + n * size].view(t.dtype).view(t.shape)
        v.copy_(t)
        return buf, start, n * size, v

    def kept(b):
        buf, start, n, _ = b
        return bool((buf[:start] == 0xA5).all()) and bool((buf[start + n:] == 0xA5).all())

    o = nts.add_rmsnorm_blockcast(c["x"], c["r"], c["gamma"], want_rinv=True)
    b = nts.add_rmsnorm_backward(c["dy"], o.h, o.rinv, c["gamma"], dres=c["e"])
    ins = {k: odd(v) for k, v in c.items()}
    outs = [odd(t) for t in o]
    a = nts.add_rmsnorm_blockcast(ins["x"][3], ins["r"][3], ins["gamma"][3], out=outs[0][3],
                                  codes=outs[1][3], scales=outs[2][3], rinv=outs[3][3])
    backs = [odd(t) if t is not None else None for t in b]
    ws = torch.empty(nts.add_rmsnorm_backward_workspace(D), dtype=torch.uint8, device=DEV)
    g = nts.add_rmsnorm_backward(ins["dy"][3], a.h, a.rinv, ins["gamma"][3], dres=ins["e"][3],
                                 out=backs[0][3], out_x=backs[1] and backs[1][3], dgamma=backs[2][3],
                                 workspace=ws)
    nts.check_status()
    for got, want in zip((*a, *g), (*o, *b)):
        assert (got is None and want is None) or torch.equal(got, want)
    assert all(kept(t) for t in (*outs, *ins.values(), *backs) if t is not None)


@pytest.mark.parametrize("res", TYPES)
@pytest.mark.parametrize("T,D", [(3, 64), (2000, 4096), (700, 8208)])
def test_in_place(T, D, res):
    c = make(T, D, res, seed=T)
    o = nts.add_rmsnorm_blockcast(c["x"], c["r"], c["gamma"], want_rinv=True)
    b = nts.add_rmsnorm_backward(c["dy"], o.h, o.rinv, c["gamma"], dres=c["e"])
    r = c["r"].clone()
    got = nts.add_rmsnorm_blockcast(c["x"], r, c["gamma"], out=r)
    assert got.h.data_ptr() == r.data_ptr() and torch.equal(r, o.h) and torch.equal(got.codes, o.codes)
    over = [dict(dres=c["e"].clone()), dict(dres=c["e"], h=o.h.clone())]
    for kw in over:
        h = kw.pop("h", o.h)
        out = kw["dres"] if h is o.h else h
        dy = c["dy"].clone()
        got = nts.add_rmsnorm_backward(dy, h, o.rinv, c["gamma"], out=out,
                                       out_x=dy if res is torch.float32 else None, **kw)
        for x, want in zip(got, b):
            assert want is None or torch.equal(x, want)
    if res is torch.bfloat16:
        x, dy = c["x"].clone(), c["dy"].clone()
        assert torch.equal(nts.add_rmsnorm_blockcast(x, c["r"], c["gamma"], out=x).h, o.h)
        assert torch.equal(nts.add_rmsnorm_backward(dy, o.h, o.rinv, c["gamma"], dres=c["e"],
                                                    out=dy)[0], b[0])
    nts.check_status()


@pytest.mark.parametrize("D", [64, 8208])
def test_gradient_against_differences(D):
    """Along a direction of x and of gamma, against differences of the fp64 formula."""
    T = 5
    c = make(T, D, torch.float32, seed=11)
    o = nts.add_rmsnorm_blockcast(c["x"], c["r"], c["gamma"], want_rinv=True)
    dres, _, dg = nts.add_rmsnorm_backward(c["dy"], o.h, o.rinv, c["gamma"], dres=c["e"])
    g = torch.Generator(device=DEV).manual_seed(12)
    u = torch.randn(T, D, generator=g, device=DEV, dtype=torch.float64)
    v = torch.randn(D, generator=g, device=DEV, dtype=torch.float64)

    def value(s):
        h = o.h.double() + s * u
        w = h * (h.square().mean(1, keepdim=True) + EPS).rsqrt() * (c["gamma"].double() + s * v)
        return (w * c["dy"].double()).sum() + (h * c["e"].double()).sum()

    step = 1e-5
    want = (value(step) - value(-step)) / (2 * step)
    got = (dres.double() * u).sum() + (dg.double() * v).sum()
    mag = (dres.double() * u).abs().sum() + (dg.double() * v).abs().sum()
    # rinv's rounding and the sums', (D + T + 32) of U32; the differences' of step^2
    assert abs(got - want) <= (D + T + 32) * ref.U32 * mag + 1e-7 * mag


def test_equal_calls_give_equal_bits():
    for T, D in ((3000, 4096), (200, 16384), (5000, 256)):
        c = make(T, D, torch.bfloat16, seed=1)
        o = nts.add_rmsnorm_blockcast(c["x"], c["r"], c["gamma"], want_rinv=True)
        b = nts.add_rmsnorm_backward(c["dy"], o.h, o.rinv, c["gamma"], dres=c["e"])
        for _ in range(5):
            p = nts.add_rmsnorm_blockcast(c["x"], c["r"], c["gamma"], want_rinv=True)
            q = nts.add_rmsnorm_backward(c["dy"], o.h, o.rinv, c["gamma"], dres=c["e"])
            assert all(torch.equal(s, t) for s, t in zip(p, o))
            assert torch.equal(q[0], b[0]) and torch.equal(q[2], b[2])
    nts.check_status()


def test_empty_batch():
    c = make(1, 256, torch.float32, seed=2)
    x, r = c["x"][:0], c["r"][:0]
    o = nts.add_rmsnorm_blockcast(x, r, c["gamma"], want_rinv=True)
    assert o.h.shape == (0, 256) and o.scales.shape == (0, 2)
    got = nts.add_rmsnorm_backward(x, r, o.rinv, c["gamma"],
                                   dgamma=torch.full((256,), 3.0, device=DEV))
    assert not got[2].any()
    nts.check_status()


@pytest.mark.parametrize("res", TYPES)
def test_beyond_32_bit_offsets(res):
    T, D = 66000, 32768                           # 2.2e9 values
    g = torch.Generator(device=DEV).manual_seed(6)
    x = torch.randn(1000, D, generator=g, device=DEV).to(torch.bfloat16).repeat(66, 1)
    r = x.clone().to(res)
    o = nts.add_rmsnorm_blockcast(x, r, out=r, want_rinv=True)
    n = 40
    tail = nts.AddNormOut(*(t[-n:] for t in o))
    check_forward(dict(x=x[-n:], r=x[-n:].to(res), gamma=None), tail)
    h = tail.h.clone()
    got = nts.add_rmsnorm_backward(x, o.h, o.rinv, out=o.h,
                                   out_x=x if res is torch.float32 else None)
    dy = torch.randn(1000, D, generator=torch.Generator(device=DEV).manual_seed(6),
                     device=DEV).to(torch.bfloat16)[-n:]
    check_backward(dict(dy=dy, gamma=None, e=None), h, tail.rinv,
                   (got[0][-n:], None if got[1] is None else got[1][-n:], None))
    nts.check_status()


def test_refusals():
    T, D = 6, 256
    c = make(T, D, torch.bfloat16, seed=9)
    x, r, gm = c["x"], c["r"], c["gamma"]
    rinv = torch.ones(T, device=DEV)
    for args, match in (((x.float(), r, gm), "x must be torch.bfloat16"),
                        ((x, r.half(), gm), "residual must be torch.bfloat16 or torch.float32"),
                        ((x, r[:5], gm), "residual has the wrong shape"),
                        ((x.t(), r, gm), "x must be contiguous"),
                        ((x, r.float().t(), gm), "residual must be contiguous"),
                        ((x, r.cpu(), gm), "residual must be a CUDA tensor"),
                        ((x, r, gm[:128]), "gamma must hold D values")):
        with pytest.raises(ValueError, match=match):
            nts.add_rmsnorm_blockcast(*args)
    with pytest.raises(ValueError, match="out must be torch.bfloat16"):
        nts.add_rmsnorm_blockcast(x, r, gm, out=r.float())
    with pytest.raises(ValueError, match="codes has the wrong shape"):
        nts.add_rmsnorm_blockcast(x, r, gm, codes=torch.zeros(T, D // 2, dtype=torch.uint8, device=DEV))
    with pytest.raises(nts.NtsError, match="INVALID_ARG"):
        nts.add_rmsnorm_blockcast(x, r, gm, eps=0.0)
    wide = torch.zeros(1, 32768 + 16, dtype=torch.bfloat16, device=DEV)
    with pytest.raises(nts.NtsError, match="UNSUPPORTED"):
        nts.add_rmsnorm_blockcast(wide, wide)
    thin = torch.zeros(2, 24, dtype=torch.bfloat16, device=DEV)
    with pytest.raises(nts.NtsError, match="UNSUPPORTED"):
        nts.add_rmsnorm_backward(thin, thin, rinv[:2])
    for kw, match in ((dict(dres=r.float()), "dres must be torch.bfloat16"),
                      (dict(dres=r[:5]), "dres has the wrong shape"),
                      (dict(out_x=x), "out is bfloat16 already"),
                      (dict(gamma=None, dgamma=gm), "no gamma"),
                      (dict(workspace=gm), "workspace must be torch.uint8")):
        with pytest.raises(ValueError, match=match):
            nts.add_rmsnorm_backward(x, r, rinv, **{"gamma": gm, **kw})
    with pytest.raises(ValueError, match="rinv must hold a factor per row"):
        nts.add_rmsnorm_backward(x, r, rinv[:5], gm)
    with pytest.raises(nts.NtsError, match="INVALID_ARG.*workspace"):
        nts.add_rmsnorm_backward(x, r, rinv, gm, workspace=torch.zeros(64, dtype=torch.uint8, device=DEV))
    nts.check_status()
