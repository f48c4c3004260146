"""A training step of a layer -- residual, norm and cast, 8-bit projection, rotation, and
all of it back -- with every tensor of it held to its formula in fp64, one value at a time:
each formula takes what the step before it gave."""
import pytest
import torch

import block_reference as ref
from test_gpu_addnorm import gradient
from test_gpu_layer_calls import AXES, DEV, EPS, check_addnorm, check_axes, gen, grid_positions, randn

pytestmark = pytest.mark.gpu

nts = pytest.importorskip("normalization_token_split_gb300")
HQ, HK, HD = 4, 2, 128


def step(T, D, res, seed):
    g = gen(seed)
    N = (HQ + HK) * HD
    w = (randn(g, N, D) * D ** -0.5).to(torch.bfloat16)
    c = dict(W=nts.blockcast(w, block_rows=128), Wt=nts.blockcast(w.t().contiguous(), block_rows=128),
             gain=1 + 0.1 * randn(g, D), gq=1 + 0.1 * randn(g, HD), gk=1 + 0.1 * randn(g, HD),
             table=nts.rope_table(64, HD), pos=grid_positions(T), x=randn(g, T, D).to(torch.bfloat16),
             r=randn(g, T, D).to(res), dyq=randn(g, T, HQ * HD).to(torch.bfloat16),
             dyk=randn(g, T, HK * HD).to(torch.bfloat16), behind=randn(g, T, D).to(res))
    c["pos"][T - 9:] = -1                         # padding behind the last sequence
    c["n"] = n = nts.add_rmsnorm_blockcast(c["x"], c["r"], c["gain"], want_rinv=True)
    c["y"] = y = nts.gemm_blockscaled(n.codes, n.scales, c["W"].codes, c["W"].scales)
    c["q"], c["k"] = y[:, :HQ * HD], y[:, HQ * HD:]
    rot = (c["q"], c["gq"], c["k"], c["gk"], c["pos"], c["table"], AXES)
    c["yq"], c["yk"], _, _ = nts.qknorm_rope_axes(*rot, head_dim=HD)
    c["dy"] = torch.empty_like(y)
    c["dq"], c["dk"], c["dgq"], c["dgk"] = nts.qknorm_rope_axes_backward(
        c["dyq"], c["dyk"], *rot, head_dim=HD, out_dq=c["dy"][:, :HQ * HD], out_dk=c["dy"][:, HQ * HD:])
    c["dY"] = nts.blockcast(c["dy"])
    c["dn"] = nts.gemm_blockscaled(c["dY"].codes, c["dY"].scales, c["Wt"].codes, c["Wt"].scales)
    c["dres"], c["dx"], c["dgain"] = nts.add_rmsnorm_backward(c["dn"], n.h, n.rinv, c["gain"],
                                                              dres=c["behind"])
    nts.check_status()
    return c


def within(got, want, room):
    if got.dtype is torch.bfloat16:
        room = ref.UBF16 * want.abs() + (1 + ref.UBF16) * room + 2.0 ** -133
    return (got.double() - want).abs() <= room


@pytest.mark.parametrize("res", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,D", [(200, 1024), (77, 528)])
def test_every_tensor_of_a_training_step(T, D, res):
    c = step(T, D, res, seed=T)
    n = c["n"]
    check_addnorm(c["x"], c["r"], c["gain"], n)
    check_axes(c["yq"], c["q"], c["gq"], c["pos"], c["table"])
    check_axes(c["yk"], c["k"], c["gk"], c["pos"], c["table"])
    for y, a, w, K in ((c["y"], n, c["W"], D), (c["dn"], c["dY"], c["Wt"], (HQ + HK) * HD)):
        want, mag = ref.gemm(a.codes, a.scales, w.codes, w.scales, 128)
        assert torch.all((y.double() - want).abs() <= ref.gemm_bound(want, mag, K, False))
    dy = c["dy"].float().cpu()
    scales = ref.block_scales(dy, 1)
    assert torch.equal(c["dY"].scales.cpu(), scales)
    assert torch.equal(c["dY"].codes.cpu(), ref.block_codes(dy, scales, 1))
    axis = torch.tensor(list(AXES))
    keep, t = (c["pos"] >= 0).all(1).cpu(), c["table"].cpu()
    at, i = c["pos"].cpu().clamp_min(0)[:, axis], torch.arange(len(AXES))
    rows = torch.cat((t[at, i], t[at, len(AXES) + i]), 1)
    for dx, dg, dyv, xv, gm in ((c["dq"], c["dgq"], c["dyq"], c["q"], c["gq"]),
                                (c["dk"], c["dgk"], c["dyk"], c["k"], c["gk"])):
        wx, wg, bx, bg = ref.rope_backward(dyv.cpu(), xv.cpu(), gm.cpu(),
                                           torch.where(keep, torch.arange(T), -1), rows, HD, EPS, False)
        assert torch.all((dx.cpu().double() - wx).abs() <= bx)
        assert torch.all((dg.cpu().double() - wg).abs() <= bg)
    case = dict(dy=c["dn"], gamma=c["gain"], e=c["behind"])
    want, wg, room, bg = gradient(case, n.h, n.rinv)
    assert within(c["dres"], want, room).all()
    assert (c["dx"] is None) == (res is torch.bfloat16)
    if c["dx"] is not None:
        assert torch.equal(c["dx"], c["dres"].to(torch.bfloat16))
    assert torch.all((c["dgain"].double() - wg).abs() <= bg)


def mistakes(c):
    """Formulas of dres and dgain that lack or turn a term."""
    v, dy, r, gm = c["n"].h.double(), c["dn"].double(), c["n"].rinv.double()[:, None], c["gain"].double()
    u, e = dy * gm, c["behind"].double()
    mean = v * r ** 3 * (u * v).mean(1, keepdim=True)
    plain = v * r ** 3 * (dy * v).mean(1, keepdim=True)
    return dict(no_mean=r * u + e, mean_turned=r * u + mean + e, no_gain=r * dy - plain + e,
                no_norm=e, nothing_from_behind=r * u - mean), \
        dict(no_factor=(dy * v).sum(0), of_the_gain=(u * v * r).sum(0))


@pytest.mark.parametrize("res", [torch.bfloat16, torch.float32])
def test_a_formula_without_one_of_its_terms_is_seen(res):
    """The bounds above tell the gradient from each of these, on the CPU's side of the
    comparison: the kernels' values are right for one formula alone."""
    c = step(200, 1024, res, seed=5)
    c = {k: v.cpu() if torch.is_tensor(v) else v for k, v in c.items()}
    c["n"] = nts.AddNormOut(*(t.cpu() for t in c["n"]))
    _, _, room, bg = gradient(dict(dy=c["dn"], gamma=c["gain"], e=c["behind"]), c["n"].h, c["n"].rinv)
    wrong, wrong_gain = mistakes(c)
    for name, want in wrong.items():
        assert not within(c["dres"], want, room).all(), name
    for name, want in wrong_gain.items():
        assert not torch.all((c["dgain"].double() - want).abs() <= bg), name
