"""Cases of the operators beside the QKV projection's, in plain torch and through
the package: the residual's addition with RMSNorm and the 8-bit cast, its
gradient, products of few rows with 4-bit weights, and headwise QK-RMSNorm with
a rotation of several position axes, forward and backward.

``run`` computes an operator from elementary torch operations in fp32 while
``own`` is false, and calls the package's entry point when it is true.
``exact`` gives the same outputs from the definitions in fp64.
"""
from __future__ import annotations

import math

import torch

own = False

DEV = "cuda"
BLOCK = 128          # values per scale of the 8-bit operands
E4M3_MAX = 448.0
AMAX_MIN = 2.0 ** -100   # block absmaxes below this take its scale
EPS = 1e-6

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)   # magnitudes of codes 0 .. 7; bit 3 is the sign
HEAD_DIMS = (32, 48, 64, 80, 96, 112, 128, 160, 192, 256)


# ------------------------------------------------------------------- cases

def listed():
    return [
        # between two layers of a decode batch
        dict(name="addnorm_decode", op="addnorm", T=8, D=4096, res="bf16", gain=True),
        # a ragged batch whose residual stream is kept in fp32
        dict(name="addnorm_fp32", op="addnorm", T=1237, D=5120, res="fp32", gain=True),
        # between two layers of a prefill
        dict(name="addnorm_prefill", op="addnorm", T=16384, D=4096, res="bf16", gain=True),
        # gradients of a short sequence, the residual stream in fp32
        dict(name="addnorm_bwd_short", op="addnorm_bwd", T=333, D=4096, res="fp32", gain=True,
             onward=True),
        # gradients of a training batch at the 13B-like width
        dict(name="addnorm_bwd_long", op="addnorm_bwd", T=8192, D=5120, res="bf16", gain=True,
             onward=True),
        # QKV projection of one decoded token, 7B-like, straight from bf16 activations
        dict(name="gemv_decode_1", op="gemv", M=1, N=12288, K=4096, fmt="e2m1", group=32, act="bf16",
             out="bf16"),
        # the wide projection back of a small batch, on the norm's 8-bit activations
        dict(name="gemv_batch_8", op="gemv", M=8, N=5120, K=16384, fmt="int4", group=128, act="e4m3",
             out="bf16"),
        # QKV projection of a decode batch, 13B-like
        dict(name="gemv_batch_32", op="gemv", M=32, N=15360, K=5120, fmt="e2m1", group=64, act="bf16",
             out="bf16"),
        # one decoded token behind a video: q and k are views of its packed QKV row
        dict(name="axes_decode_1", op="axes", T=1, hq=32, hk=32, d=128, rot=128, naxes=3,
             order="sections", restart=False, interleaved=False, packed=True, far=True, pad=False,
             by_axis=False),
        # a prompt of text and video frames
        dict(name="axes_prefill", op="axes", T=8192, hq=40, hk=40, d=128, rot=128, naxes=3,
             order="sections", restart=False, interleaved=False, packed=True, far=False, pad=False,
             by_axis=True),
        # gradients of a short padded sequence of images, grouped heads, rows and columns turned
        # by their own frequencies, pairs side by side
        dict(name="axes_bwd_short", op="axes_bwd", T=333, hq=32, hk=8, d=64, rot=64, naxes=2,
             order="sections", restart=True, interleaved=True, packed=True, far=False, pad=True,
             by_axis=False),
        # gradients of a training sequence of video, the axes taking the pairs in turn
        dict(name="axes_bwd_long", op="axes_bwd", T=8192, hq=40, hk=40, d=128, rot=128, naxes=3,
             order="cyclic", restart=False, interleaved=False, packed=True, far=False, pad=False,
             by_axis=False),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _cost(case):
    w = work(case)
    return w["bytes"] / 6.7e12 + w["flops"] / 1.9e15


def draw(rng):
    op = rng.choice(("addnorm", "addnorm_bwd", "gemv", "gemv", "axes", "axes_bwd"))
    most = max(_cost(c) for c in listed() if c["op"] == op)
    while True:
        if op in ("addnorm", "addnorm_bwd"):
            case = dict(op=op, T=_log_int(rng, 1, 16384), D=16 * _log_int(rng, 1, 2048),
                        res=rng.choice(("bf16", "fp32")), gain=rng.random() < 0.8)
            if op == "addnorm_bwd":
                case["onward"] = rng.random() < 0.7
        elif op == "gemv":
            case = dict(op=op, M=_log_int(rng, 1, 64), N=_log_int(rng, 16, 16384),
                        K=32 * _log_int(rng, 1, 512), fmt=rng.choice(("e2m1", "int4")),
                        group=rng.choice((32, 64, 128)), act=rng.choice(("bf16", "bf16", "e4m3")),
                        out=rng.choice(("bf16", "bf16", "fp32")))
        else:
            d = rng.choice(HEAD_DIMS)
            hk = _log_int(rng, 1, 40)
            case = dict(op=op, T=_log_int(rng, 1, 8192), hq=hk * rng.choice((1, 1, 2, 4, 8)), hk=hk,
                        d=d, rot=rng.choice((d, d, 16 * rng.randint(1, d // 16))),
                        naxes=rng.choice((2, 3, 3)), order=rng.choice(("sections", "cyclic")),
                        restart=rng.random() < 0.4, interleaved=rng.random() < 0.4,
                        packed=rng.random() < 0.6, far=rng.random() < 0.3, pad=rng.random() < 0.3,
                        by_axis=rng.random() < 0.5)
            if case["hq"] > 80:
                continue
        if _cost(case) <= most:
            return case


def work(case):
    op = case["op"]
    if op in ("axes", "axes_bwd"):
        values = case["T"] * (case["hq"] + case["hk"]) * case["d"]
        side = case["T"] * (8 * case["naxes"] + 4 * case["rot"]) + 8 * case["d"]
        if op == "axes":
            return {"bytes": 4 * values + side, "flops": 7 * values}
        return {"bytes": 6 * values + side + 8 * case["d"], "flops": 15 * values}
    if op in ("addnorm", "addnorm_bwd"):
        T, D = case["T"], case["D"]
        size = 2 if case["res"] == "bf16" else 4
        gain = 4 * D if case["gain"] else 0
        if op == "addnorm":     # x and the residual in; the sum, codes, scales and factors out
            return {"bytes": T * D * (3 + 2 * size) + 4 * T * -(-D // BLOCK) + gain + 4 * T,
                    "flops": 7 * T * D}
        # dy, the sum and the gradient from behind in; the gradient in the stream's type, and
        # in bf16 beside it, out
        n = 2 + size + (size if case["onward"] else 0) + size + (2 if size == 4 else 0)
        return {"bytes": T * D * n + 4 * T + 2 * gain, "flops": 11 * T * D}
    M, N, K = case["M"], case["N"], case["K"]
    a = M * K + 4 * M * -(-K // BLOCK) if case["act"] == "e4m3" else 2 * M * K
    size = 4 if case["out"] == "fp32" else 2
    return {"bytes": a + N * (K // 2 + 2 * -(-K // case["group"])) + size * M * N,
            "flops": 2 * M * N * K}


# ------------------------------------------------------------------ inputs

def _gen(seed, k=0):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 1013 + k)
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32)


def _activations(g, T, D):
    """N(0, 1) with one channel in a hundred twenty times as large."""
    x = _randn(g, T, D)
    big = torch.rand(D, generator=g, device=DEV) < 0.01
    return x.mul_(torch.where(big, 20.0, 1.0))


def _type(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def _addnorm_inputs(case, seed):
    g = _gen(seed)
    T, D, res = case["T"], case["D"], _type(case["res"])
    gamma = 1.0 + 0.1 * _randn(g, D) if case["gain"] else None
    if case["op"] == "addnorm":
        return dict(x=_randn(g, T, D).to(torch.bfloat16),
                    residual=_activations(g, T, D).mul_(2.0).to(res), gamma=gamma)
    h = _activations(g, T, D).mul_(2.0).to(res)
    rinv = torch.rsqrt(h.double().square().mean(-1) + EPS).float()
    return dict(dy=_randn(g, T, D).to(torch.bfloat16), h=h, rinv=rinv, gamma=gamma,
                onward=_randn(g, T, D).to(res) if case["onward"] else None)


def _blocks_of(v, size):
    """v [N, K] as [N, blocks, size], zeros behind the last value."""
    N, K = v.shape
    n = -(-K // size)
    return torch.nn.functional.pad(v, (0, n * size - K)).reshape(N, n, size)


def _group_codes(w, group, fmt):
    """fp32 w [N, K] -> (4-bit codes [N, K/2], the even value's in bits 0 to 3, bf16 scales)."""
    N, K = w.shape
    top = 6.0 if fmt == "e2m1" else 7.0
    b = _blocks_of(w, group)
    scales = (b.abs().amax(-1).clamp_min(AMAX_MIN) / top).to(torch.bfloat16)
    v = (b / scales.float()[..., None]).reshape(N, -1)[:, :K]
    if fmt == "e2m1":
        middles = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=DEV)
        codes = torch.bucketize(v.abs(), middles) + 8 * (v < 0)
    else:
        codes = v.round().clamp(-7, 7).long() & 15
    codes = codes.to(torch.uint8)
    return codes[:, 0::2] | codes[:, 1::2] << 4, scales


def _gemv_inputs(case, seed):
    g = _gen(seed)
    M, N, K = case["M"], case["N"], case["K"]
    w = _randn(g, N, K) * (0.5 * _randn(g, N, 1)).exp() * K ** -0.5
    state = {}
    state["w"], state["sw"] = _group_codes(w, case["group"], case["fmt"])
    a = _activations(g, M, K)
    if case["act"] == "bf16":
        state["a"] = a.to(torch.bfloat16)
        return state
    b = _blocks_of(a, BLOCK)
    state["sa"] = b.abs().amax(-1).clamp_min(AMAX_MIN) / E4M3_MAX
    codes = (b / state["sa"][..., None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    state["a"] = codes.view(torch.uint8).reshape(M, -1)[:, :K].contiguous()
    return state


def _axis_of_pairs(case):
    """The axis that turns each pair: runs of pairs for the axes one after another, or the axes
    in turn for as long as the shorter ones last."""
    half, n = case["rot"] // 2, case["naxes"]
    rest = half * 3 // 8 if n == 3 else half // 2   # pairs of each axis but the first
    if case["order"] == "sections":
        return [0] * (half - (n - 1) * rest) + [a for a in range(1, n) for _ in range(rest)]
    return [i % n if i < n * rest else 0 for i in range(half)]


def _table(P, case, axes, base=10000.0):
    """fp32 [P, rot]: the cosines of each pair's angle at each position, then the sines. A pair's
    frequency goes by its number among all pairs, or (restart) among its axis's."""
    half = case["rot"] // 2
    if case["restart"]:
        seen = [axes[:i].count(a) for i, a in enumerate(axes)]
        exponent = [s / axes.count(a) for s, a in zip(seen, axes)]
    else:
        exponent = [i / half for i in range(half)]
    freq = base ** -torch.tensor(exponent, device=DEV, dtype=torch.float64)
    angle = torch.arange(P, device=DEV, dtype=torch.float64)[:, None] * freq
    return torch.cat((angle.cos(), angle.sin()), dim=1).float()


def _positions(g, case):
    T, n = case["T"], case["naxes"]
    if case["far"]:     # every row its own far position, as in a decode batch
        P = 131072
        pos = torch.randint(0, P, (T, n), generator=g, device=DEV)
    else:               # text, its positions alike on all axes, then frames of rows and columns
        P = 8192
        text = T // 8
        i = torch.arange(T, device=DEV)
        j = (i - text).clamp_min(0)
        cols = max(1, math.isqrt(T // 4))
        grid = torch.stack((j // (cols * cols), j // cols % cols, j % cols), -1)[:, 3 - n:]
        pos = torch.where(i[:, None] < text, i[:, None], (text + grid).clamp_max(P - 1))
    if case["pad"]:     # the rows behind the last sequence
        pos[T - T // 8:] = -1
    # [T, axes], or kept as one row per axis
    return (pos.t().contiguous().t() if case["by_axis"] else pos.contiguous()), P


def _axes_inputs(case, seed):
    g = _gen(seed)
    T, d, hq, hk = case["T"], case["d"], case["hq"], case["hk"]
    pos, P = _positions(g, case)
    axes = _axis_of_pairs(case)
    state = dict(positions=pos, axes=bytes(axes), pair_axis=torch.tensor(axes, device=DEV),
                 table=_table(P, case, axes),
                 gamma_q=1.0 + 0.1 * _randn(g, d), gamma_k=1.0 + 0.1 * _randn(g, d))
    names = (("q", "k"), ("dyq", "dyk")) if case["op"] == "axes_bwd" else (("q", "k"),)
    for qn, kn in names:
        if case["packed"]:      # q and k are columns of the projection's output [q | k | v]
            qkv = _activations(g, T, (hq + 2 * hk) * d).to(torch.bfloat16)
            state[qn], state[kn] = qkv[:, :hq * d], qkv[:, hq * d:(hq + hk) * d]
        else:
            state[qn] = _activations(g, T, hq * d).to(torch.bfloat16)
            state[kn] = _activations(g, T, hk * d).to(torch.bfloat16)
    return state


def prepare(case, seed):
    make = {"addnorm": _addnorm_inputs, "addnorm_bwd": _addnorm_inputs, "gemv": _gemv_inputs,
            "axes": _axes_inputs, "axes_bwd": _axes_inputs}[case["op"]]
    return dict(make(case, seed), case=dict(case))


# ------------------------------------------------------------------- plain

def _plain_addnorm(st):
    h = (st["x"].float() + st["residual"].float()).to(st["residual"].dtype)
    v = h.float()
    rinv = torch.rsqrt((v * v).mean(-1, keepdim=True) + EPS)
    w = v * rinv if st["gamma"] is None else v * st["gamma"] * rinv
    b = _blocks_of(w, BLOCK)
    scales = b.abs().amax(-1).clamp_min(AMAX_MIN) / E4M3_MAX
    codes = (b * (1.0 / scales)[..., None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    codes = codes.view(torch.uint8).reshape(len(v), -1)[:, :v.shape[1]].contiguous()
    return [h, codes.view(torch.float8_e4m3fn), scales, rinv[:, 0]]


def _plain_addnorm_bwd(st):
    v, rinv = st["h"].float(), st["rinv"][:, None]
    n = v * rinv
    g = st["dy"].float()
    dgamma = None
    if st["gamma"] is not None:
        dgamma = (g * n).sum(0)
        g = g * st["gamma"]
    dh = (g - n * (g * n).mean(-1, keepdim=True)) * rinv
    if st["onward"] is not None:
        dh = dh + st["onward"].float()
    out = [dh.to(st["h"].dtype)]
    if st["h"].dtype is torch.float32:
        out.append(dh.to(torch.bfloat16))
    return out if dgamma is None else out + [dgamma]


def _values(codes, fmt):
    """fp32 values of 4-bit codes [N, K/2]."""
    c = torch.stack((codes & 15, codes >> 4), -1).flatten(1).long()
    table = E2M1 + tuple(-m for m in E2M1) if fmt == "e2m1" else tuple(range(8)) + tuple(range(-8, 0))
    return torch.tensor(table, device=DEV, dtype=torch.float32)[c]


def _plain_gemv(st):
    case = st["case"]
    K, group = case["K"], case["group"]
    w = _values(st["w"], case["fmt"]) * st["sw"].float().repeat_interleave(group, 1)[:, :K]
    if case["act"] == "bf16":
        a = st["a"].float()
    else:
        a = st["a"].view(torch.float8_e4m3fn).float() * st["sa"].repeat_interleave(BLOCK, 1)[:, :K]
    return (a @ w.t()).to(_type(case["out"]))


def _rotate(v, c, s, rot, interleaved, back):
    """Rotate the first rot values of v [T, h, d] by the angles of c, s [T, rot/2]."""
    c, s = c[:, None, :], (-s if back else s)[:, None, :]
    head, rest = v[..., :rot], v[..., rot:]
    if interleaved:
        a, b = head[..., 0::2], head[..., 1::2]
        return torch.cat((torch.stack((a * c - b * s, b * c + a * s), -1).flatten(-2), rest), -1)
    a, b = head[..., :rot // 2], head[..., rot // 2:]
    return torch.cat((a * c - b * s, b * c + a * s, rest), -1)


def _table_rows(st):
    """Each token's cosines and sines: a pair's from the row of the position on its axis."""
    half = st["case"]["rot"] // 2
    keep = (st["positions"] >= 0).all(1)
    rows = st["positions"].clamp_min(0)[:, st["pair_axis"]]
    i = torch.arange(half, device=DEV)
    return st["table"][rows, i], st["table"][rows, half + i], keep


def _plain_axes(st):
    case = st["case"]
    T, d, rot, il = case["T"], case["d"], case["rot"], case["interleaved"]
    c, s, keep = _table_rows(st)
    out = []
    for x, gamma in ((st["q"], st["gamma_q"]), (st["k"], st["gamma_k"])):
        v = x.float().reshape(T, -1, d)
        n = v * torch.rsqrt((v * v).mean(-1, keepdim=True) + EPS) * gamma
        y = _rotate(n, c, s, rot, il, False) * keep[:, None, None]
        out.append(y.reshape(T, -1).to(torch.bfloat16))
    return out


def _plain_axes_bwd(st):
    case = st["case"]
    T, d, rot, il = case["T"], case["d"], case["rot"], case["interleaved"]
    c, s, keep = _table_rows(st)
    dx, dg = [], []
    for x, dy, gamma in ((st["q"], st["dyq"], st["gamma_q"]), (st["k"], st["dyk"], st["gamma_k"])):
        v = x.float().reshape(T, -1, d)
        rinv = torch.rsqrt((v * v).mean(-1, keepdim=True) + EPS)
        n = v * rinv
        g = _rotate(dy.float().reshape(T, -1, d), c, s, rot, il, True) * keep[:, None, None]
        dg.append((g * n).sum((0, 1)))
        g = g * gamma
        dx.append(((g - n * (g * n).mean(-1, keepdim=True)) * rinv).reshape(T, -1).to(torch.bfloat16))
    return dx + dg


# --------------------------------------------------------------------- own

def _own(st):
    import normalization_token_split_gb300 as nts

    case = st["case"]
    op = case["op"]
    if op == "addnorm":
        o = nts.add_rmsnorm_blockcast(st["x"], st["residual"], st["gamma"], eps=EPS, want_rinv=True)
        return [o.h, o.codes.view(torch.float8_e4m3fn), o.scales, o.rinv]
    if op == "addnorm_bwd":
        out = nts.add_rmsnorm_backward(st["dy"], st["h"], st["rinv"], st["gamma"],
                                       dres=st["onward"])
        return [t for t in out if t is not None]
    if op == "gemv":
        return nts.gemv_groupscaled(st["a"], st["w"], st["sw"], a_scales=st.get("sa"),
                                    group=case["group"], fmt=case["fmt"], out_dtype=_type(case["out"]))
    a = (st["q"], st["gamma_q"], st["k"], st["gamma_k"], st["positions"], st["table"], st["axes"])
    if op == "axes":
        return nts.qknorm_rope_axes(*a, head_dim=case["d"], eps=EPS,
                                    interleaved=case["interleaved"])[:2]
    return nts.qknorm_rope_axes_backward(st["dyq"], st["dyk"], *a, head_dim=case["d"], eps=EPS,
                                         interleaved=case["interleaved"])


def run(state):
    if own:
        return _own(state)
    return {"addnorm": _plain_addnorm, "addnorm_bwd": _plain_addnorm_bwd, "gemv": _plain_gemv,
            "axes": _plain_axes, "axes_bwd": _plain_axes_bwd}[state["case"]["op"]](state)


# ------------------------------------------------------------------- exact

def _exact_addnorm(st):
    """The sum as it is stored (its one rounding is part of the definition); codes: the unrounded
    quotients by the block's scale."""
    kept = torch.add(st["x"].double(), st["residual"].double())
    kept = kept.float().to(st["residual"].dtype).double()
    D = kept.shape[1]
    rms = (kept.square().sum(1) / D + EPS).sqrt()
    w = kept / rms[:, None]
    if st["gamma"] is not None:
        w = w * st["gamma"].double()
    scales, values = [], []
    for part in w.split(BLOCK, 1):
        s = part.abs().amax(1).clamp(min=AMAX_MIN) / E4M3_MAX
        scales.append(s)
        values.append(part / s[:, None])
    return [kept, torch.cat(values, 1), torch.stack(scales, 1), rms.reciprocal()]


def _exact_addnorm_bwd(st):
    h, dy, rinv = st["h"].double(), st["dy"].double(), st["rinv"].double()
    u = dy if st["gamma"] is None else dy * st["gamma"].double()
    dot = torch.einsum("td,td->t", u, h) / h.shape[1]
    dh = torch.einsum("td,t->td", u, rinv) - torch.einsum("td,t->td", h, dot * rinv ** 3)
    if st["onward"] is not None:
        dh += st["onward"].double()
    out = [dh] if st["h"].dtype is torch.bfloat16 else [dh, dh]
    return out if st["gamma"] is None else out + [torch.einsum("td,td,t->d", dy, h, rinv)]


def _exact_gemv(st):
    """The sum over the even and the odd values of each group of the scaled partial products."""
    case = st["case"]
    group, half = case["group"], case["group"] // 2
    sign = torch.tensor([1.0, -1.0], device=DEV, dtype=torch.float64)
    mags = torch.tensor(E2M1, device=DEV, dtype=torch.float64)
    a = st["a"]
    a = a.double() if case["act"] == "bf16" else a.view(torch.float8_e4m3fn).double()
    y = torch.zeros(case["M"], case["N"], dtype=torch.float64, device=DEV)
    for j in range(st["sw"].shape[1]):
        packed = st["w"][:, j * half:(j + 1) * half].long()
        part = a[:, j * group:(j + 1) * group]
        for k, code in enumerate((packed % 16, packed // 16)):
            if case["fmt"] == "e2m1":
                v = mags[code % 8] * sign[code // 8]
            else:
                v = ((code + 8) % 16 - 8).double()
            # the group lies inside one block of 128 activations
            s = 1.0 if case["act"] == "bf16" else st["sa"][:, j * group // BLOCK, None].double()
            y += (part[:, k::2] * s) @ (v * st["sw"][:, j, None].double()).t()
    return y


def _exact_axes(st):
    """Each rotated pair as one complex number, times exp(i angle) (forward) or its conjugate."""
    case = st["case"]
    T, d, rot, half = case["T"], case["d"], case["rot"], case["rot"] // 2
    order = torch.arange(rot, device=DEV)
    order = order.reshape(half, 2).t() if case["interleaved"] else order.reshape(2, half)
    ok = (st["positions"].amin(1) >= 0).nonzero()[:, 0]
    turn = torch.empty(len(ok), 1, half, dtype=torch.complex128, device=DEV)
    for a in set(st["axes"]):
        mine = (st["pair_axis"] == a).nonzero()[:, 0]
        tab = st["table"][st["positions"][ok, a]].double()
        turn[:, 0, mine] = torch.complex(tab[:, mine], tab[:, half + mine])

    def rotated(v, z):
        pairs = torch.complex(v[..., order[0]], v[..., order[1]]) * z
        v = v.clone()
        v[..., order[0]], v[..., order[1]] = pairs.real, pairs.imag
        return v

    def whole(v, width):
        y = torch.zeros(T, width, dtype=torch.float64, device=DEV)
        y[ok] = v.reshape(len(ok), width)
        return y

    if case["op"] == "axes":
        out = []
        for x, gamma in ((st["q"], st["gamma_q"]), (st["k"], st["gamma_k"])):
            v = x.double()[ok].reshape(len(ok), -1, d)
            rms = torch.sqrt(v.square().sum(-1, keepdim=True) / d + EPS)
            out.append(whole(rotated(v / rms * gamma.double(), turn), x.shape[1]))
        return out
    dx, dg = [], []
    for x, dy, gamma in ((st["q"], st["dyq"], st["gamma_q"]), (st["k"], st["dyk"], st["gamma_k"])):
        v = x.double()[ok].reshape(len(ok), -1, d)
        rms = torch.sqrt(v.square().sum(-1, keepdim=True) / d + EPS)
        g = rotated(dy.double()[ok].reshape(len(ok), -1, d), turn.conj())
        dg.append(torch.einsum("thd,thd->d", g, v / rms))
        u = g * gamma.double()
        dot = torch.einsum("thd,thd->th", u, v)[..., None]
        dx.append(whole(u / rms - v * dot / (d * rms ** 3), x.shape[1]))
    return dx + dg


def exact(case, seed):
    state = prepare(case, seed)
    return {"addnorm": _exact_addnorm, "addnorm_bwd": _exact_addnorm_bwd, "gemv": _exact_gemv,
            "axes": _exact_axes, "axes_bwd": _exact_axes}[case["op"]](state)
