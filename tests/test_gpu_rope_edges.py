"""The rotation's gradient of heads whose sum of squares is beyond fp32."""
import pytest
import torch

pytestmark = pytest.mark.gpu

nts = pytest.importorskip("normalization_token_split_gb300")
DEV = "cuda:0"


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("axes", [False, True])
@pytest.mark.parametrize("T", [5, 3000])          # direct loads, a ring
def test_heads_beyond_fp32(T, axes, interleaved):
    """Such a head's rinv is 0: it gets zeros, adds nothing to dgamma, and the other heads'
    values are what they are beside a head of zeros (which adds nothing either).  Head 0's
    sum of u x is infinite, head 2's has infinite parts of both signs."""
    d, hq, hk = 64, 4, 2
    g = torch.Generator(device=DEV).manual_seed(T)

    def randn(*shape):
        return torch.randn(*shape, generator=g, device=DEV).to(torch.bfloat16)

    q, k, dyq, dyk = (randn(T, h * d) for h in (hq, hk, hq, hk))
    gain, table = torch.rand(d, generator=g, device=DEV) + 0.5, nts.rope_table(64, d)
    pos = torch.arange(T, device=DEV) % 64
    rows = [0, T // 2, T - 1]
    zeros, far = q.view(T, hq, d).clone(), q.view(T, hq, d).clone()
    dy = dyq.view(T, hq, d)
    for t in rows:
        zeros[t, 0], zeros[t, 2] = 0, 0
        dy[t, 0] = 2                              # turned, g is dy's size and of both signs
        far[t, 0] = 3e38 * torch.sign(torch.randn(d, generator=g, device=DEV))
        far[t, 2] = 3e38

    def call(x):
        x = x.reshape(T, -1)
        if axes:
            p = torch.stack((pos, pos.flip(0)), -1)
            return nts.qknorm_rope_axes_backward(dyq, dyk, x, gain, k, gain, p, table,
                                                 nts.rope_axes((16, 16)), d, interleaved=interleaved)
        return nts.qknorm_rope_backward(dyq, dyk, x, gain, k, gain, pos, table, d,
                                        interleaved=interleaved)

    want, got = call(zeros), call(far)
    nts.check_status()
    dq, wq = got[0].view(T, hq, d), want[0].view(T, hq, d).clone()
    for t in rows:
        assert not dq[t, 0].any() and not dq[t, 2].any()
        wq[t, 0], wq[t, 2] = 0, 0
    assert torch.equal(dq, wq)
    for a, b in zip(got[1:], want[1:]):
        assert torch.equal(a, b)
