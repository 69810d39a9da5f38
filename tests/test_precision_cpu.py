"""The bounds of test_gpu_window_precision catch what they are there for: mistakes planted in the 64-bit reference."""
import torch

from tests import test_gpu_window_precision as w


def test_two_bf16_parts_would_fail_the_weight_bound():
    s = w.two_token_case().double()
    top = s.clamp(min=0.0)
    p = torch.exp2((s - top) * 1.4426950408889634).float()     # the second token's weight, in 32 bits
    hi = p.bfloat16().float()
    lo = (p - hi).bfloat16().float()
    total = p.double() + torch.exp(-top)
    got, want = (hi.double() + lo.double()) / total, torch.sigmoid(s)
    for dtype in ("bf16", "f16"):
        bound = w.weight_bound(dtype, s.abs(), 2)[..., 0] * want + 2.0 ** -24 * want
        assert ((got - want).abs() > bound).double().mean() > 0.02
    third = (p - hi - lo).bfloat16()
    got = (hi.double() + lo.double() + third.double()) / total
    assert ((got - want).abs() <= w.weight_bound("bf16", s.abs(), 2)[..., 0] * want).all()


def test_approximate_step_factors_would_fail_the_rotation_bound():
    """Step factors off by up to 2^-21.4, as __sincosf's may be, in an otherwise exact recurrence."""
    d, ctx, g = 128, 256, torch.Generator().manual_seed(1)
    theta = 1e4 ** (-torch.arange(0, d, 2).double() / d)
    off = (torch.rand((2, d // 2), generator=g).double() * 2 - 1) * 2.0 ** -21.4
    t = torch.arange(ctx)
    step = torch.complex(torch.cos(4 * theta) + off[0], torch.sin(4 * theta) + off[1])
    turn = torch.polar(torch.ones(ctx, d // 2, dtype=torch.float64), (t % 4).double()[:, None] * theta)
    k = turn * step[None] ** (t // 4)[:, None]
    q = torch.polar(torch.ones(d // 2, dtype=torch.float64), ctx * theta)
    exact = torch.cos((ctx - t).double()[:, None] * theta)
    p, want = (torch.softmax(w.SCORE * x, 0) for x in ((q.conj() * k).real, exact))
    p, want = (x.view(2, d, d // 2).sum(0) for x in (p, want))     # v of token t is the unit vector t mod D
    rms = (p / want - 1).pow(2).mean().sqrt()
    assert rms > 1.5 * (2 ** 0.5 * w.ROTATION_RMS * w.SCORE + 5e-7), rms
