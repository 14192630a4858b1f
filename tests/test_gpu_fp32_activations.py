"""softplus and silu of the operators around the scan in fp32, each seen alone
through an entry point: sizes, weights and states are chosen so that every
other product is by 1 and every other sum with 0.

Bounds in roundings of U = 2^-24 of the value, none of which grows with the
argument: exp(-|x|) takes the hardware exponential's unit in the last place
(2 U) and one rounding of its correction (1 U); below 2^-126 the exponential
flushes to zero.
    softplus = max(x, 0) + e Q(e): e 3 U; Q's coefficients 8e-9 (0.14 U), its
    last two sums 2 U (Q is 0.69 at least; the second enters with e / 2 of it at
    most); the last multiply-add 1 U: below 8 U.
    silu = x e / (1 + e) or x / (1 + e): e 3 U, the product 1 U, the corrected
    reciprocal 1 U and its correction's own roundings (second order), the last
    product 1 U: below 7 U.
"""
import numpy as np
import pytest
import torch

import mamba_ssd_scan_06_amd as ssd

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
FLUSHED = 2.0 ** -126


def arguments(n, lo=-80.0, hi=40.0):
    """n fp32 values over [lo, hi], dense around the ordinary ones."""
    g = torch.Generator()
    g.manual_seed(7)
    wide = lo + (hi - lo) * torch.rand(n // 2, generator=g)
    return torch.cat([wide, 3.0 * torch.randn(n - n // 2, generator=g)]).clamp(lo, hi)


def within(name, got, want, x, roundings, floor):
    got = got.detach().double().cpu().numpy().ravel()
    err = np.maximum(np.abs(got - want) - floor, 0.0) / np.abs(want) / U
    k = int(np.argmax(err))
    print(f"\n  {name}: worst {err[k]:.2f} U at {x[k]!r}, rms {np.sqrt((err ** 2).mean()):.3f} U", flush=True)
    assert err[k] <= roundings, f"{name}({x[k]!r}): {err[k]:.1f} roundings off: got {got[k]!r}, want {want[k]!r}"


def softplus64(x):
    return np.logaddexp(x, 0.0)


def silu64(x):
    return np.where(x >= 0, x / (1.0 + np.exp(-np.abs(x))), x * np.exp(-np.abs(x)) / (1.0 + np.exp(-np.abs(x))))


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("T", [1, 20])
def test_softplus_of_the_scan(dt, T):
    # One token with u = B = 1 from a zero state: the state is the step.  A
    # call of 20 tokens (another kernel) asks for the state after token 0.
    # States are fp32 whatever the inputs' type.
    Dm, N = 4096, 16
    x = arguments(Dm).to(torch.bfloat16 if dt == "bf16" else torch.float32)
    delta = x.view(1, 1, Dm).repeat(1, T, 1).cuda()
    one = torch.ones_like(delta)
    B = torch.ones(1, T, 1, N, dtype=x.dtype, device="cuda")
    idx = torch.zeros(1, dtype=torch.int32, device="cuda")
    _, _, at = ssd.ssd_selective_scan_fwd(one, delta, torch.full((Dm, N), -1.0, device="cuda"), B, B,
                                          state_out_idx=idx, delta_softplus=True)
    torch.cuda.synchronize()
    x = x.double().numpy()
    assert torch.equal(at[..., :1].expand_as(at), at)
    within("softplus", at[0, :, 0], softplus64(x), x, 8.0, FLUSHED)


@pytest.mark.parametrize("T", [1, 20])
def test_silu_of_the_scan(T):
    # A zero state (B = 0) and u = D = 1: y is silu(z).
    Dm, N = 4096, 16
    x = arguments(Dm)
    z = x.view(1, 1, Dm).repeat(1, T, 1).cuda()
    zero = torch.zeros(1, T, 1, N, device="cuda")
    y, _, _ = ssd.ssd_selective_scan_fwd(torch.ones_like(z), torch.ones_like(z),
                                         torch.full((Dm, N), -1.0, device="cuda"), zero, zero,
                                         torch.ones(Dm, device="cuda"), z)
    torch.cuda.synchronize()
    x = x.double().numpy()
    within("silu", y[0, T - 1], silu64(x), x, 7.0, 80 * FLUSHED)


def test_silu_of_the_convolution():
    # Taps 0 and 1: the sum is the input itself.
    x = arguments(8192)
    w = torch.tensor([[0.0, 1.0]]).repeat(64, 1).cuda()
    out, _, _ = ssd.ssd_causal_conv_fwd(x.view(1, 128, 64).cuda(), w)
    torch.cuda.synchronize()
    x = x.double().numpy()
    within("silu", out, silu64(x), x, 7.0, 80 * FLUSHED)


def test_silu_of_the_norm():
    # x = 1 and eps = 0: the scale is 1 and the output silu(z).
    z = arguments(8192).view(64, 128)
    out = ssd.ssd_gated_norm_fwd(torch.ones(64, 128, device="cuda"), z.cuda(), eps=0.0, norm_before_gate=True)
    torch.cuda.synchronize()
    x = z.double().numpy().ravel()
    within("silu", out, silu64(x), x, 7.0, 80 * FLUSHED)


def test_activations_at_the_ends():
    # Beyond the exponential's range the limits, NaN stays NaN (by the way of
    # the convolution and of the scan's step).
    inf, nan = float("inf"), float("nan")
    x = torch.tensor([inf, 200.0, 90.0, 0.0, -0.0, -90.0, -104.0, -200.0, -3e38, 3e38, nan])
    w = torch.tensor([[0.0, 1.0]]).repeat(len(x), 1).cuda()
    out, _, _ = ssd.ssd_causal_conv_fwd(x.view(1, 1, -1).cuda(), w)
    got = out.cpu().view(-1)
    assert got[0] == inf and got[1] == 200.0 and got[2] == 90.0 and got[3] == 0.0 and got[4] == 0.0
    assert (got[5:9].abs() < 1e-35).all() and (got[5:9] <= 0).all()
    assert got[9] == x[9] and torch.isnan(got[10])
    ones = torch.ones(1, 1, len(x), device="cuda")
    B = torch.ones(1, 1, 1, 8, device="cuda")
    _, fin, _ = ssd.ssd_selective_scan_fwd(ones, x.view(1, 1, -1).cuda(), torch.full((len(x), 8), -1.0, device="cuda"), B,
                                           B, delta_softplus=True)
    got = fin.cpu()[0, :, 0]
    # With an infinite or huge step the empty state's decay is 0, 0 * 0 = 0.
    assert got[0] == inf and got[1] == 200.0 and got[2] == 90.0
    assert abs(got[3].item() - 0.6931471805599453) <= 8 * U * 0.6931471805599453 and got[4] == got[3]
    assert (got[5:9] >= 0).all() and (got[5:9] < 1e-38).all() and got[9] == x[9] and torch.isnan(got[10])
