"""Outputs of the gated delta rule where what they sum nearly cancels: they hold
the last bits of the fp32 states, updates and products that they are made of,
whether a call runs token by token or in chunks."""
import pytest
import torch

import block_refs as ref
import mamba_ssd_scan_06_amd as ssd
from test_gpu_gated_delta import ranges_of
from test_gpu_layer_ops import TD, announce, f64

pytestmark = pytest.mark.gpu

# Its last bit stands two below the eight of a bf16 fraction, so that of
# BIG + 2^-20 neither one bf16 holds the 2^-20 nor what a second one has room for.
BIG = 1 + 2.0 ** -9


def empty(b, T, H, P, N, dtype, lead=0):
    """Zeros throughout: q, k, v start `lead` elements into their rows."""
    def rows(n, inner):
        full = torch.zeros(b, T, lead + n * inner, dtype=TD[dtype], device="cuda")
        return full[:, :, lead:].unflatten(2, (n, inner))

    return dict(q=rows(1, N), k=rows(1, N), v=rows(H, P), g=None, beta=torch.zeros(b, T, H, device="cuda"))


@pytest.mark.parametrize("dtype,lead", [("bf16", 0), ("bf16", 1), ("f32", 0)])
@pytest.mark.parametrize("N", [16, 48, 80, 128, 144, 192, 208, 256])
@pytest.mark.parametrize("T", [9, 70])
def test_state_under_a_query(T, N, dtype, lead):
    # The state stands still (beta 0).  Row p holds BIG + (p + 1) 2^-20 and -BIG, each
    # query picks such a pair: every partial sum is a multiple of 2^-20 below 2, so
    # exact in 24 bits, and so is the output's rounding of a number up to 64 = 2^6.
    announce(T, N, dtype, lead)
    P = 64
    s = empty(2, T, 2, P, N, dtype, lead)
    small = (torch.arange(P, device="cuda") + 1.0) * 2.0 ** -20
    init = torch.zeros(2, 2, P, N, device="cuda")
    init[..., 0::2] = BIG + small[:, None]
    init[..., 1::2] = -BIG
    for t in range(T):
        n = 2 * (t % (N // 2))
        s["q"][:, t, :, n:n + 2] = 1.0
    y, fin, _ = ssd.ssd_gated_delta_fwd(**s, init_state=init, scale=1.0)
    torch.cuda.synchronize()
    assert torch.equal(fin, init)
    assert torch.equal(y.float(), small.expand(2, T, 2, P))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_state_under_a_query_in_ranges(dtype):
    T, P, N = 1300, 16, 32
    assert ranges_of(1, T, 1, P, N, 1, dtype) >= 3
    s = empty(1, T, 1, P, N, dtype)
    small = (torch.arange(P, device="cuda") + 1.0) * 2.0 ** -20
    init = torch.zeros(1, 1, P, N, device="cuda")
    init[..., 3], init[..., 20] = BIG + small, -BIG
    s["q"][..., [3, 20]] = 1.0
    y, fin, _ = ssd.ssd_gated_delta_fwd(**s, init_state=init, scale=1.0)
    torch.cuda.synchronize()
    assert torch.equal(fin, init)
    assert torch.equal(y.float(), small.expand(1, T, 1, P))


PAIRS = [(0, 1), (2, 13), (3, 20), (17, 30), (16, 31)]


@pytest.mark.parametrize("dtype,lead", [("bf16", 0), ("bf16", 1), ("f32", 0)])
@pytest.mark.parametrize("first,second", PAIRS)
def test_updates_of_one_chunk(first, second, dtype, lead):
    # Two tokens write under keys of their own, BIG + (h + 1) 2^-20 and -BIG (beta's
    # values); every query from the second on sums both: exact, as above.
    announce(first, second, dtype, lead)
    T, H, P, N = 40, 4, 80, 64
    s = empty(2, T, H, P, N, dtype, lead)
    small = (torch.arange(H, device="cuda") + 1.0) * 2.0 ** -20
    s["k"][:, first, :, 5] = s["k"][:, second, :, 44] = 1.0
    s["v"][:, first], s["v"][:, second] = 1.0, -1.0
    s["beta"][:, first], s["beta"][:, second] = BIG + small, BIG
    s["q"][:, second:, :, [5, 44]] = 1.0
    y, fin, _ = ssd.ssd_gated_delta_fwd(**s, scale=1.0)
    torch.cuda.synchronize()
    assert torch.equal(fin[..., 5], (BIG + small)[None, :, None].expand(2, H, P)) and (fin[..., 44] == -BIG).all()
    assert not y[:, :second].any()
    assert torch.equal(y[:, second:].float(), small[None, None, :, None].expand(2, T - second, H, P))


@pytest.mark.parametrize("dtype,lead", [("bf16", 0), ("bf16", 1), ("f32", 0)])
@pytest.mark.parametrize("first,second", PAIRS)
def test_decayed_products_of_one_chunk(first, second, dtype, lead):
    # The same with beta 1 and a small decay at the second token: y = e^g - 1.  An
    # exponential of one unit (2^-23), a sum of decays of half a unit, two products
    # and two sums of numbers below 2 (2^-24 each): under 2^-21 in all.
    announce(first, second, dtype, lead)
    T, H, P, N = 32, 4, 80, 64
    s = empty(2, T, H, P, N, dtype, lead)
    s["k"][:, first, :, 5] = s["k"][:, second, :, 44] = 1.0
    s["v"][:, first], s["v"][:, second] = 1.0, -1.0
    s["beta"][:, [first, second]] = 1.0
    s["g"] = torch.zeros(2, T, H, device="cuda")
    s["g"][:, second] = -0.7 * 2.0 ** -13 * (torch.arange(H, device="cuda") + 1)
    s["q"][:, second:, :, [5, 44]] = 1.0
    y, _, _ = ssd.ssd_gated_delta_fwd(**s, scale=1.0)
    torch.cuda.synchronize()
    want = torch.expm1(s["g"][:, second].double()).cpu().numpy()[:, None, :, None]
    bound = 2.0 ** -21 + ref.HALF_STEP[dtype] * abs(want)
    worst = (abs(f64(y[:, second:]) - want) / bound).max()
    print(f"  worst element {worst:.2f} of its bound", flush=True)
    assert worst <= 1
