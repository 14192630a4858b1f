"""The selective scan where a token range's decay grows instead of shrinking
(A > 0, or negative steps without softplus): a range's growth factor may pass
the fp32 range while the states stay inside it.  Every length here is run in
token ranges, whose lengths are whole tiles of 32 tokens.

The bound of layer_refs covers a range's joined decay too: of one exponential
in place of 32 or more it asks one rounding in the exponent more (the sum of
steps, |x| U, with |x| below 128 U in these tests) and 2 U per token less."""
import numpy as np
import pytest
import torch

import layer_refs as ref
import mamba_ssd_scan_06_amd as ssd
from test_gpu_layer_ops import announce, close, f64, gen, run_scan, scan_inputs

pytestmark = pytest.mark.gpu


def growing(dt, N, T=600, Dm=72, G=1):
    """Inputs of one sequence with steps of zero, for a test to fill in."""
    s = scan_inputs(gen(81), 1, T, Dm, N, G, dt, False, True, True, True, 0)
    s["u"] = s["u"].clone()
    s["delta"] = torch.zeros_like(s["delta"])
    return s


def check(s, dt, js=None):
    idx = None if js is None else torch.from_numpy(js).cuda()
    shape = ssd.ssd_selective_shape(1, s["u"].shape[1], s["u"].shape[2], s["A"].shape[1], s["B"].shape[2])
    assert ssd.ssd_selective_scan_workspace_bytes(shape, ssd.SSD_DTYPE_BF16 if dt == "bf16" else ssd.SSD_DTYPE_F32) > 0
    y, fin, at = run_scan(s, False, idx)
    torch.cuda.synchronize()
    wy, by, wf, bf, wa, ba = ref.selective_scan(f64(s["u"]), f64(s["delta"]), f64(s["A"]), f64(s["B"]), f64(s["C"]),
                                                f64(s["D"]), f64(s["z"]), None, False, f64(s["init"]), js, dt)
    assert np.abs(wf).max() < 1e30
    close("y", y, wy, by)
    close("final_state", fin, wf, bf)
    if js is not None:
        close("state_out", at, wa, ba)


@pytest.mark.parametrize("dt,N,sign", [("bf16", 8, 1), ("f32", 16, 1), ("bf16", 16, -1), ("f32", 32, 1), ("f32", 64, -1),
                                       ("bf16", 64, 1)])
def test_zero_states_stay_zero_while_the_decay_grows(dt, N, sign):
    # Left padding: no input and no state until token 300, but steps whose
    # exponents add up to 100 .. 200 in each range before it.
    announce(dt, N, sign)
    s = growing(dt, N)
    g = gen(82)
    s["A"] = sign * (4 + 2 * torch.rand(s["A"].shape, generator=g)).cuda()
    s["u"][:, :300] = 0
    s["init"] = None
    s["delta"][:, :300] = sign * 1.0                     # 32 tokens: 128 .. 192 in the exponent
    s["delta"][:, 300:] = sign * 2.0 ** -6
    check(s, dt, np.array([450], np.int32))


@pytest.mark.parametrize("dt,N,sign", [("f32", 8, 1), ("bf16", 16, 1), ("f32", 64, -1)])
def test_small_states_outgrow_one_factor(dt, N, sign):
    # States of 1e-30 grow by e^92 .. e^120 within one range and its
    # neighbour (e^88 is beyond fp32), later shrink again: finite throughout.
    announce(dt, N, sign)
    s = growing(dt, N)
    g = gen(83)
    s["A"] = sign * (0.92 + 0.2 * torch.rand(s["A"].shape, generator=g)).cuda()
    s["init"] = s["init"] * 1e-30
    s["u"][:] = 0
    s["delta"][:, 32:64] = sign * 3.125                  # one tile: the exponent gains 92 .. 112
    s["delta"][:, 400:420] = -sign * 2.5                 # and loses 46 .. 56 again
    check(s, dt, np.array([399], np.int32))


def test_an_infinite_decay_forgets_the_range_before():
    # A of -inf and finite steps: h is the last input's share alone, also
    # where a range starts.
    s = growing("f32", 16)
    s["A"] = s["A"].clone()
    s["A"][3] = -float("inf")
    s["A"][5, 7] = -float("inf")
    s["delta"][:] = 0.25
    y, fin, _ = run_scan(s, False)
    torch.cuda.synchronize()
    assert torch.isfinite(y).all() and torch.isfinite(fin).all()
    last = 0.25 * s["u"][0, -1, 3] * s["B"][0, -1, 0]
    assert torch.equal(fin[0, 3], last)
    assert fin[0, 5, 7] == 0.25 * s["u"][0, -1, 5] * s["B"][0, -1, 0, 7]
