"""Log decays that empty the state of the gated delta rule, from just beyond the
exponential's range down to -inf, on the GPU against its definition in fp64: what
follows them decays as without them, token by token and in chunks."""
import numpy as np
import pytest
import torch

import block_refs as ref
import mamba_ssd_scan_06_amd as ssd
from test_gpu_gated_delta import check, inputs, ranges_of
from test_gpu_layer_ops import announce

pytestmark = pytest.mark.gpu

RESETS = [-1e3, -1e5, -1e9, -1e14, -1e16, -1e30, float(np.finfo(np.float32).min), -float("inf")]


def with_resets(s, value, at):
    """Resets at `at` in the first head, one token later in each further head, and
    several in a row in the last."""
    s["g"] = s["g"].clone()
    T, H = s["g"].shape[1:]
    for h in range(H):
        for t in at:
            s["g"][:, min(t + h, T - 1), h] = value
    s["g"][:, at[0]:at[0] + 4, H - 1] = value
    return s


@pytest.mark.parametrize("dtype,lead", [("bf16", 0), ("bf16", 1), ("f32", 0)])
@pytest.mark.parametrize("T,at", [(10, (0,)), (10, (4,)), (60, (0, 32)), (60, (7, 30)), (100, (14, 44, 93))])
@pytest.mark.parametrize("value", RESETS)
def test_resets(value, T, at, dtype, lead):
    announce(value, T, at, dtype, lead)
    s = with_resets(inputs(40, 5, T, 4, 48, 64, 2, dtype, lead=lead, unit=True), value, at)
    # The accepted index on, before and after the first reset.
    s["state_out_idx"] = torch.tensor([at[0], at[0] - 1, at[0] + 3, T - 1, T // 2], dtype=torch.int32, device="cuda")
    check(s, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("value", RESETS)
def test_resets_in_ranges(value, dtype):
    announce(value, dtype)
    b, T, H, P, N, G = 2, 1300, 2, 32, 64, 1
    assert ranges_of(b, T, H, P, N, G, dtype) >= 3
    s = inputs(41, b, T, H, P, N, G, dtype, unit=True)
    s["g"] = s["g"] * 0.02
    with_resets(s, value, (5, 640, 700))
    s["state_out_idx"] = torch.tensor([645, T - 1], dtype=torch.int32, device="cuda")
    check(s, dtype, tol=3 * ref.delta_tolerance(N))


@pytest.mark.parametrize("T", [12, 40])
def test_nan_decays_stay_nan(T):
    s = inputs(42, 2, T, 2, 32, 64, 1, "bf16", unit=True, idx=False)
    want, _, _ = ssd.ssd_gated_delta_fwd(**s)
    s["g"] = s["g"].clone()
    s["g"][1, 3, 0] = float("nan")
    y, fin, _ = ssd.ssd_gated_delta_fwd(**s)
    torch.cuda.synchronize()
    assert torch.isnan(fin[1, 0]).all() and torch.isnan(y[1, 3:, 0].float()).all()
    assert torch.equal(y[0], want[0]) and torch.equal(y[1, :, 1], want[1, :, 1])


@pytest.mark.parametrize("T", [12, 40])
def test_growth_after_a_reset(T):
    # What a reset removes does not come back, however much follows: e^30 here,
    # within the range of fp32.
    s = inputs(43, 2, T, 2, 32, 64, 1, "f32", unit=True)
    s["g"] = torch.zeros_like(s["g"])
    s["g"][:, 2], s["g"][:, 5] = -200.0, 30.0
    s["beta"][:, 2:6] = 0.0
    s["init_state"] = s["init_state"] * 1e3
    check(s, "f32")
