"""The gated delta rule for a few tokens on both sides of its choice of one or two
rows of the state per lane: head sizes that fill 64 rows, leave a third, a quarter
or half of them empty, and calls of few and many workgroups."""
import pytest
import torch

import mamba_ssd_scan_06_amd as ssd
from test_gpu_gated_delta import check, inputs
from test_gpu_layer_ops import announce

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("b,T,H,P,N,dtype", [
    (18, 5, 64, 32, 128, "f32"), (18, 5, 64, 48, 96, "f32"), (9, 5, 64, 80, 128, "f32"), (9, 5, 64, 96, 112, "bf16"),
    (18, 5, 64, 96, 32, "bf16"), (18, 3, 64, 96, 64, "f32"), (6, 5, 64, 160, 128, "f32"), (9, 5, 64, 128, 160, "f32"),
    (9, 4, 64, 112, 192, "bf16"),
])
def test_rows_per_lane(b, T, H, P, N, dtype):
    announce(b, T, H, P, N, dtype)
    s = inputs(60, b, T, H, P, N, 8, dtype, idx=True)
    y, fin, at = check(s, dtype, l2=True)
    # A row's sums are the same whichever lane holds it: the bits of one sequence
    # alone, whose few workgroups take one row per lane.
    one = {k: t[b - 1:] for k, t in s.items()}
    for all_, alone in zip((y, fin, at), ssd.ssd_gated_delta_fwd(**one, qk_l2norm=True)):
        torch.cuda.synchronize()
        assert torch.equal(all_[b - 1:], alone)
