"""The gated delta rule with so many chunks that one wave prepares several heads of
a group, which share their keys and queries but not their decays, betas and values."""
import pytest
import torch

import block_refs as ref
import mamba_ssd_scan_06_amd as ssd
from test_gpu_gated_delta import check, inputs, ranges_of
from test_gpu_layer_ops import announce

pytestmark = pytest.mark.gpu


def heads_per_wave(b, T, H, G):
    """As many heads of a group as leave two waves per SIMD (2 x 1024)."""
    chunks, each = b * -(-T // 32), H // G
    return max([1] + [d for d in range(2, min(each, 8) + 1) if each % d == 0 and chunks * (H // d) >= 2048])


CASES = [
    # heads per wave, b, T, H, P, N, G, lead
    (2, 16, 300, 32, 16, 32, 8, 0),
    (2, 16, 300, 32, 16, 32, 4, 1),
    (2, 70, 100, 16, 32, 144, 8, 0),
    (3, 52, 300, 12, 16, 32, 4, 0),
    (4, 16, 300, 64, 16, 32, 8, 0),
    (5, 52, 300, 20, 16, 16, 4, 3),
    (6, 35, 300, 36, 16, 48, 6, 0),
    (7, 30, 300, 49, 16, 32, 7, 0),
    (8, 26, 300, 64, 16, 32, 8, 0),
    (8, 86, 97, 64, 32, 64, 4, 0),
]


@pytest.mark.parametrize("dtype,l2", [("bf16", True), ("f32", False)])
@pytest.mark.parametrize("case", CASES, ids=["-".join(map(str, c)) for c in CASES])
def test_heads_of_a_wave(case, dtype, l2):
    d, b, T, H, P, N, G, lead = case
    announce(*case, dtype, l2)
    assert heads_per_wave(b, T, H, G) == d
    s = inputs(50, b, T, H, P, N, G, dtype, lead=lead, unit=not l2)
    # Heads of a group are told apart: none decays, betas and values as its neighbour.
    assert all(not torch.equal(s[k][:, :, h], s[k][:, :, h + 1]) for k in ("g", "beta", "v") for h in range(H - 1))
    check(s, dtype, l2=l2)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_heads_of_a_wave_in_ranges(dtype):
    b, T, H, P, N, G = 1, 16401, 8, 16, 32, 1
    announce(dtype)
    assert heads_per_wave(b, T, H, G) == 2 and ranges_of(b, T, H, P, N, G, dtype) >= 3
    s = inputs(51, b, T, H, P, N, G, dtype)
    s["g"] = s["g"] * 0.005                           # a range's state reaches the next one
    s["state_out_idx"] = torch.tensor([9000], dtype=torch.int32, device="cuda")
    check(s, dtype, l2=True, tol=3 * ref.delta_tolerance(N))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_heads_of_a_wave_without_decay(dtype):
    s = inputs(52, 16, 300, 32, 16, 32, 8, dtype, decay=False, init=False, unit=True)
    check(s, dtype)


def test_the_same_bits_as_alone():
    # A sequence's outputs do not depend on how many heads its waves prepare.
    assert heads_per_wave(52, 300, 20, 4) == 5 and heads_per_wave(1, 300, 20, 4) == 1
    s = inputs(53, 52, 300, 20, 16, 32, 4, "bf16", idx=False)
    y, fin, _ = ssd.ssd_gated_delta_fwd(**s, qk_l2norm=True)
    for i in (0, 17, 51):
        one = {k: None if t is None else t[i:i + 1] for k, t in s.items()}
        y1, fin1, _ = ssd.ssd_gated_delta_fwd(**one, qk_l2norm=True)
        torch.cuda.synchronize()
        assert torch.equal(y[i:i + 1], y1) and torch.equal(fin[i:i + 1], fin1)
