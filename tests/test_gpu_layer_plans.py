"""Launch plans of the operators around the scan that only larger calls take:
the convolution's long token runs, the norm's four and five pieces per thread,
wide states in tiles and ranges, and draft verification in two launches with
residuals that leave nothing."""
import numpy as np
import pytest
import torch

import layer_refs as ref
import mamba_ssd_scan_06_amd as ssd
from test_gpu_layer_ops import announce, close, f64, gen, ref_scan, rnd, run_scan, same, scan_inputs, verify_inputs

pytestmark = pytest.mark.gpu


# A run is 32 tokens where (vectors of 16 bytes) x runs x sequences reach
# 131072 that way, else 16 where that many runs do.  T ends inside a batch of
# eight.
@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("run,T,ch", [
    (32, 2037, 1024),       # whole vectors
    (32, 2037, 1021),       # a partial last vector, rows at odd offsets
    (16, 1003, 1024),
])
def test_conv_long_runs(W, dt, run, T, ch):
    vec = 8 if dt == "bf16" else 4
    threads = lambda length, b: -(-ch // vec) * -(-T // length) * b
    b = next(b for b in range(1, 200) if threads(32, b + (run == 16)) >= 131072)
    assert threads(run, b) >= 131072 and (run == 32 or threads(32, b) < 131072)
    announce(W, dt, run, T, ch, b)
    g = gen(91 + W)
    # Two sequences against fp64, the others (copies of them) by equality.
    copies = torch.arange(b, device="cuda") % 2
    wide = rnd(g, (2, T, ch + 2 * (ch % 2)), dt)[copies]
    x = wide[..., 1:1 + ch] if ch % 2 else wide
    w, bias = rnd(g, (ch, W), scale=0.5), rnd(g, (ch,), scale=0.2)
    init = rnd(g, (2, W - 1, ch), dt)[copies]
    out, fin, _ = ssd.ssd_causal_conv_fwd(x, w, bias, init, activation=None)
    torch.cuda.synchronize()
    wo, bound, wf, _ = ref.conv(f64(x[:2]), f64(w), f64(bias), f64(init[:2]), None, False, dt)
    close("out", out[:2], wo, bound)
    assert np.array_equal(f64(fin[:2]), wf)
    assert torch.equal(out, out[:2][copies]) and torch.equal(fin, fin[:2][copies])


# 16-byte pieces a thread holds (rows are many, so that lanes stay few).
@pytest.mark.parametrize("norm_first", [False, True])
@pytest.mark.parametrize("rows,dim,dt,lead", [
    (4100, 2560, "bf16", 0),     # 64 lanes, 5 whole pieces
    (4100, 2555, "bf16", 3),     # 5, the last moved back
    (4100, 2051, "bf16", 0),     # 5 pieces, the fifth of one lane, moved back
    (4100, 2000, "bf16", 1),     # 4, some lanes without a last one
    (4100, 1030, "f32", 0),      # 5, fp32, moved back
    (4100, 1020, "f32", 1),      # 4
    (2060, 5117, "bf16", 0),     # 128 lanes, 5
    (9001, 1281, "f32", 0),      # beyond 64 lanes' registers by one element
])
def test_norm_four_and_five_pieces(rows, dim, dt, lead, norm_first):
    announce(rows, dim, dt, lead, norm_first)
    g = gen(95)
    x = rnd(g, (rows, dim), dt, pad=2)
    z = rnd(g, (rows, dim), dt, scale=2.0, lead=lead)
    w = 1 + rnd(g, (dim,), scale=0.2)
    out = ssd.ssd_gated_norm_fwd(x, z, w, norm_before_gate=norm_first)
    torch.cuda.synchronize()
    want, bound = ref.gated_norm(f64(x), f64(z), f64(w), 1, 1e-5, norm_first, dt)
    close("out", out, want, bound)


@pytest.mark.parametrize("b,T,Dm,N,G,dt,pad", [
    (2, 70, 192, 32, 1, "bf16", 8),         # tiles, no ranges
    (2, 61, 100, 64, 2, "bf16", 3),         # groups of 50: element by element
    (1, 700, 72, 32, 1, "bf16", 0),         # ranges
    (1, 700, 104, 64, 2, "bf16", 1),        # ranges, groups of 52
    (2, 515, 72, 64, 2, "f32", 0),          # ranges of wide states
    (1, 1300, 75, 64, 3, "f32", 5),         # many ranges, groups of 25
    (1, 333, 40, 32, 1, "f32", 2),
])
def test_scan_wide_states_in_tiles_and_ranges(b, T, Dm, N, G, dt, pad):
    announce(b, T, Dm, N, G, dt, pad)
    s = scan_inputs(gen(97), b, T, Dm, N, G, dt, True, True, True, True, pad)
    js = np.array([(T - 1, T // 3, -1)[i % 3] for i in range(b)], np.int32)
    y, fin, at = run_scan(s, True, torch.from_numpy(js).cuda())
    torch.cuda.synchronize()
    wy, by, wf, bf, wa, ba = ref_scan(s, True, js, dt)
    close("y", y, wy, by)
    close("final_state", fin, wf, bf)
    close("state_out", at, wa, ba)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_scan_few_tokens_of_wide_states(dt):
    for T, N in ((9, 32), (16, 32), (9, 64), (3, 32)):
        s = scan_inputs(gen(98), 2, T, 136, N, 2, dt, True, True, True, True, 8)
        js = np.array([T - 1, T // 2], np.int32)
        y, fin, at = run_scan(s, True, torch.from_numpy(js).cuda())
        torch.cuda.synchronize()
        wy, by, wf, bf, wa, ba = ref_scan(s, True, js, dt)
        close("y", y, wy, by)
        close("final_state", fin, wf, bf)
        close("state_out", at, wa, ba)


@pytest.mark.parametrize("V", [30011, 128256])
def test_verify_two_launches_without_residual(V):
    # p equal to q where drafts are rejected: nothing is left and p_n itself is
    # drawn from; NaN and negative entries count as 0 in sums and draws.
    shape = ssd.ssd_verify_shape(4, 2, V, 3 * V, V, 2 * V, V)
    assert ssd.ssd_verify_workspace_bytes(shape, ssd.SSD_DTYPE_F32) > 0
    p, tok, u, q = verify_inputs(99, 4, 2, V)
    for i, n in ((0, 0), (1, 1), (2, 0)):
        q[i, n] = p[i, n]
        tok[i, n] = V                                  # never accepted
    p[1, 1, 7:2000:5] = float("nan")
    q[1, 1] = torch.nan_to_num(p[1, 1])
    p[3, 0, 1::3] = -1.0
    q[3, 0, 2::7] = float("nan")
    p[2, 0] = 0.0                                      # no residual and no mass: V - 1
    q[2, 0] = 0.25
    got = ssd.ssd_verify_drafts(p, tok, u, q)
    torch.cuda.synchronize()
    want = ref.verify(f64(p), tok.cpu().numpy(), f64(u), f64(q))
    assert want[0][0] == 0 and want[0][2] == 0 and want[1][2] == V - 1
    same(got, want)
    # The same from a lookup: the zeroed token held all of the row's mass.
    p = torch.zeros(2, 2, V, device="cuda")
    p[:, 0, 12345] = 0.25
    p[1, 0, V - 2] = 0.5
    tok = torch.full((2, 1), 12345, dtype=torch.int32, device="cuda")
    u = torch.tensor([[0.9, 0.3], [0.9, 0.3]], device="cuda")
    got = ssd.ssd_verify_drafts(p, tok, u)
    torch.cuda.synchronize()
    assert got[0].cpu().tolist() == [0, 0] and got[1].cpu().tolist() == [12345, V - 2]
