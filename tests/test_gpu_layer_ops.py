"""The operators around the scan on the GPU against their definitions in fp64
(layer_refs), element by element within bounds counted in roundings."""
import numpy as np
import pytest
import torch

import layer_refs as ref
import mamba_ssd_scan_06_amd as ssd

pytestmark = pytest.mark.gpu

TD = {"bf16": torch.bfloat16, "f32": torch.float32}


def announce(*what):
    print("\n[case]", *what, flush=True)


def rnd(g, shape, dtype="f32", scale=1.0, pad=0, lead=0):
    """Normal values on the GPU, rounded to dtype; with pad or lead the last
    dimension is a slice of wider rows that start `lead` elements in."""
    full = list(shape)
    full[-1] += pad + lead
    t = (torch.randn(full, generator=g) * scale).to(TD[dtype]).cuda()
    return t[..., lead:lead + shape[-1]]


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def f64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def close(name, got, want, bound):
    got = f64(got)
    assert got.shape == want.shape, (name, got.shape, want.shape)
    if got.size == 0:
        return
    assert np.isfinite(got).all(), f"{name}: non-finite values"
    off = np.abs(got - want) / bound
    k = np.unravel_index(np.argmax(off), off.shape)
    print(f"  {name}: worst {off[k]:.3f} of the bound at {k}: got {got[k]:.6e}, want {want[k]:.6e}", flush=True)
    assert off[k] <= 1.0, f"{name}: {off[k]:.2f} times the bound at {k}: got {got[k]!r}, want {want[k]!r}"


# ------------------------------------------------------------ causal conv
CONV = [
    # name, b, T, split, width, dtype, act, bias, init, idx, lead, pad
    ("one_token", 5, 1, [64, 16, 16], 4, "bf16", True, True, True, True, 0, 0),
    ("one_token_f32_w2", 3, 1, [40], 2, "f32", False, False, True, True, 0, 0),
    ("two_tokens_w4", 2, 2, [24, 8, 8], 4, "bf16", True, True, True, True, 8, 16),
    ("three_tokens_no_init", 2, 3, [72, 8], 4, "f32", True, False, False, True, 4, 4),
    ("run_edges", 2, 33, [520, 8, 8], 4, "bf16", True, True, True, True, 0, 8),
    ("long_odd", 1, 517, [264, 24, 40], 3, "bf16", False, True, True, True, 8, 0),
    ("odd_channels", 2, 67, [65, 3, 2], 4, "bf16", True, True, True, True, 0, 0),
    ("odd_start", 2, 40, [64, 8, 8], 4, "bf16", True, True, True, True, 3, 2),
    ("even_start", 2, 40, [64, 8, 8], 4, "bf16", True, True, True, True, 2, 4),
    ("f32_odd", 2, 131, [129, 7], 2, "f32", True, True, True, True, 1, 0),
    ("f32_wide", 1, 70, [1032, 16, 16], 4, "f32", True, True, False, False, 0, 0),
    ("tiny_outputs", 2, 21, [3, 2, 5], 4, "bf16", True, True, True, True, 1, 3),
    ("tiny_then_wide", 2, 21, [3, 70, 1], 3, "f32", True, True, True, True, 0, 0),
    ("one_channel", 2, 12, [1], 2, "bf16", False, True, True, True, 0, 1),
    ("layer_2_7b", 2, 100, [5120, 128, 128], 4, "bf16", True, True, False, True, 5120, 80),
]


@pytest.mark.parametrize("case", CONV, ids=[c[0] for c in CONV])
def test_conv(case):
    name, b, T, split, W, dt, act, has_bias, has_init, has_idx, lead, pad = case
    announce(*case)
    g = gen(11)
    ch = sum(split)
    x = rnd(g, (b, T, ch), dt, pad=pad, lead=lead)
    w = rnd(g, (ch, W), scale=0.5)
    bias = rnd(g, (ch,), scale=0.2) if has_bias else None
    init = rnd(g, (b, W - 1, ch), dt) if has_init else None
    js = np.array([(-1, T - 1, T // 2, 0, 1)[i % 5] % max(T, 1) if i % 5 else -1 for i in range(b)], np.int32)
    idx = torch.from_numpy(js).cuda() if has_idx else None
    outs, fin, at = ssd.ssd_causal_conv_fwd(x, w, bias, init, idx, split=split, activation="silu" if act else None)
    torch.cuda.synchronize()
    want, bound, wfin, wat = ref.conv(f64(x), f64(w), f64(bias), f64(init), js if has_idx else None, act, dt)
    c0 = 0
    for k, n in enumerate(split):
        close(f"out{k}", outs[k], want[..., c0:c0 + n], bound[..., c0:c0 + n])
        c0 += n
    assert np.array_equal(f64(fin), wfin)             # raw inputs: the same bits
    if has_idx:
        assert np.array_equal(f64(at), wat)


@pytest.mark.parametrize("ch", [48, 53, 5, 2051])
def test_conv_steps_in_place_equal_one_call(ch):
    # Token by token with the state updated in place gives the whole call's bits.
    g = gen(3)
    b, T = 3, 9
    x, w, bias = rnd(g, (b, T, ch), "bf16"), rnd(g, (ch, 4)), rnd(g, (ch,))
    state = rnd(g, (b, 3, ch), "bf16").contiguous()
    whole, fin, _ = ssd.ssd_causal_conv_fwd(x, w, bias, state)
    held = state.clone()
    steps = [ssd.ssd_causal_conv_fwd(x[:, t:t + 1], w, bias, held, final_state=held)[0] for t in range(T)]
    torch.cuda.synchronize()
    assert torch.equal(torch.cat(steps, 1), whole) and torch.equal(held, fin)
    # A long call in place: many runs, state read by the first and written.
    T = 300
    x = rnd(g, (b, T, ch), "bf16")
    want, wfin, _ = ssd.ssd_causal_conv_fwd(x, w, bias, state)
    held = state.clone()
    got, _, _ = ssd.ssd_causal_conv_fwd(x, w, bias, held, final_state=held)
    torch.cuda.synchronize()
    assert torch.equal(got, want) and torch.equal(held, wfin)


def test_conv_broadcast_rows():
    # One row for all tokens, one sequence for all (strides of 0).
    g = gen(5)
    x = rnd(g, (1, 1, 40), "bf16").expand(2, 19, 40)
    w, bias = rnd(g, (40, 3)), rnd(g, (40,))
    o, fin, _ = ssd.ssd_causal_conv_fwd(x, w, bias)
    torch.cuda.synchronize()
    want, bound, wfin, _ = ref.conv(f64(x), f64(w), f64(bias), None, None, True, "bf16")
    close("out", o, want, bound)
    assert np.array_equal(f64(fin), wfin)


def test_conv_empty_calls():
    w = torch.zeros(16, 4, device="cuda")
    init = torch.randn(2, 3, 16, device="cuda")
    o, fin, _ = ssd.ssd_causal_conv_fwd(torch.zeros(2, 0, 16, device="cuda"), w, None, init)
    torch.cuda.synchronize()
    assert o.shape == (2, 0, 16) and torch.equal(fin, init)
    idx = torch.full((2,), -1, dtype=torch.int32, device="cuda")
    _, fin, at = ssd.ssd_causal_conv_fwd(torch.zeros(2, 0, 16, device="cuda"), w, None, None, idx)
    torch.cuda.synchronize()
    assert not fin.any() and not at.any()
    o, fin, _ = ssd.ssd_causal_conv_fwd(torch.zeros(0, 5, 16, device="cuda"), w)
    assert o.shape == (0, 5, 16) and fin.shape == (0, 3, 16)


def test_conv_keeps_non_finite_values_in_their_place():
    g = gen(4)
    x = rnd(g, (2, 70, 24), "f32").contiguous()
    x[0, 31, 5] = float("nan")
    x[1, 66, 7] = float("inf")
    w = rnd(g, (24, 4))
    o, _, _ = ssd.ssd_causal_conv_fwd(x, w, activation=None)
    torch.cuda.synchronize()
    bad = ~torch.isfinite(o.cpu())
    want = torch.zeros_like(bad)
    want[0, 31:35, 5] = True
    want[1, 66:70, 7] = True
    assert torch.equal(bad, want)


# --------------------------------------------------------- selective scan
SCAN = [
    # name, b, T, Dm, N, G, dtype, softplus, gate, skip, init, idx, pad
    ("one_token", 3, 1, 64, 16, 1, "bf16", True, True, True, True, True, 0),
    ("one_token_n8", 2, 1, 24, 8, 1, "f32", False, False, False, True, True, 0),
    ("one_token_odd_channels", 2, 1, 37, 16, 1, "bf16", True, True, True, True, True, 1),
    ("few_tokens_n64", 2, 7, 72, 64, 2, "bf16", True, True, True, True, True, 8),
    ("sixteen_n32", 2, 16, 200, 32, 1, "f32", True, True, True, True, True, 0),
    ("few_n16_groups", 3, 13, 72, 16, 2, "bf16", True, True, True, True, True, 8),
    ("few_n16_f32", 2, 8, 37, 16, 1, "f32", False, True, False, False, False, 3),
    ("few_n8", 2, 11, 40, 8, 1, "bf16", True, True, True, True, True, 0),
    ("few_n64_plain", 1, 15, 33, 64, 1, "f32", True, False, True, True, False, 0),
    ("seventeen", 2, 17, 136, 16, 2, "bf16", True, True, True, False, True, 8),
    ("tile_edges", 2, 65, 128, 16, 1, "bf16", True, True, True, True, True, 0),
    ("odd_everything", 3, 131, 75, 16, 3, "bf16", True, True, True, True, True, 5),
    ("f32_odd", 2, 101, 33, 8, 1, "f32", True, True, True, True, True, 3),
    ("f32_fours", 2, 70, 2 * 500, 64, 2, "f32", False, False, True, True, True, 1),
    ("f32_four_channels", 3, 60, 12, 16, 3, "f32", True, True, True, True, True, 0),
    ("no_extras", 1, 150, 64, 16, 1, "bf16", False, False, False, False, False, 0),
    ("n64_groups", 2, 90, 160, 64, 4, "f32", False, True, True, True, True, 4),
    ("long_few", 1, 1501, 72, 16, 1, "bf16", True, True, True, True, True, 8),
    ("long_few_f32", 2, 1000, 40, 32, 1, "f32", True, False, True, True, True, 0),
    ("long_n8", 1, 700, 64, 8, 2, "bf16", False, True, True, True, True, 0),
    ("many", 4, 70, 2048, 16, 1, "bf16", True, True, True, False, False, 0),
]


def scan_inputs(g, b, T, Dm, N, G, dt, softplus, gate, skip, init, pad):
    s = {}
    s["u"] = rnd(g, (b, T, Dm), dt, pad=pad)
    s["delta"] = rnd(g, (b, T, Dm), dt, pad=pad)
    s["bias"] = rnd(g, (Dm,), scale=1.5) - 3.0 if softplus else None
    if not softplus:
        s["delta"] = (torch.rand(b, T, Dm, generator=g) ** 3 * 0.3).to(TD[dt]).cuda()
    s["A"] = (-torch.exp(torch.rand(Dm, N, generator=g) * 3 - 0.7)).cuda()
    # B and C are slices of one projection's rows, as x, dt and z slices are.
    lead = pad
    rows = rnd(g, (b, T, 2 * G * N), dt, pad=pad, lead=lead)
    s["B"] = rows[..., :G * N].unflatten(2, (G, N))
    s["C"] = rows[..., G * N:].unflatten(2, (G, N))
    s["D"] = rnd(g, (Dm,)) if skip else None
    s["z"] = rnd(g, (b, T, Dm), dt, pad=pad, lead=pad) if gate else None
    s["init"] = rnd(g, (b, Dm, N), scale=0.5) if init else None
    return s


def run_scan(s, softplus, idx=None, **kw):
    return ssd.ssd_selective_scan_fwd(s["u"], s["delta"], s["A"], s["B"], s["C"], s["D"], s["z"], s["bias"], s["init"],
                                      idx, delta_softplus=softplus, **kw)


def ref_scan(s, softplus, js, dt):
    return ref.selective_scan(f64(s["u"]), f64(s["delta"]), f64(s["A"]), f64(s["B"]), f64(s["C"]), f64(s["D"]),
                              f64(s["z"]), f64(s["bias"]), softplus, f64(s["init"]), js, dt)


@pytest.mark.parametrize("case", SCAN, ids=[c[0] for c in SCAN])
def test_scan(case):
    name, b, T, Dm, N, G, dt, softplus, gate, skip, init, has_idx, pad = case
    announce(*case)
    s = scan_inputs(gen(21), b, T, Dm, N, G, dt, softplus, gate, skip, init, pad)
    js = np.array([(T - 1, -1, T // 2)[i % 3] for i in range(b)], np.int32) if has_idx else None
    idx = torch.from_numpy(js).cuda() if has_idx else None
    y, fin, at = run_scan(s, softplus, idx)
    torch.cuda.synchronize()
    wy, by, wf, bf, wa, ba = ref_scan(s, softplus, js, dt)
    close("y", y, wy, by)
    close("final_state", fin, wf, bf)
    if has_idx:
        close("state_out", at, wa, ba)


@pytest.mark.parametrize("T,j", [(301, j) for j in (0, 15, 16, 31, 32, 63, 64, 299, 300)] + [(10, j) for j in range(10)])
def test_scan_state_at_every_kind_of_index(T, j):
    s = scan_inputs(gen(22), 1, T, 64, 16, 1, "f32", True, False, True, True, 0)
    js = np.array([j], np.int32)
    y, fin, at = run_scan(s, True, torch.from_numpy(js).cuda())
    torch.cuda.synchronize()
    wy, by, wf, bf, wa, ba = ref_scan(s, True, js, "f32")
    close("y", y, wy, by)
    close("state_out", at, wa, ba)
    close("final_state", fin, wf, bf)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_scan_steps_in_place_follow_the_whole_call(dt):
    b, T, Dm, N = 2, 24, 72, 16
    s = scan_inputs(gen(23), b, T, Dm, N, 1, dt, True, True, True, True, 0)
    wy, by, wf, bf, _, _ = ref_scan(s, True, None, dt)
    held = s["init"].clone()
    ys = []
    for t in range(T):
        part = {k: (v[:, t:t + 1] if k in ("u", "delta", "B", "C", "z") else v) for k, v in s.items()}
        part["init"] = held
        ys.append(run_scan(part, True, final_state=held)[0])
    torch.cuda.synchronize()
    close("y", torch.cat(ys, 1), wy, by)
    close("final_state", held, wf, bf)


@pytest.mark.parametrize("T,Dm", [(300, 64), (40, 2048)])
def test_scan_in_place_long(T, Dm):
    s = scan_inputs(gen(24), 2, T, Dm, 16, 1, "bf16", True, True, True, True, 0)
    y0, f0, _ = run_scan(s, True)
    held = s["init"].clone()
    y1, f1, _ = run_scan(dict(s, init=held), True, final_state=held)
    torch.cuda.synchronize()
    assert torch.equal(y0, y1) and torch.equal(f0, held) and f1 is held


def test_scan_empty_calls():
    s = scan_inputs(gen(25), 2, 1, 16, 16, 1, "f32", False, False, True, True, 0)
    s0 = {k: (v[:, :0] if k in ("u", "delta", "B", "C") else v) for k, v in s.items()}
    idx = torch.full((2,), -1, dtype=torch.int32, device="cuda")
    y, fin, at = run_scan(s0, False, idx)
    torch.cuda.synchronize()
    assert y.shape == (2, 0, 16) and torch.equal(fin, s["init"]) and torch.equal(at, s["init"])
    s0["init"] = None
    _, fin, at = run_scan(s0, False, idx)
    torch.cuda.synchronize()
    assert not fin.any() and not at.any()
    y, fin, _ = run_scan({k: (v[:0] if v is not None and v.dim() > 2 else v) for k, v in s.items()}, False)
    assert y.shape == (0, 1, 16) and fin.shape == (0, 16, 16)


@pytest.mark.parametrize("T", [1, 5, 100, 1500])
def test_scan_keeps_non_finite_values_in_their_channel(T):
    # Channel 5 gets an inf, channel 70 a NaN, in the last token: nothing else
    # of any other channel or earlier token turns non-finite.
    s = scan_inputs(gen(26), 1, T, 80, 16, 1, "f32", True, True, True, True, 0)
    s["u"] = s["u"].clone()
    s["u"][0, T - 1, 5] = float("inf")
    s["u"][0, T - 1, 70] = float("nan")
    y, fin, _ = run_scan(s, True)
    torch.cuda.synchronize()
    bad = ~torch.isfinite(y.cpu())
    want = torch.zeros_like(bad)
    want[0, T - 1, 5] = want[0, T - 1, 70] = True
    assert torch.equal(bad, want)
    badf = ~torch.isfinite(fin.cpu())
    assert badf[0, 5].all() and badf[0, 70].all() and int(badf.sum()) == 2 * 16


def test_scan_extreme_steps():
    # Steps so large that every decay underflows, so small that none shows,
    # and delta far outside softplus's bend.
    b, T, Dm, N = 1, 60, 64, 16
    s = scan_inputs(gen(27), b, T, Dm, N, 1, "f32", True, False, False, True, 0)
    s["delta"] = s["delta"].clone()
    s["delta"][:, :20] = 60.0
    s["delta"][:, 20:40] = -40.0
    s["bias"] = torch.zeros(Dm, device="cuda")
    y, fin, _ = run_scan(s, True)
    torch.cuda.synchronize()
    wy, by, wf, bf, _, _ = ref_scan(s, True, None, "f32")
    close("y", y, wy, by)
    close("final_state", fin, wf, bf)


@pytest.mark.parametrize("b,Dm,T", [(12, 4096, 40), (1, 64, 4000), (3, 520, 333)])
def test_scan_many_workgroups_and_many_ranges(b, Dm, T):
    # More workgroups than the GPU holds at once; ranges of one and more tiles.
    s = scan_inputs(gen(29), b, T, Dm, 8, 1, "bf16", True, True, True, True, 0)
    js = np.array([(T - 1, T // 3, -1)[i % 3] for i in range(b)], np.int32)
    y, fin, at = run_scan(s, True, torch.from_numpy(js).cuda())
    torch.cuda.synchronize()
    wy, by, wf, bf, wa, ba = ref_scan(s, True, js, "bf16")
    close("y", y, wy, by)
    close("final_state", fin, wf, bf)
    close("state_out", at, wa, ba)


def test_scan_broadcast_inputs():
    # One row of steps for all tokens and sequences (strides of 0).
    b, T, Dm, N = 3, 50, 64, 16
    s = scan_inputs(gen(28), b, T, Dm, N, 1, "f32", True, True, True, False, 0)
    s["delta"] = s["delta"][:1, :1].expand(b, T, Dm)
    s["B"] = s["B"][:, :1].expand(b, T, 1, N)
    y, fin, _ = run_scan(s, True)
    torch.cuda.synchronize()
    wy, by, wf, bf, _, _ = ref_scan(s, True, None, "f32")
    close("y", y, wy, by)
    close("final_state", fin, wf, bf)


# -------------------------------------------------------------- gated norm
NORM = [
    # name, rows, dim, groups, dtype, gate, weight, norm_first, eps, lead, pad
    ("one_row", 1, 64, 1, "bf16", True, True, False, 1e-5, 0, 0),
    ("odd_dim", 5, 77, 1, "bf16", True, True, False, 1e-5, 0, 0),
    ("odd_dim_f32", 5, 33, 3, "f32", True, True, True, 1e-6, 1, 2),
    ("one_element", 7, 4, 4, "f32", True, True, False, 1e-5, 0, 0),
    ("groups", 9, 4096, 8, "bf16", True, True, False, 1e-5, 16, 80),
    ("no_gate", 6, 1024, 1, "bf16", False, True, False, 1e-5, 0, 0),
    ("no_weight", 6, 1000, 2, "f32", True, False, True, 0.0, 0, 8),
    ("layer", 33, 5120, 1, "bf16", True, True, False, 1e-5, 0, 5456),
    ("unaligned", 9, 640, 1, "bf16", True, True, True, 1e-5, 3, 4),
    ("half_aligned", 9, 640, 1, "bf16", True, True, True, 1e-5, 2, 4),
    ("wide", 3, 20000, 1, "bf16", True, True, False, 1e-5, 0, 0),
    ("very_wide", 2, 70001, 1, "f32", True, True, True, 1e-5, 0, 0),
    ("many_rows", 3001, 136, 1, "bf16", True, True, False, 1e-5, 8, 0),
    ("wide_groups", 4, 16384, 2, "f32", True, True, False, 1e-5, 0, 0),
]


@pytest.mark.parametrize("case", NORM, ids=[c[0] for c in NORM])
def test_norm(case):
    name, rows, dim, groups, dt, gate, has_w, norm_first, eps, lead, pad = case
    announce(*case)
    g = gen(31)
    x = rnd(g, (rows, dim), dt, pad=pad)
    z = rnd(g, (rows, dim), dt, scale=2.0, pad=pad, lead=lead) if gate else None
    w = 1 + rnd(g, (dim,), scale=0.2) if has_w else None
    out = ssd.ssd_gated_norm_fwd(x, z, w, ngroups=groups, eps=eps, norm_before_gate=norm_first)
    torch.cuda.synchronize()
    want, bound = ref.gated_norm(f64(x), f64(z), f64(w), groups, eps, norm_first, dt)
    close("out", out, want, bound)


def test_norm_shapes_and_in_place():
    g = gen(32)
    x, z, w = rnd(g, (3, 5, 256), "bf16"), rnd(g, (3, 5, 256), "bf16"), rnd(g, (256,))
    want = ssd.ssd_gated_norm_fwd(x, z, w)
    assert want.shape == x.shape
    for which in (0, 1):
        a, b = x.clone(), z.clone()
        got = ssd.ssd_gated_norm_fwd(a, b, w, out=(a, b)[which])
        torch.cuda.synchronize()
        assert torch.equal(got, want)
    assert ssd.ssd_gated_norm_fwd(x[:0], z[:0], w).shape == (0, 5, 256)
    # A token range of a padded batch, one row, and four dimensions.
    assert torch.equal(ssd.ssd_gated_norm_fwd(x[:, 1:4], z[:, 1:4], w), want[:, 1:4])
    assert torch.equal(ssd.ssd_gated_norm_fwd(x[1, 2], z[1, 2], w), want[1, 2])
    four = lambda t: t.unflatten(2, (4, 64)).contiguous()
    assert torch.equal(ssd.ssd_gated_norm_fwd(four(x), four(z), w[:64]).flatten(1, 2),
                       ssd.ssd_gated_norm_fwd(x.view(3, 20, 64), z.view(3, 20, 64), w[:64]))
    # A zero row keeps its zeros; a NaN row touches no other.
    x = x.clone()
    x[0, 0] = 0
    x[1, 1, 7] = float("nan")
    got = ssd.ssd_gated_norm_fwd(x, z, w).cpu()
    assert not got[0, 0].any()
    bad = torch.isnan(got).any(-1)
    assert bad[1, 1] and int(bad.sum()) == 1


# ------------------------------------------------------ draft verification
def verify_inputs(seed, b, K, V, dt="f32", spread=1.0, near=0.7):
    g = gen(seed)
    lg = torch.randn(b, K + 1, V, generator=g) * spread
    q = torch.softmax(lg[:, :K] + near * torch.randn(b, K, V, generator=g), -1).to(TD[dt])
    p = torch.softmax(lg, -1).to(TD[dt])
    u = torch.rand(b, K + 1, generator=g)
    tok = torch.zeros(b, K, dtype=torch.int32)
    for i in range(K):
        tok[:, i] = torch.multinomial(q[:, i].float(), 1, generator=g)[:, 0].to(torch.int32)
    return p.cuda(), tok.cuda(), u.cuda(), q.cuda()


def same(got, want):
    for name, a, w in zip(("n_accepted", "next_token", "tokens"), got, want):
        a = a.cpu().numpy()
        assert np.array_equal(a, w), f"{name}: {a.tolist()} != {w.tolist()}"


VERIFY = [
    # name, b, K, V, dtype, q, ragged
    ("one", 1, 8, 128256, "f32", True, False),
    ("batch", 17, 5, 1000, "f32", True, True),
    ("odd_vocab", 9, 3, 50277, "f32", True, False),
    ("lookup", 33, 4, 777, "f32", False, True),
    ("bf16", 12, 6, 4099, "bf16", True, True),
    ("bf16_lookup", 12, 2, 32000, "bf16", False, False),
    ("no_drafts", 8, 0, 5000, "f32", True, False),
    ("tiny_vocab", 40, 3, 2, "f32", True, True),
    ("one_token_vocab", 3, 2, 1, "f32", True, False),
    ("many_drafts", 3, 70, 64, "f32", True, True),
    ("big_batch", 600, 2, 300, "f32", True, True),
    ("big_batch_wide", 300, 1, 20011, "f32", True, False),
    ("rows_of_two_turns", 70, 1, 40009, "f32", True, True),     # a wave's piece passes 4096 elements
    ("split_odd", 3, 2, 30011, "bf16", False, False),
]


@pytest.mark.parametrize("case", VERIFY, ids=[c[0] for c in VERIFY])
def test_verify(case):
    name, b, K, V, dt, has_q, ragged = case
    announce(*case)
    for seed in (41, 42, 43):
        p, tok, u, q = verify_inputs(seed, b, K, V, dt)
        q = q if has_q else None
        if not has_q:
            u[:, :K] *= 0.01
        lens = torch.randint(0, K + 1, (b,), generator=gen(seed), dtype=torch.int32).cuda() if ragged else None
        got = ssd.ssd_verify_drafts(p, tok, u, q, lens)
        torch.cuda.synchronize()
        same(got, ref.verify(f64(p), tok.cpu().numpy(), f64(u), f64(q), None if lens is None else lens.cpu().numpy()))


def test_verify_strided_rows_and_given_outputs():
    b, K, V = 4, 3, 1001
    p, tok, u, q = verify_inputs(44, b, K, V)
    pw = torch.full((b, K + 1, V + 23), 9.0, device="cuda")
    pw[..., :V] = p
    qw = torch.full((b, K, V + 5), 9.0, device="cuda")
    qw[..., :V] = q
    flat = torch.full((b * (K + 1) + 8,), -7, dtype=torch.int32, device="cuda")
    n, nxt = torch.empty(b, dtype=torch.int32, device="cuda"), torch.empty(b, dtype=torch.int32, device="cuda")
    got = ssd.ssd_verify_drafts(pw[..., :V], tok, u, qw[..., :V], n_accepted=n, next_token=nxt,
                                tokens=flat[:b * (K + 1)].view(b, K + 1))
    torch.cuda.synchronize()
    same(got, ref.verify(f64(p), tok.cpu().numpy(), f64(u), f64(q)))
    assert got[0] is n and got[1] is nxt and (flat[b * (K + 1):] == -7).all()


def test_verify_exact_borders():
    # Dyadic probabilities: every product and sum is exact, so ties are ties.
    p = torch.tensor([[[0.25, 0.25, 0.5, 0.0], [0.5, 0.0, 0.25, 0.25]]]).cuda()
    q = torch.tensor([[[0.5, 0.25, 0.25, 0.0]]]).cuda()
    cases = [
        # draft, u_0, u_1 -> n, next
        (0, 0.5, 0.0, 0, 2),     # u q == p is a rejection; the residual is all on token 2
        (0, 0.49, 0.0, 1, 0),    # accepted; bonus from row 1, u 0: first token with mass
        (0, 0.49, 0.5, 1, 2),    # cut exactly at 0.5: token 0's mass does not exceed it, token 1 has none
        (0, 0.49, 0.75, 1, 3),
        (0, 0.49, 0.7499999, 1, 2),
        (3, 0.0, 0.9, 0, 2),     # no mass under either: rejected
        (2, 0.999, 0.25, 1, 0),
        (-1, 0.0, 0.3, 0, 2),    # outside the vocabulary
        (4, 0.0, 0.3, 0, 2),
    ]
    for tok, u0, u1, n, nxt in cases:
        t = torch.tensor([[tok]], dtype=torch.int32, device="cuda")
        u = torch.tensor([[u0, u1]], device="cuda")
        got = [v.cpu().tolist() for v in ssd.ssd_verify_drafts(p, t, u, q)]
        assert got[0] == [n] and got[1] == [nxt], (tok, u0, u1, got)
        assert got[2] == ([[nxt, -1]] if n == 0 else [[tok, nxt]])
    # Looked-up drafts: q is one at the token; an unknown token takes nothing.
    one = lambda tok, u0, u1: [v.cpu().tolist() for v in ssd.ssd_verify_drafts(
        p, torch.tensor([[tok]], dtype=torch.int32, device="cuda"), torch.tensor([[u0, u1]], device="cuda"))]
    assert one(2, 0.49, 0.0)[0] == [1]
    assert one(2, 0.5, 0.5)[:2] == [[0], [1]]             # residual 0.25, 0.25, 0, 0: the cut at 0.25
    assert one(9, 0.0, 0.5)[:2] == [[0], [2]]             # p itself


def test_verify_rows_without_mass_and_strange_values():
    V = 300
    p = torch.zeros(4, 2, V, device="cuda")
    q = torch.zeros(4, 1, V, device="cuda")
    tok = torch.zeros(4, 1, dtype=torch.int32, device="cuda")
    u = torch.full((4, 2), 0.5, device="cuda")
    p[1, 0, 7] = 0.25
    q[1, 0, 7] = 0.25                                     # the residual is empty: p itself
    p[2, 0, :] = float("nan")
    p[2, 0, 11] = 1.0
    p[3, 0, 5] = -1.0
    p[3, 0, 250] = 1e-30
    got = ssd.ssd_verify_drafts(p, tok, u, q)
    torch.cuda.synchronize()
    assert got[0].cpu().tolist() == [0, 0, 0, 0]
    assert got[1].cpu().tolist() == [V - 1, 7, 11, 250]
    # Uniforms of 1 and above take the last token with mass; lengths are clamped.
    p = torch.zeros(2, 2, V, device="cuda")
    p[:, :, 3] = 0.5
    p[:, :, 290] = 0.5
    u = torch.tensor([[0.1, 1.0], [0.1, 7.0]], device="cuda")
    lens = torch.tensor([-5, 99], dtype=torch.int32, device="cuda")
    tok = torch.full((2, 1), 3, dtype=torch.int32, device="cuda")
    got = ssd.ssd_verify_drafts(p, tok, u, None, lens)
    torch.cuda.synchronize()
    assert got[0].cpu().tolist() == [0, 1] and got[1].cpu().tolist() == [290, 290]


# --------------------------------------------- what holds for all of them
def test_outputs_end_where_they_end():
    """Rows behind each output's last keep their values."""
    g = gen(51)
    b, T, ch = 2, 37, 72

    def room(n, dtype):
        t = torch.full((n + 64,), 5.0 if dtype.is_floating_point else 5, dtype=dtype, device="cuda")
        return t, t[:n]

    x = rnd(g, (b, T, ch), "bf16")
    bufs = [room(b * T * n, torch.bfloat16) for n in (56, 8, 8)]
    fin = room(b * 3 * ch, torch.bfloat16)
    at = room(b * 3 * ch, torch.bfloat16)
    idx = torch.tensor([3, 36], dtype=torch.int32, device="cuda")
    ssd.ssd_causal_conv_fwd(x, rnd(g, (ch, 4)), None, None, idx, split=[56, 8, 8],
                            out=[t.view(b, T, n) for (_, t), n in zip(bufs, (56, 8, 8))],
                            final_state=fin[1].view(b, 3, ch), state_out=at[1].view(b, 3, ch))
    for T2, Dm in ((37, 72), (1, 72), (900, 72)):
        s = scan_inputs(g, b, T2, Dm, 16, 1, "bf16", True, True, True, True, 0)
        y, f, a = room(b * T2 * Dm, torch.bfloat16), room(b * Dm * 16, torch.float32), room(b * Dm * 16, torch.float32)
        run_scan(s, True, idx.clamp(max=T2 - 1), y=y[1].view(b, T2, Dm), final_state=f[1].view(b, Dm, 16),
                 state_out=a[1].view(b, Dm, 16))
        bufs += [y, f, a]
    o = room(5 * 100, torch.bfloat16)
    ssd.ssd_gated_norm_fwd(rnd(g, (5, 100), "bf16"), rnd(g, (5, 100), "bf16"), out=o[1].view(5, 100))
    torch.cuda.synchronize()
    for whole, used in bufs + [fin, at, o]:
        assert (whole[used.numel():] == 5).all()


def test_offsets_beyond_32_bits():
    """Token rows so far apart that element offsets pass 2^31."""
    b, T, ch, row = 2, 300, 64, 4_000_000
    g = gen(52)
    wide = torch.empty(b * T * row, dtype=torch.bfloat16, device="cuda")     # 4.8 GB
    x = wide.view(b, T, row)[:, :, row - ch:]
    x.copy_(rnd(g, (b, T, ch), "bf16"))
    assert x.stride(0) + x.stride(1) * (T - 1) > 2 ** 31
    w = rnd(g, (ch, 4))
    o, fin, _ = ssd.ssd_causal_conv_fwd(x, w)
    o2, fin2, _ = ssd.ssd_causal_conv_fwd(x.contiguous(), w)
    assert torch.equal(o, o2) and torch.equal(fin, fin2)
    s = scan_inputs(g, b, T, ch, 16, 1, "bf16", True, True, True, True, 0)
    want = run_scan(s, True)
    for k in ("u", "delta", "z"):
        x.copy_(s[k])
        got = run_scan(dict(s, **{k: x}), True)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]), k
    BC = wide.view(b, T, row)[:, :, row - 16:].unflatten(2, (1, 16))
    for k in ("B", "C"):
        BC.copy_(s[k])
        got = run_scan(dict(s, **{k: BC}), True)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]), k
    n = ssd.ssd_gated_norm_fwd(x.flatten(0, 1), x.flatten(0, 1))
    xc = x.flatten(0, 1).contiguous()
    assert torch.equal(n, ssd.ssd_gated_norm_fwd(xc, xc))
    del wide, x, BC
    torch.cuda.empty_cache()


def layer_run(s, c, nrm, ver):
    """One call of each operator, for the graph and stream tests."""
    out = []
    o, f, a = ssd.ssd_causal_conv_fwd(*c)
    out += [o, f, a]
    out += list(run_scan(s, True, c[4]))
    out.append(ssd.ssd_gated_norm_fwd(*nrm))
    out += list(ssd.ssd_verify_drafts(*ver))
    return out


def layer_inputs(seed, T):
    g = gen(seed)
    b, ch = 2, 72
    s = scan_inputs(g, b, T, ch, 16, 1, "bf16", True, True, True, True, 0)
    idx = torch.tensor([T // 2, T - 1], dtype=torch.int32, device="cuda")
    c = (rnd(g, (b, T, ch), "bf16"), rnd(g, (ch, 4)), rnd(g, (ch,)), rnd(g, (b, 3, ch), "bf16"), idx)
    nrm = (rnd(g, (b * T, ch), "bf16"), rnd(g, (b * T, ch), "bf16"), rnd(g, (ch,)))
    p, tok, u, q = verify_inputs(seed, b, 4, 32000)
    return s, c, nrm, (p, tok, u, q)


@pytest.mark.parametrize("T", [1, 45, 1200])
def test_captured_and_replayed(T):
    static = layer_inputs(61, T)
    layer_run(*static)                                 # before capture: the library is loaded
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = layer_run(*static)
    for seed in (62, 63, 64):
        fresh = layer_inputs(seed, T)
        want = [t.clone() for t in layer_run(*fresh)]
        for a, b in zip((*static[0].values(), *static[1], *static[2], *static[3]),
                        (*fresh[0].values(), *fresh[1], *fresh[2], *fresh[3])):
            if a is not None:
                a.copy_(b)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for k, (a, b) in enumerate(zip(held, want)):
            assert torch.equal(a, b), f"output {k} of replay {seed}"


@pytest.mark.parametrize("T", [1, 1200])
def test_on_a_given_stream(T):
    ins = layer_inputs(71, T)
    want = layer_run(*ins)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    raw = side.cuda_stream
    s, c, nrm, ver = ins
    got = list(ssd.ssd_causal_conv_fwd(*c, stream=raw)) + list(run_scan(s, True, c[4], stream=raw))
    got += [ssd.ssd_gated_norm_fwd(*nrm, stream=raw)] + list(ssd.ssd_verify_drafts(*ver, stream=raw))
    side.synchronize()
    for k, (a, b) in enumerate(zip(got, want)):
        assert torch.equal(a, b), k
    with torch.cuda.stream(side):
        got = layer_run(*ins)
    side.synchronize()
    for k, (a, b) in enumerate(zip(got, want)):
        assert torch.equal(a, b), k
    got = ssd.ssd_gated_norm_fwd(*nrm, stream=0)
    torch.cuda.synchronize()
    assert torch.equal(got, want[6])


@pytest.mark.parametrize("T", [5, 1200])
def test_two_streams_at_once(T):
    """Calls that may overlap on two streams, each with its own workspace."""
    ins = [layer_inputs(k, T) for k in (74, 75)]
    want = [[t.clone() for t in layer_run(*i)] for i in ins]
    torch.cuda.synchronize()
    side = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for turn in range(4):
        for k in (0, 1):
            with torch.cuda.stream(side[k]):
                got[k].append(layer_run(*ins[k]))
    torch.cuda.synchronize()
    for k in (0, 1):
        for turn, outs in enumerate(got[k]):
            for i, (a, b) in enumerate(zip(outs, want[k])):
                assert torch.equal(a, b), (k, turn, i)


@pytest.mark.parametrize("T", [1, 45, 1200])
def test_short_and_long_way_through_the_binding(T, monkeypatch):
    s, c, nrm, ver = layer_inputs(91, T)
    layer_run(s, c, nrm, ver)
    assert ssd._fast is not None

    def calls():
        init = s["init"].clone()
        out = list(run_scan(dict(s, init=init), True, None, final_state=init))          # in place, no index
        held = c[3].clone()
        out += list(ssd.ssd_causal_conv_fwd(c[0], c[1], None, held, split=(40, 32), activation=None, final_state=held)[0])
        out += [held]
        out += [ssd.ssd_causal_conv_fwd(c[0], c[1], return_final_state=False)[1]]
        out += [run_scan(s, 1, return_final_state=0)[1]]                                  # truth values of other types
        out += [ssd.ssd_gated_norm_fwd(nrm[0].view(2, T, -1), None, None, eps=0, norm_before_gate=True)]
        out += [ssd.ssd_gated_norm_fwd(*nrm, ngroups=8, norm_before_gate=True)]
        out += list(ssd.ssd_verify_drafts(ver[0], ver[1], ver[2], None, torch.tensor([1, 3], dtype=torch.int32).cuda()))
        return layer_run(s, c, nrm, ver) + out

    short = calls()
    monkeypatch.setattr(ssd, "_fast", None)
    long_ = calls()
    torch.cuda.synchronize()
    assert len(short) == len(long_)
    for k, (a, b) in enumerate(zip(short, long_)):
        assert (a is None and b is None) or (a.dtype == b.dtype and torch.equal(a, b)), k


def test_refusals_on_the_gpu():
    """Calls on GPU tensors that do not fit are refused whichever way they take."""
    s, c, nrm, ver = layer_inputs(92, 5)
    layer_run(s, c, nrm, ver)
    x, w, bias, init, idx = c
    bad = [
        (TypeError, lambda: ssd.ssd_causal_conv_fwd(x, w.bfloat16(), bias)),
        (ValueError, lambda: ssd.ssd_causal_conv_fwd(x, w[:-1], bias)),
        (ValueError, lambda: ssd.ssd_causal_conv_fwd(x, w, bias, init[:, :2])),
        (ValueError, lambda: ssd.ssd_causal_conv_fwd(x, w, bias, split=[72, 8])),
        (ValueError, lambda: ssd.ssd_causal_conv_fwd(x, w, bias, split=[-8, 80])),
        (ValueError, lambda: ssd.ssd_causal_conv_fwd(x, w, bias, activation="gelu")),
        (ValueError, lambda: ssd.ssd_causal_conv_fwd(x, w.cpu(), bias)),
        (TypeError, lambda: ssd.ssd_causal_conv_fwd(x.half(), w, bias)),
        (ValueError, lambda: ssd.ssd_causal_conv_fwd(x, w, bias, init, final_state=init[:1])),
        (TypeError, lambda: ssd.ssd_causal_conv_fwd(x, w, bias, init, idx.long())),
        (ssd.SsdError, lambda: ssd.ssd_causal_conv_fwd(x, w, bias, final_state=x[:, :3].contiguous()[:, :3], out=x)),
        (ssd.SsdError, lambda: ssd.ssd_causal_conv_fwd(x, torch.zeros(72, 5, device="cuda"))),
        (ValueError, lambda: run_scan(dict(s, B=s["B"].transpose(1, 3).contiguous().transpose(1, 3)), True)),
        (TypeError, lambda: run_scan(dict(s, A=s["A"].double()), True)),
        (ValueError, lambda: run_scan(dict(s, z=s["z"][:, :4]), True)),
        (ssd.SsdError, lambda: run_scan(dict(s, A=s["A"][:, :4].contiguous(), B=s["B"][..., :4].contiguous(),
                                             C=s["C"][..., :4].contiguous(), init=None), True)),
        (ssd.SsdError, lambda: run_scan(s, True, final_state=s["init"].view(-1)[:2 * 72 * 16].view(2, 72, 16),
                                        y=s["init"].view(torch.bfloat16).view(-1)[:2 * 5 * 72].view(2, 5, 72))),
        (ValueError, lambda: ssd.ssd_gated_norm_fwd(nrm[0], nrm[1][:-1], nrm[2])),
        (TypeError, lambda: ssd.ssd_gated_norm_fwd(nrm[0], nrm[1].float(), nrm[2])),
        (ssd.SsdError, lambda: ssd.ssd_gated_norm_fwd(*nrm, ngroups=5)),
        (ssd.SsdError, lambda: ssd.ssd_gated_norm_fwd(*nrm, ngroups=-1)),
        (ssd.SsdError, lambda: ssd.ssd_gated_norm_fwd(*nrm, eps=-1.0)),
        (ValueError, lambda: ssd.ssd_verify_drafts(ver[0], ver[1][:, :3], ver[2], ver[3])),
        (TypeError, lambda: ssd.ssd_verify_drafts(ver[0], ver[1].long(), ver[2], ver[3])),
        (TypeError, lambda: ssd.ssd_verify_drafts(ver[0], ver[1], ver[2], ver[3].bfloat16())),
        (ValueError, lambda: ssd.ssd_verify_drafts(ver[0], ver[1], ver[2].cpu(), ver[3])),
    ]
    for k, (kind, call) in enumerate(bad):
        print("refusal", k, flush=True)
        with pytest.raises(kind):
            call()
