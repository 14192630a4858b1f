"""The gated delta rule on the GPU against its definition in fp64."""
import numpy as np
import pytest
import torch

import block_refs as ref
import mamba_ssd_scan_06_amd as ssd
from test_gpu_layer_ops import TD, announce, f64, gen, rnd

pytestmark = pytest.mark.gpu


def inputs(seed, b, T, H, P, N, G, dtype="bf16", init=True, idx=True, lead=0, pad=0, decay=True, unit=False):
    """q, k, v as slices of wider rows that start `lead` elements in; with unit
    the keys and queries have norm 1 (up to their rounding)."""
    g = gen(seed)

    def rows(n, inner, norm):
        t = torch.randn(b, T, n, inner, generator=g)
        if norm:
            t = t / t.square().sum(-1, keepdim=True).sqrt()
        full = torch.zeros(b, T, lead + n * inner + pad, dtype=TD[dtype])
        full[:, :, lead:lead + n * inner] = t.flatten(2).to(TD[dtype])
        return full.cuda()[:, :, lead:lead + n * inner].unflatten(2, (n, inner))

    s = dict(q=rows(G, N, unit), k=rows(G, N, unit), v=rows(H, P, False))
    rate = torch.exp(torch.rand(H, generator=g) * 5 - 4)
    s["g"] = (-rate * torch.rand(b, T, H, generator=g)).cuda() if decay else None
    s["beta"] = torch.rand(b, T, H, generator=g).cuda()
    s["init_state"] = rnd(g, (b, H, P, N), scale=0.3) if init else None
    js = np.array([(-1, T - 1, T // 2, 0, T // 3)[i % 5] for i in range(b)], np.int32)
    s["state_out_idx"] = torch.from_numpy(js).cuda() if idx else None
    return s


def want_of(s, **kw):
    js = s["state_out_idx"]
    return ref.gated_delta(f64(s["q"]), f64(s["k"]), f64(s["v"]), f64(s["g"]), f64(s["beta"]),
                           init=f64(s["init_state"]), idx=None if js is None else js.cpu().numpy(), **kw)


def near(name, got, want, tol, dtype="f32"):
    """In the 2-norm within tol plus the final rounding; single elements within
    that of the root mean square and 8 times tol of it (the share of one element
    in an error that is spread over all: six sigma and more)."""
    got = f64(got)
    assert got.shape == want.shape, (name, got.shape, want.shape)
    assert np.isfinite(got).all(), f"{name}: non-finite values"
    if want.size == 0 or not want.any():
        assert not got.any(), name
        return
    d, rms = got - want, np.sqrt((want * want).mean())
    half = ref.HALF_STEP[dtype]
    rel = np.sqrt((d * d).mean()) / rms
    worst = (np.abs(d) - half * np.abs(want)).max() / rms
    print(f"  {name}: rel {rel:.2e} (bound {tol + half:.2e}), worst element beyond its rounding {worst:.2e}", flush=True)
    assert rel <= tol + half, name
    assert worst <= 8 * tol, name


def y_tolerance(N, dtype):
    """The outputs of bf16 calls read the state and the chunk's own part in 16
    bits of fraction (two bf16 each): 2^-15 of their terms."""
    return ref.delta_tolerance(N) + (2.0 ** -13 if dtype == "bf16" else 0.0)


def check(s, dtype, scale=None, l2=False, tol=None, **kw):
    N = s["q"].shape[3]
    y, fin, at = ssd.ssd_gated_delta_fwd(**s, scale=scale, qk_l2norm=l2, **kw)
    torch.cuda.synchronize()
    wy, wf, wa = want_of(s, scale=scale, l2=l2)
    tol = ref.delta_tolerance(N) if tol is None else tol
    near("final_state", fin, wf, tol)
    if wa is not None:
        near("state_out", at, wa, tol)
        for i, j in enumerate(s["state_out_idx"].tolist()):
            if j < 0:
                held = s["init_state"]
                assert torch.equal(at[i], torch.zeros_like(at[i]) if held is None else held[i])
    near("y", y, wy, y_tolerance(N, dtype) + tol - ref.delta_tolerance(N), dtype)
    return y, fin, at


CASES = [
    # b, T, H, P, N, G, dtype, l2, init, idx, lead, pad, decay
    (1, 1, 1, 16, 16, 1, "bf16", False, True, True, 0, 0, True),
    (3, 1, 4, 128, 128, 2, "bf16", True, True, True, 0, 0, True),
    (2, 1, 3, 80, 96, 1, "f32", True, True, False, 3, 2, True),
    (5, 2, 2, 32, 48, 1, "f32", False, False, True, 0, 0, False),
    (2, 7, 6, 64, 64, 3, "bf16", True, True, True, 8, 8, True),
    (5, 9, 4, 128, 128, 2, "bf16", True, True, True, 0, 0, True),
    (2, 8, 2, 256, 256, 2, "f32", True, True, True, 0, 0, True),
    (2, 16, 2, 48, 80, 1, "bf16", True, False, True, 5, 0, True),
    (5, 17, 2, 64, 128, 1, "f32", True, True, True, 0, 0, True),
    (3, 24, 2, 128, 128, 1, "f32", True, True, True, 0, 0, True),
    (3, 25, 2, 128, 128, 1, "f32", True, True, True, 0, 0, True),
    (3, 17, 2, 128, 128, 1, "bf16", True, True, True, 0, 0, True),
    (2, 31, 2, 32, 32, 1, "bf16", True, True, True, 0, 0, True),
    (2, 32, 3, 16, 64, 3, "bf16", True, True, True, 0, 0, True),
    (5, 33, 4, 48, 16, 2, "bf16", True, True, True, 1, 0, True),
    (2, 63, 2, 112, 112, 1, "f32", True, False, True, 0, 0, False),
    (5, 64, 2, 128, 128, 2, "bf16", True, True, True, 0, 0, True),
    (2, 65, 2, 128, 64, 1, "f32", True, True, True, 7, 3, True),
    (3, 100, 4, 80, 192, 2, "bf16", True, True, True, 0, 24, True),
    (1, 129, 2, 256, 256, 1, "bf16", True, True, True, 0, 0, True),
    (1, 130, 1, 256, 256, 1, "f32", True, True, True, 0, 0, True),
    (2, 200, 2, 144, 176, 1, "bf16", False, True, True, 0, 0, True),
    (5, 257, 8, 64, 128, 2, "bf16", True, True, True, 0, 0, True),
    (1, 515, 3, 32, 224, 3, "f32", True, False, True, 0, 0, True),
    (1, 1000, 2, 128, 128, 1, "bf16", True, False, False, 0, 0, True),
]


@pytest.mark.parametrize("case", CASES, ids=["-".join(str(v) for v in c[:7]) for c in CASES])
def test_against_definition(case):
    b, T, H, P, N, G, dtype, l2, init, idx, lead, pad, decay = case
    announce(*case)
    check(inputs(1, b, T, H, P, N, G, dtype, init, idx, lead, pad, decay, unit=not l2), dtype, l2=l2)


@pytest.mark.parametrize("dtype,lead", [("bf16", 0), ("bf16", 1), ("f32", 0)])
@pytest.mark.parametrize("N", [16, 48, 80, 128, 144, 192, 208, 256])
def test_many_heads(N, dtype, lead):
    # More workgroups than compute units: the other split of the work.
    announce(N, dtype, lead)
    check(inputs(20, 9, 70, 32, 16, N, 8, dtype, lead=lead, unit=True), dtype)


@pytest.mark.parametrize("T", [1, 3, 4, 9, 16])
@pytest.mark.parametrize("P,N,dtype", [(16, 160, "bf16"), (48, 16, "f32"), (64, 64, "bf16"), (80, 96, "f32"),
                                       (112, 128, "bf16"), (144, 48, "bf16"), (32, 176, "f32")])
def test_many_heads_few_tokens(P, N, dtype, T):
    # Enough rows for two per lane.
    announce(P, N, dtype, T)
    check(inputs(28, 18, T, 64, P, N, 8, dtype, pad=8), dtype, l2=True)


@pytest.mark.parametrize("dtype,lead", [("bf16", 0), ("bf16", 3), ("f32", 0)])
def test_many_heads_several_slices(dtype, lead):
    check(inputs(21, 5, 97, 32, 80, 128, 4, dtype, lead=lead), dtype, l2=True)


def ranges_of(b, T, H, P, N, G, dtype):
    """The number of token ranges a call is cut into, from the workspace: behind
    the chunks' tables and the accepted indices' stand the ranges' states, maps
    and a copy of init_state."""
    code = ssd.SSD_DTYPE_BF16 if dtype == "bf16" else ssd.SSD_DTYPE_F32
    need = ssd.ssd_gated_delta_workspace_bytes(ssd.ssd_delta_shape(b, T, H, P, N, G, *([0] * 10)), code)
    up = lambda n: (n + 255) // 256 * 256
    one = up(b * H * -(-T // 32) * (8192 if dtype == "bf16" else 9728)) + up(b * H * 144)
    for r in range(2, 17):
        if one + up(4 * (r - 1) * b * H * P * N) + up(4 * (r - 2) * b * H * N * N) + 4 * b * H * P * N == need:
            return r
    assert need == one
    return 1


RANGES = [
    # b, T, H, P, N, G, dtype, init, lead
    (1, 1300, 1, 16, 16, 1, "bf16", True, 0),
    (2, 1111, 2, 80, 48, 1, "bf16", True, 1),
    (1, 2100, 4, 128, 128, 2, "bf16", True, 0),
    (1, 1500, 2, 256, 64, 2, "bf16", False, 0),
    (1, 1200, 1, 64, 144, 1, "bf16", True, 0),
    (1, 1025, 2, 32, 256, 1, "bf16", True, 0),
    (1, 1025, 1, 48, 208, 1, "bf16", True, 8),
    (1, 1300, 3, 16, 96, 3, "f32", True, 0),
    (2, 1057, 2, 144, 128, 1, "f32", True, 3),
    (1, 999, 1, 64, 256, 1, "f32", False, 0),
]


@pytest.mark.parametrize("case", RANGES, ids=["-".join(map(str, c)) for c in RANGES])
def test_token_ranges(case):
    b, T, H, P, N, G, dtype, init, lead = case
    announce(*case)
    r = ranges_of(b, T, H, P, N, G, dtype)
    assert r >= 3
    s = inputs(22, b, T, H, P, N, G, dtype, init=init, lead=lead)
    s["g"] = s["g"] * 0.02                            # the first range's state reaches the last one
    tol = 3 * ref.delta_tolerance(N)                  # the maps' and the joins' roundings on top
    for js in ([0, T - 1], [T // r + 3, T // 2], [-1, T - 40]):
        s["state_out_idx"] = torch.tensor(js[:b], dtype=torch.int32, device="cuda")
        want = check(s, dtype, l2=True, tol=tol)
    held = s["init_state"].clone() if init else None
    got = ssd.ssd_gated_delta_fwd(**dict(s, init_state=held), qk_l2norm=True, final_state=held)
    torch.cuda.synchronize()
    for a, c in zip(want, got):
        assert torch.equal(a, c)


def test_ranges_only_where_few_heads_leave_the_gpu_idle():
    assert ranges_of(8, 2048, 32, 128, 128, 8, "bf16") == 1
    assert ranges_of(1, 16384, 32, 128, 128, 8, "bf16") >= 4
    assert ranges_of(1, 300, 1, 64, 64, 1, "bf16") == 1
    assert ranges_of(2, 25, 1, 64, 64, 1, "f32") == 1


def test_token_ranges_captured_and_on_two_streams():
    s = inputs(23, 1, 1400, 2, 64, 64, 1, "bf16")
    assert ranges_of(1, 1400, 2, 64, 64, 1, "bf16") >= 3
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        want = ssd.ssd_gated_delta_fwd(**s, qk_l2norm=True)
    again = [ssd.ssd_gated_delta_fwd(**s, qk_l2norm=True) for _ in range(2)]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = ssd.ssd_gated_delta_fwd(**s, qk_l2norm=True)
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        for a, c, d, e in zip(want, out, *again):
            assert torch.equal(a, c) and torch.equal(a, d) and torch.equal(a, e)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T", [9, 150])
def test_scale(T, dtype):
    check(inputs(2, 2, T, 2, 32, 64, 1, dtype, unit=True), dtype, scale=1.7)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T", [12, 100])
def test_equal_keys_replace_what_they_hold(T, dtype):
    # One key throughout, beta 1, no decay: the system of a chunk is as far from
    # the identity as it gets, and the state holds the last value only.
    s = inputs(3, 2, T, 2, 32, 64, 1, dtype, init=False, decay=False, unit=True)
    s["k"] = torch.zeros_like(s["k"])
    s["k"][..., 5] = 1.0
    s["beta"] = torch.ones_like(s["beta"])
    _, fin, _ = check(s, dtype)
    last = f64(s["v"][:, -1])
    assert np.abs(f64(fin)[..., 5] - last).max() <= 64 * ref.U * np.abs(f64(s["v"])).max()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T", [12, 100])
def test_alternating_overshoot(T, dtype):
    # beta 2 reflects the state along the key (norm 1): the rule neither grows
    # nor forgets.
    s = inputs(4, 2, T, 2, 32, 64, 1, dtype, decay=False, unit=True)
    s["k"] = torch.zeros_like(s["k"])
    s["k"][:, ::2, :, 3] = 1.0
    s["k"][:, 1::2, :, 40] = 1.0
    s["beta"] = torch.full_like(s["beta"], 2.0)
    # Errors of T tokens add (no contraction).
    check(s, dtype, tol=T * ref.delta_tolerance(64))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T", [10, 100])
def test_strong_and_vanishing_decay(T, dtype):
    # Decays that empty the state within a token, and none at all, in one chunk.
    s = inputs(5, 2, T, 4, 32, 64, 2, dtype, unit=True)
    s["g"][:, :, 0] = -200.0
    s["g"][:, :, 1] = 0.0
    s["g"][:, ::3, 2] = -90.0
    s["g"][:, 1, 3] = -1e4
    check(s, dtype)


@pytest.mark.parametrize("T", [10, 100])
def test_growth_is_computed_as_given(T):
    s = inputs(6, 2, T, 2, 32, 64, 1, "f32", unit=True)
    s["g"] = s["g"].abs() * 0.2
    check(s, "f32", tol=20 * ref.delta_tolerance(64))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("size", [1e-30, 1e-12, 1e-5, 1e5, 1e12, 1e30])
def test_values_of_any_size(size, dtype):
    s = inputs(24, 2, 100, 2, 32, 64, 1, dtype, unit=True)
    s["v"], s["init_state"] = (s["v"].float() * size).to(s["v"].dtype), s["init_state"] * size
    check(s, dtype)
    s["init_state"] = None
    check(s, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("size", [1e-15, 1e-4, 1e4, 1e15])
def test_keys_and_queries_of_any_size(size, dtype):
    # The rule with keys s k, beta / s^2 and values v is that of keys k, beta and
    # values v / s (and the state times 1 / s); queries are scaled back.
    s = inputs(25, 2, 100, 2, 32, 64, 1, dtype, init=False, unit=True)
    s["k"], s["q"] = ((s[n].float() * f).to(s[n].dtype) for n, f in (("k", size), ("q", 1 / size)))
    s["beta"] = s["beta"] / size ** 2
    check(s, dtype)
    check(dict(s, beta=s["beta"] * size ** 2), dtype, l2=True)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T", [200, 1100])
def test_sizes_that_change_along_the_sequence(T, dtype):
    # Values grow and shrink by 1e7 from one part to the next while strong decays
    # let the state follow; columns of the values differ as much, so each is
    # held to its own size.
    s = inputs(26, 2, T, 2, 32, 64, 1, dtype, unit=True)
    f = torch.ones(T)
    f[T // 3:] = 1e7
    f[T // 2:] = 1e-6
    s["v"] = (s["v"].float() * f.cuda()[None, :, None, None]).to(s["v"].dtype)
    s["g"] = s["g"].clone()
    s["g"][:, [T // 3, T // 2]] = -80.0
    y, fin, at = ssd.ssd_gated_delta_fwd(**s)
    torch.cuda.synchronize()
    wy, wf, wa = want_of(s)
    tol = 3 * ref.delta_tolerance(64)
    near("final_state", fin, wf, tol)
    for i in range(2):
        near("state_out", at[i], wa[i], tol)
    for a, e in ((0, T // 3), (T // 3, T // 2), (T // 2, T)):
        near("y", y[:, a:e], wy[:, a:e], 3 * y_tolerance(64, dtype), dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_columns_of_different_sizes(dtype):
    s = inputs(27, 2, 150, 2, 64, 64, 1, dtype, unit=True)
    f = torch.logspace(-3, 3, 64).cuda()
    s["v"], s["init_state"] = (s["v"].float() * f).to(s["v"].dtype), s["init_state"] * f[:, None]
    y, fin, _ = ssd.ssd_gated_delta_fwd(**s)
    torch.cuda.synchronize()
    wy, wf, _ = want_of(s)
    for c in range(0, 64, 7):
        near(f"column {c}", fin[:, :, c], wf[:, :, c], ref.delta_tolerance(64))
        near(f"column {c}", y[..., c], wy[..., c], y_tolerance(64, dtype), dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T", [5, 100])
def test_zero_beta_and_zero_keys(T, dtype):
    s = inputs(7, 2, T, 2, 32, 64, 1, dtype, unit=True)
    s["beta"][:, :, 0] = 0.0
    s["k"][0] = 0.0
    check(s, dtype, l2=True)


def test_empty_calls_copy_states():
    s = inputs(8, 3, 4, 2, 32, 64, 1, "bf16")
    for key in ("q", "k", "v"):
        s[key] = s[key][:, :0]
    s["g"], s["beta"] = s["g"][:, :0], s["beta"][:, :0].contiguous()
    s["state_out_idx"] = torch.full((3,), -1, dtype=torch.int32, device="cuda")
    y, fin, at = ssd.ssd_gated_delta_fwd(**s)
    torch.cuda.synchronize()
    assert y.shape == (3, 0, 2, 32) and torch.equal(fin, s["init_state"]) and torch.equal(at, s["init_state"])
    s["init_state"] = None
    _, fin, at = ssd.ssd_gated_delta_fwd(**s)
    torch.cuda.synchronize()
    assert not fin.any() and not at.any()
    s = inputs(8, 1, 4, 2, 32, 64, 1, "bf16")
    y, fin, at = ssd.ssd_gated_delta_fwd(**{k: v[:0] for k, v in s.items()})
    assert y.numel() == fin.numel() == at.numel() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T", [6, 77])
def test_in_place_and_given_outputs(T, dtype):
    s = inputs(9, 2, T, 4, 64, 128, 2, dtype)
    want = ssd.ssd_gated_delta_fwd(**s, qk_l2norm=True)
    given = dict(y=torch.full_like(want[0], float("nan")), state_out=torch.full_like(want[2], float("nan")))
    held = s["init_state"].clone()
    got = ssd.ssd_gated_delta_fwd(**dict(s, init_state=held), qk_l2norm=True, final_state=held, **given)
    torch.cuda.synchronize()
    assert got[1] is held and got[0] is given["y"] and got[2] is given["state_out"]
    for a, b in zip(want, got):
        assert torch.equal(a, b)
    y, fin, at = ssd.ssd_gated_delta_fwd(**dict(s, state_out_idx=None), qk_l2norm=True, return_final_state=False)
    torch.cuda.synchronize()
    assert fin is None and at is None and torch.equal(y, want[0])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("cut", [1, 5, 32, 50, 64])
def test_two_calls_continue_one(cut, dtype):
    T = 130
    s = inputs(10, 2, T, 2, 48, 64, 1, dtype, idx=False)
    part = lambda a, e: {k: (t if t is None or k == "init_state" else t[:, a:e]) for k, t in s.items()}
    y0, st, _ = ssd.ssd_gated_delta_fwd(**part(0, cut), qk_l2norm=True)
    y1, fin, _ = ssd.ssd_gated_delta_fwd(**dict(part(cut, T), init_state=st), qk_l2norm=True)
    torch.cuda.synchronize()
    wy, wf, _ = want_of(s, l2=True)
    tol = ref.delta_tolerance(64)
    near("final_state", fin, wf, 2 * tol)
    near("y", torch.cat([y0, y1], 1), wy, tol + y_tolerance(64, dtype), dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T", [5, 100])
def test_outputs_at_odd_addresses(T, dtype):
    s = inputs(30, 2, T, 2, 48, 64, 1, dtype)
    y, fin, at = ssd.ssd_gated_delta_fwd(**s, qk_l2norm=True)
    room = torch.full((y.numel() + 2,), 7.0, dtype=y.dtype, device="cuda")
    got = room[1:-1].view(y.shape)
    _, fin2, at2 = ssd.ssd_gated_delta_fwd(**s, qk_l2norm=True, y=got)
    torch.cuda.synchronize()
    # The way through registers computes the same bits.
    assert torch.equal(got, y) and torch.equal(fin, fin2) and torch.equal(at, at2)
    assert room[0] == 7 and room[-1] == 7


@pytest.mark.parametrize("T", [3, 70])
def test_indices_out_of_range_are_clamped(T):
    s = inputs(11, 4, T, 2, 32, 64, 1, "bf16")
    s["state_out_idx"] = torch.tensor([-7, T + 5, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32, device="cuda")
    _, fin, at = ssd.ssd_gated_delta_fwd(**s, qk_l2norm=True)
    torch.cuda.synchronize()
    assert torch.equal(at[0], s["init_state"][0]) and torch.equal(at[3], s["init_state"][3])
    assert torch.equal(at[1], fin[1]) and torch.equal(at[2], fin[2])


@pytest.mark.parametrize("T", [4, 90])
def test_free_strides_of_every_input(T):
    # Batch and token strides of each input on its own, rows shared by all
    # sequences (stride 0), g and beta as slices of wider rows.
    b, H, P, N, G = 3, 4, 32, 64, 2
    s = inputs(12, b, T, H, P, N, G, "bf16")
    want = ssd.ssd_gated_delta_fwd(**s, qk_l2norm=True)
    t = dict(s)
    for i, key in enumerate(("q", "k", "v", "g", "beta")):
        x = s[key].flatten(2)
        full = torch.full((T, b + 1, x.shape[2] + 3 * i + 1), float("nan"), dtype=x.dtype, device="cuda")
        full[:, :b, i:i + x.shape[2]] = x.transpose(0, 1)
        t[key] = full[:, :b, i:i + x.shape[2]].transpose(0, 1).unflatten(2, s[key].shape[2:])
    got = ssd.ssd_gated_delta_fwd(**t, qk_l2norm=True)
    torch.cuda.synchronize()
    for a, c in zip(want, got):
        assert torch.equal(a, c)
    one = {k: (s[k][:1].expand(b, *s[k].shape[1:]) if k in ("q", "k", "v", "g", "beta") else s[k]) for k in s}
    got = ssd.ssd_gated_delta_fwd(**one, qk_l2norm=True)
    want = ssd.ssd_gated_delta_fwd(**{k: (v if k in ("init_state", "state_out_idx") else v.contiguous()) for k, v in one.items()},
                                   qk_l2norm=True)
    torch.cuda.synchronize()
    for a, c in zip(want, got):
        assert torch.equal(a, c)


@pytest.mark.parametrize("T", [9, 96])
def test_same_bits_every_time_and_nothing_else_written(T):
    s = inputs(13, 3, T, 4, 48, 64, 2, "bf16")
    runs = []
    for fill in (float("nan"), 1e30):
        frame = torch.full((3 * T * 4 * 48 + 64,), fill, dtype=torch.bfloat16, device="cuda")
        y = frame[32:-32].view(3, T, 4, 48)
        held = torch.full((2, 3 * 4 * 48 * 64 + 64), fill, device="cuda")
        fin, at = (held[i, 32:-32].view(3, 4, 48, 64) for i in range(2))
        need = 16
        shape = ssd.ssd_delta_shape(3, T, 4, 48, 64, 2, *([0] * 10))
        need += ssd.ssd_gated_delta_workspace_bytes(shape, ssd.SSD_DTYPE_BF16)
        ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
        ssd.ssd_gated_delta_fwd(**s, qk_l2norm=True, y=y, final_state=fin, state_out=at, workspace=ws[:need - 16])
        torch.cuda.synchronize()
        for edge in (frame[:32], frame[-32:], held[:, :32], held[:, -32:]):
            assert torch.equal(edge.nan_to_num(7.0), torch.full_like(edge, fill).nan_to_num(7.0))
        assert (ws[need - 16:] == 255).all()
        runs.append((y.clone(), fin.clone(), at.clone()))
    for a, c in zip(*runs):
        assert torch.isfinite(a).all() and torch.equal(a, c)


def test_short_and_long_way_through_the_binding():
    for T in (1, 70):
        s = inputs(14, 2, T, 4, 64, 64, 2, "bf16", lead=4)
        a = ssd.ssd_gated_delta_fwd(**s, qk_l2norm=True, scale=0.5)
        b = ssd.ssd_gated_delta_fwd(**s, qk_l2norm=True, scale=0.5, y=torch.empty_like(a[0]))
        torch.cuda.synchronize()
        for u, w in zip(a, b):
            assert torch.equal(u, w)


@pytest.mark.parametrize("T", [1, 70])
def test_captured_and_replayed(T):
    s = inputs(15, 2, T, 4, 64, 64, 2, "bf16")
    held = s["init_state"].clone()
    out = [None]

    def step():
        out[0] = ssd.ssd_gated_delta_fwd(**dict(s, init_state=held), qk_l2norm=True, final_state=held)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    state = s["init_state"].clone()
    held.copy_(state)
    for turn in range(3):
        s["v"].copy_(rnd(gen(100 + turn), tuple(s["v"].shape), "bf16"))
        want = ssd.ssd_gated_delta_fwd(**dict(s, init_state=state), qk_l2norm=True)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out[0][0], want[0]) and torch.equal(held, want[1]) and torch.equal(out[0][2], want[2])
        state = want[1]


def test_two_streams_at_once():
    a, c = inputs(16, 2, 200, 4, 64, 128, 2, "bf16"), inputs(17, 2, 200, 4, 64, 128, 2, "bf16")
    want = [ssd.ssd_gated_delta_fwd(**s, qk_l2norm=True) for s in (a, c)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(4):
        for i, s in enumerate((a, c)):
            with torch.cuda.stream(streams[i]):
                got[i].append(ssd.ssd_gated_delta_fwd(**s, qk_l2norm=True))
    torch.cuda.synchronize()
    for i in range(2):
        for r in got[i]:
            for u, w in zip(r, want[i]):
                assert torch.equal(u, w)
    # A stream given by its handle.
    r = ssd.ssd_gated_delta_fwd(**a, qk_l2norm=True, stream=streams[0].cuda_stream)
    torch.cuda.synchronize()
    for u, w in zip(r, want[0]):
        assert torch.equal(u, w)


def test_padded_batch_takes_each_sequences_state():
    # Values behind a sequence's end do not reach its outputs or its state.
    lens = [40, 1, 33, 64, 7]
    s = inputs(18, 5, 64, 2, 48, 64, 1, "bf16")
    s["state_out_idx"] = torch.tensor([n - 1 for n in lens], dtype=torch.int32, device="cuda")
    y, _, at = ssd.ssd_gated_delta_fwd(**s, qk_l2norm=True)
    torch.cuda.synchronize()
    tol = ref.delta_tolerance(64)
    for i, n in enumerate(lens):
        one = {k: t[i:i + 1, :n] for k, t in s.items() if k not in ("init_state", "state_out_idx")}
        wy, wf, _ = want_of(dict(one, init_state=s["init_state"][i:i + 1], state_out_idx=None), l2=True)
        near("state", at[i:i + 1], wf, tol)
        near("y", y[i:i + 1, :n], wy, y_tolerance(64, "bf16"), "bf16")


def test_large_offsets():
    # Rows whose offsets pass 2^32 bytes: tokens 2^28 elements apart.
    T, stride = 20, 1 << 28
    base = torch.empty((T - 1) * stride + 64, dtype=torch.bfloat16, device="cuda")
    s = inputs(19, 1, T, 1, 32, 64, 1, "bf16")
    far = base.as_strided((1, T, 1, 64), (0, stride, 64, 1))
    far.copy_(s["k"])
    want = ssd.ssd_gated_delta_fwd(**s, qk_l2norm=True)
    got = ssd.ssd_gated_delta_fwd(**dict(s, k=far), qk_l2norm=True)
    torch.cuda.synchronize()
    for u, w in zip(got, want):
        assert torch.equal(u, w)
