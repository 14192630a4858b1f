"""Norms before and after a block with gate, scales and residual stream, on the
GPU against their definition in fp64, element by element."""
import numpy as np
import pytest
import torch

import block_refs as ref
import mamba_ssd_scan_06_amd as ssd
from test_gpu_layer_ops import TD, announce, close, f64, gen, rnd

pytestmark = pytest.mark.gpu


def inputs(seed, shape, dtype, stream, post, gate, act, layer, res=True, weight=True, lead=0, pad=0):
    g = gen(seed)
    d = shape[-1]
    s = dict(x=rnd(g, shape, dtype, 0.7, pad, lead), residual=rnd(g, shape, stream, 2.0, pad, lead) if res else None,
             weight=1 + rnd(g, (d,), scale=0.2) if weight else None, post_norm=post,
             post_weight=1 + rnd(g, (d,), scale=0.2) if post and weight else None, gate_activation=act,
             layer_scale=rnd(g, (d,)) if layer else None, residual_scale=0.9, branch_scale=1.3)
    s["gate"] = None
    if gate == "token":
        s["gate"] = rnd(g, shape, dtype, 1.0, pad, lead)
    elif gate == "sequence":
        s["gate"] = rnd(g, (*shape[:-2], 1, d), dtype, 1.0, pad, lead)
    return s


def want_of(s, dtype, stream, eps=1e-5):
    shape = s["x"].shape
    flat = lambda t: None if t is None else f64(t.expand(shape)).reshape(-1, shape[-1])
    return ref.residual_norm(flat(s["x"]), flat(s["residual"]), f64(s["weight"]), s["post_norm"], f64(s["post_weight"]),
                             flat(s["gate"]), s["gate_activation"], f64(s["layer_scale"]), np.float32(0.9).astype(float),
                             np.float32(1.3).astype(float), float(np.float32(eps)), dtype, stream)


def check(s, dtype, stream, **kw):
    out, h = ssd.ssd_residual_norm_fwd(**s, **kw)
    torch.cuda.synchronize()
    wo, bo, wh, bh = want_of(s, dtype, stream)
    assert out.shape == s["x"].shape and out.dtype == TD[dtype] and h.dtype == TD[stream]
    close("out", out.reshape(wo.shape), wo, bo)
    close("h", h.reshape(wh.shape), wh, bh)
    return out, h


CASES = [
    # shape, dtype, stream, post, gate, act, layer, residual, weight, lead, pad
    ((1, 1, 1), "bf16", "bf16", True, "token", "silu", True, True, True, 0, 0),
    ((2, 3, 7), "bf16", "f32", True, "sequence", None, False, True, True, 0, 0),
    ((2, 3, 3), "f32", "f32", False, "token", "sigmoid", True, True, True, 1, 1),
    ((3, 5, 8), "bf16", "bf16", False, None, None, False, True, True, 0, 0),
    ((2, 5, 9), "bf16", "f32", True, "token", "sigmoid", True, True, True, 3, 0),
    ((64, 1, 4096), "bf16", "bf16", True, "token", "sigmoid", False, True, True, 0, 32),
    ((2, 33, 64), "f32", "f32", True, "sequence", "silu", True, True, True, 0, 4),
    ((3, 17, 1000), "bf16", "f32", True, "sequence", "sigmoid", True, True, True, 5, 2),
    ((2, 9, 2049), "f32", "f32", True, "sequence", None, True, True, True, 5, 0),
    ((2, 9, 2047), "bf16", "bf16", True, "token", None, True, True, True, 1, 0),
    ((1, 300, 5120), "bf16", "f32", False, None, None, False, True, True, 0, 0),
    ((4, 700, 520), "bf16", "bf16", True, "token", "silu", False, True, True, 0, 8),
    ((1, 3, 8192), "f32", "f32", True, "token", "silu", True, True, True, 0, 0),
    ((1, 2, 16384), "f32", "f32", True, "token", None, True, True, True, 0, 0),
    ((1, 2, 16388), "f32", "f32", True, "token", "silu", True, True, True, 0, 0),
    ((1, 2, 33003), "bf16", "f32", True, "sequence", "silu", True, True, True, 1, 0),
    ((1, 2, 40001), "bf16", "bf16", False, "token", "sigmoid", True, True, True, 0, 0),
    ((1, 2, 100003), "f32", "f32", True, None, None, False, True, True, 0, 0),
    ((37, 100), "bf16", "bf16", True, "token", "silu", True, True, True, 0, 0),
    ((6,), "f32", "f32", True, "token", None, True, True, True, 0, 0),
    ((2, 3, 4, 72), "bf16", "f32", True, "token", "silu", True, True, True, 0, 0),
    ((2, 30, 256), "bf16", "bf16", True, None, None, False, False, True, 0, 0),
    ((2, 30, 256), "f32", "f32", False, "token", None, False, True, False, 0, 0),
]


@pytest.mark.parametrize("case", CASES, ids=["x".join(map(str, c[0])) + f"-{c[1]}-{c[2]}" for c in CASES])
def test_against_definition(case):
    shape, dtype, stream, post, gate, act, layer, res, weight, lead, pad = case
    announce(*case)
    check(inputs(1, shape, dtype, stream, post, gate, act, layer, res, weight, lead, pad), dtype, stream)


@pytest.mark.parametrize("dtype,stream", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
@pytest.mark.parametrize("dim", [5, 100, 1023, 40000])
def test_in_place(dim, dtype, stream):
    s = inputs(2, (2, 37, dim), dtype, stream, True, "token", "silu", True)
    s["x"], s["residual"] = s["x"].contiguous(), s["residual"].contiguous()
    for post in (True, False):
        s["post_norm"] = post
        if not post:
            s["post_weight"] = None
        want = ssd.ssd_residual_norm_fwd(**s)
        x, r = s["x"].clone(), s["residual"].clone()
        got = ssd.ssd_residual_norm_fwd(**dict(s, x=x, residual=r), out=x, residual_out=r)
        torch.cuda.synchronize()
        assert got[0] is x and got[1] is r and torch.equal(x, want[0]) and torch.equal(r, want[1])
        out, h = ssd.ssd_residual_norm_fwd(**s, return_residual=False)
        torch.cuda.synchronize()
        assert h is None and torch.equal(out, want[0])


@pytest.mark.parametrize("dim", [64, 1001, 40000])
def test_outputs_at_odd_addresses(dim):
    s = inputs(31, (2, 5, dim), "bf16", "bf16", True, "token", "silu", True)
    out, h = ssd.ssd_residual_norm_fwd(**s)
    rooms = [torch.full((out.numel() + 2,), 7.0, dtype=out.dtype, device="cuda") for _ in range(2)]
    got = [r[1:-1].view(out.shape) for r in rooms]
    ssd.ssd_residual_norm_fwd(**s, out=got[0], residual_out=got[1])
    torch.cuda.synchronize()
    assert torch.equal(got[0], out) and torch.equal(got[1], h)
    assert all(r[0] == 7 and r[-1] == 7 for r in rooms)


def test_without_residual_the_stream_takes_the_given_type():
    s = inputs(3, (2, 5, 96), "bf16", "bf16", True, None, None, False, res=False)
    h = torch.empty(2, 5, 96, device="cuda")
    out, got = ssd.ssd_residual_norm_fwd(**s, residual_out=h)
    torch.cuda.synchronize()
    wo, bo, wh, bh = want_of(s, "bf16", "f32")
    assert got is h
    close("out", out.reshape(wo.shape), wo, bo)
    close("h", h.reshape(wh.shape), wh, bh)


def test_rows_of_zeros_and_eps():
    s = inputs(4, (1, 4, 64), "f32", "f32", True, None, None, False)
    s["x"], s["residual"] = torch.zeros_like(s["x"]), torch.zeros_like(s["residual"])
    out, h = ssd.ssd_residual_norm_fwd(**s)
    torch.cuda.synchronize()
    assert not out.any() and not h.any()
    out, _ = ssd.ssd_residual_norm_fwd(**s, eps=0.0)
    torch.cuda.synchronize()
    assert out.isnan().all()


def test_a_row_does_not_see_the_others():
    # Infinities and NaN stay in their row; empty calls write nothing.
    s = inputs(5, (3, 40, 200), "bf16", "f32", True, "token", "sigmoid", True)
    want = ssd.ssd_residual_norm_fwd(**s)
    s["x"][1, 7, 3] = float("inf")
    s["residual"][2, 8, 5] = float("nan")
    out, h = ssd.ssd_residual_norm_fwd(**s)
    torch.cuda.synchronize()
    keep = torch.ones(3, 40, dtype=torch.bool, device="cuda")
    keep[1, 7] = keep[2, 8] = False
    assert torch.equal(out[keep], want[0][keep]) and torch.equal(h[keep], want[1][keep])
    assert out[2, 8].isnan().all()
    out, h = ssd.ssd_residual_norm_fwd(s["x"][:, :0], s["residual"][:, :0], s["weight"])
    assert out.shape == h.shape == (3, 0, 200)


def test_gates_that_saturate():
    s = inputs(6, (1, 6, 64), "f32", "f32", False, "token", "sigmoid", False)
    s["gate"] = torch.tensor([-1e4, -100.0, -30.0, 30.0, 100.0, 1e4], device="cuda")[None, :, None].expand(1, 6, 64).contiguous()
    for act in ("sigmoid", "silu"):
        s["gate_activation"] = act
        check(s, "f32", "f32")


def test_short_and_long_way_graph_and_streams():
    s = inputs(7, (5, 9, 520), "bf16", "f32", True, "token", "silu", True, lead=8)
    want = ssd.ssd_residual_norm_fwd(**s)
    got = ssd.ssd_residual_norm_fwd(**s, out=torch.empty_like(want[0]))
    side = torch.cuda.Stream()
    other = ssd.ssd_residual_norm_fwd(**s, stream=side.cuda_stream)
    torch.cuda.synchronize()
    for u, w, o in zip(got, want, other):
        assert torch.equal(u, w) and torch.equal(o, w)
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        ssd.ssd_residual_norm_fwd(**s)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = ssd.ssd_residual_norm_fwd(**s)
    for turn in range(3):
        s["x"].copy_(rnd(gen(50 + turn), (5, 9, 520), "bf16"))
        want = ssd.ssd_residual_norm_fwd(**s)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])
