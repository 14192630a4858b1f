"""The gated delta rule and the norms between blocks refuse calls that do not
fit, on the host and before any launch (no GPU needed: addresses below are never
dereferenced)."""
import pytest
import torch

import mamba_ssd_scan_06_amd as ssd
from test_layer_refusals import (BF16, ERR_ALIAS, ERR_ALIGN, ERR_ARGS, ERR_NULL, ERR_SHAPE, ERR_UNSUPPORTED,
                                 ERR_WORKSPACE, F32, OK, Call, z)

f = torch.float32


class Delta(Call):
    name = "ssd_gated_delta_fwd"

    def __init__(self, b=2, T=9, H=4, P=32, N=64, G=2, strides=None, scale=0.5):
        strides = strides or (T * G * N, G * N) * 2 + (T * H * P, H * P) + (T * H, H) * 2
        super().__init__(["q", "k", "v", "g", "beta", "init", "y", "final", "idx", "at", "ws"],
                         ["q", "k", "v", "g", "beta", "scale", "l2", "init", "y", "final", "idx", "at", "shape",
                          "dtype", "ws", "ws_bytes", "stream"],
                         ssd.ssd_delta_shape(b, T, H, P, N, G, *strides), scale=scale, l2=1, ws_bytes=1 << 30)


class Norms(Call):
    name = "ssd_residual_norm_fwd"

    def __init__(self, b=2, T=5, dim=64, strides=(320, 64) * 3, eps=1e-5, act=1, rs=1.0, bs=1.0, stream_dtype=BF16):
        super().__init__(["x", "residual", "gate", "post_weight", "layer", "weight", "out", "h"],
                         ["x", "residual", "gate", "act", "post", "post_weight", "layer", "rs", "bs", "weight", "eps",
                          "out", "h", "shape", "dtype", "sdtype", "stream"],
                         ssd.ssd_residual_norm_shape(b, T, dim, *strides), act=act, post=1, rs=rs, bs=bs, eps=eps,
                         sdtype=stream_dtype)


nan, inf = float("nan"), float("inf")


@pytest.mark.parametrize("make,status", [
    (lambda: Delta(b=-1), ERR_SHAPE), (lambda: Delta(T=-1), ERR_SHAPE), (lambda: Delta(H=0), ERR_SHAPE),
    (lambda: Delta(P=0), ERR_SHAPE), (lambda: Delta(N=-16), ERR_SHAPE), (lambda: Delta(G=0), ERR_SHAPE),
    (lambda: Delta(H=4, G=3), ERR_SHAPE), (lambda: Delta(P=24), ERR_UNSUPPORTED), (lambda: Delta(P=272), ERR_UNSUPPORTED),
    (lambda: Delta(N=8), ERR_UNSUPPORTED), (lambda: Delta(N=272), ERR_UNSUPPORTED),
    (lambda: Delta(b=65536), ERR_UNSUPPORTED), (lambda: Delta(H=65536, G=1), ERR_UNSUPPORTED),
    (lambda: Delta(T=1 << 31), ERR_UNSUPPORTED), (lambda: Delta(b=65535, H=256, P=32, G=1, T=1), OK),
    (lambda: Delta(b=65535, H=257, G=1, T=1), ERR_UNSUPPORTED),
    (lambda: Delta(scale=nan), ERR_ARGS), (lambda: Delta(scale=-inf), ERR_ARGS),
    *[(lambda i=i: Delta(strides=(64,) * i + (-1,) + (64,) * (9 - i)), ERR_SHAPE) for i in range(10)],
    *[(lambda i=i: Delta(strides=(64,) * i + (1 << 60,) + (64,) * (9 - i)), ERR_SHAPE) for i in range(10)],
    (lambda: Norms(b=-1), ERR_SHAPE), (lambda: Norms(T=-1), ERR_SHAPE), (lambda: Norms(dim=0), ERR_SHAPE),
    (lambda: Norms(dim=(1 << 20) + 1), ERR_UNSUPPORTED), (lambda: Norms(b=1 << 16, T=1 << 15), ERR_UNSUPPORTED),
    (lambda: Norms(b=1 << 62, T=4), ERR_UNSUPPORTED), (lambda: Norms(eps=-1e-9), ERR_ARGS), (lambda: Norms(eps=nan), ERR_ARGS),
    (lambda: Norms(eps=inf), ERR_ARGS), (lambda: Norms(rs=nan), ERR_ARGS), (lambda: Norms(bs=inf), ERR_ARGS),
    (lambda: Norms(act=3), ERR_ARGS), (lambda: Norms(act=-1), ERR_ARGS), (lambda: Norms(stream_dtype=7), ERR_ARGS),
    *[(lambda i=i: Norms(strides=(64,) * i + (-1,) + (64,) * (5 - i)), ERR_SHAPE) for i in range(6)],
])
def test_sizes_strides_and_scalars(make, status):
    c = make()
    if status == OK:                                  # refused for a pointer only, after the sizes
        c.p["q"] = None
        status = ERR_NULL
    assert c() == status
    assert ssd.ssd_last_error()


@pytest.mark.parametrize("cls,keys", [(Delta, ["q", "k", "v", "beta", "y"]), (Norms, ["x", "out"])])
def test_required_pointers_shape_and_dtype(cls, keys):
    for k in keys:
        c = cls()
        c.p[k] = None
        assert c() == ERR_NULL, k
    c = cls()
    c.dtype = 5
    assert c() == ERR_ARGS
    c = cls()
    c.shape = None
    assert c() == ERR_NULL


@pytest.mark.parametrize("cls,keys", [
    (Delta, [("q", 1), ("k", 1), ("v", 1), ("g", 2), ("beta", 2), ("init", 8), ("y", 1), ("final", 4), ("idx", 2),
             ("at", 8), ("ws", 8)]),
    (Norms, [("x", 1), ("residual", 1), ("gate", 1), ("post_weight", 2), ("layer", 2), ("weight", 2), ("out", 1),
             ("h", 1)]),
])
def test_alignment(cls, keys):
    for k, off in keys:
        c = cls()
        c.p[k] += off
        assert c() == ERR_ALIGN, k


@pytest.mark.parametrize("cls,pairs", [
    (Delta, [("y", "q"), ("y", "k"), ("y", "v"), ("y", "g"), ("y", "beta"), ("final", "idx"), ("at", "init"),
             ("at", "final"), ("final", "y")]),
    (Norms, [("out", "residual"), ("out", "gate"), ("out", "weight"), ("h", "x"), ("h", "gate"), ("h", "post_weight"),
             ("h", "layer"), ("out", "h")]),
])
def test_overlaps(cls, pairs):
    for a, b in pairs:
        c = cls()
        c.p[a] = c.p[b]
        assert c() == ERR_ALIAS, (a, b)


def test_in_place_only_where_the_rows_are_the_inputs_own():
    c = Delta()
    c.p["final"] = c.p["init"] + 16
    assert c() == ERR_ALIAS
    for out, of in (("out", "x"), ("h", "residual")):
        c = Norms()
        c.p[out] = c.p[of] + 16
        assert c() == ERR_ALIAS
        i = 0 if of == "x" else 2
        c = Norms(strides=(320, 64) * (i // 2) + (640, 128) + (320, 64) * (2 - i // 2))
        c.p[out] = c.p[of]
        assert c() == ERR_ALIAS
    # A stream of another type has other rows.
    c = Norms(stream_dtype=F32)
    c.p["h"] = c.p["x"]
    assert c() == ERR_ALIAS


def test_pairs_of_arguments():
    for k in ("idx", "at"):
        c = Delta()
        c.p[k] = None
        assert c() == ERR_ARGS
    c = Norms()
    c.scalars["post"] = 0
    assert c() == ERR_ARGS                            # a weight of the norm that is left out
    c = Norms(stream_dtype=BF16)
    c.dtype = F32
    assert c() == ERR_UNSUPPORTED


def test_workspace():
    c = Delta(b=1, T=500)
    need = ssd.ssd_gated_delta_workspace_bytes(c.shape, BF16)
    assert need > 0
    assert ssd.ssd_gated_delta_workspace_bytes(Delta(T=1).shape, BF16) == 0
    assert ssd.ssd_gated_delta_workspace_bytes(Delta(N=24).shape, BF16) == 0 and ssd.ssd_last_error()
    c.scalars["ws_bytes"] = need - 1
    assert c() == ERR_WORKSPACE
    c.scalars["ws_bytes"] = need
    c.p["ws"] = None
    assert c() == ERR_WORKSPACE
    for k in ("y", "final", "at", "q", "k", "v", "init", "g", "beta"):
        c.p["ws"] = c.p[k]
        assert c() == ERR_ALIAS, k
    c.p["ws"] = Delta().p["ws"] + 8
    assert c() == ERR_ALIGN


def test_chunks_of_all_heads_are_bounded():
    # The preparation numbers them in 32 bits.
    for T, status in (((1 << 25) - 32, OK), ((1 << 25), ERR_UNSUPPORTED)):
        c = Delta(b=1, T=T, H=64, P=16, N=16, G=1)
        need = ssd.ssd_gated_delta_workspace_bytes(c.shape, BF16)
        assert (need > 0) == (status == OK)
        if status != OK:
            assert c() == status


def test_nothing_to_do():
    for c in (Delta(b=0), Norms(b=0), Norms(T=0)):
        for k in c.p:
            c.p[k] = None
        assert c() == OK
    c = Delta(T=0)
    c.p["final"] = c.p["idx"] = c.p["at"] = None
    assert c() == OK


# ------------------------------------------------ the binding's own checks
def delta_args():
    return dict(q=z(2, 5, 2, 32), k=z(2, 5, 2, 32), v=z(2, 5, 4, 16), g=z(2, 5, 4, dtype=f), beta=z(2, 5, 4, dtype=f),
                init_state=z(2, 4, 16, 32, dtype=f), state_out_idx=z(2, dtype=torch.int32))


def norms_args():
    return dict(x=z(2, 6, 24), residual=z(2, 6, 24), weight=z(24, dtype=f), post_norm=True, post_weight=z(24, dtype=f),
                gate=z(2, 6, 24), layer_scale=z(24, dtype=f))


CALLS = {"delta": (ssd.ssd_gated_delta_fwd, delta_args, "q"), "norms": (ssd.ssd_residual_norm_fwd, norms_args, "x")}


@pytest.mark.parametrize("op,key", [(op, k) for op, (_, a, first) in CALLS.items() for k, t in a().items()
                                    if torch.is_tensor(t) and k != first])
def test_binding_refuses_wrong_shape_type_and_layout(op, key):
    call, args, _ = CALLS[op]
    a = args()
    t = a[key]
    with pytest.raises(ValueError):
        call(**dict(a, **{key: torch.zeros(*[n + 1 for n in t.shape], dtype=t.dtype)}))
    with pytest.raises(TypeError):
        call(**dict(a, **{key: t.double()}))
    if t.dim() > 1:
        with pytest.raises(ValueError):
            call(**dict(a, **{key: t.transpose(-1, -2).contiguous().transpose(-1, -2)}))


@pytest.mark.parametrize("op", list(CALLS))
def test_binding_refuses_cpu_tensors_and_bad_first_input(op):
    call, args, first = CALLS[op]
    a = args()
    with pytest.raises(ValueError, match="GPU"):
        call(**a)
    with pytest.raises(TypeError):
        call(**dict(a, **{first: a[first].half()}))
    with pytest.raises(ValueError):
        call(**dict(a, **{first: a[first].reshape(-1)}))


def test_binding_refuses_outputs_and_options():
    a = delta_args()
    with pytest.raises(ValueError, match="y"):
        ssd.ssd_gated_delta_fwd(**a, y=z(2, 5, 4, 17))
    with pytest.raises(ValueError, match="final_state"):
        ssd.ssd_gated_delta_fwd(**a, final_state=z(2, 4, 17, 32, dtype=f))
    with pytest.raises(ValueError, match="state_out"):
        ssd.ssd_gated_delta_fwd(**dict(a, state_out_idx=None), state_out=z(2, 4, 16, 32, dtype=f))
    with pytest.raises(TypeError, match="workspace"):
        ssd.ssd_gated_delta_fwd(**a, workspace=z(100, dtype=f))
    n = norms_args()
    with pytest.raises(ValueError, match="gate_activation"):
        ssd.ssd_residual_norm_fwd(**n, gate_activation="relu")
    with pytest.raises(ValueError, match="post_weight"):
        ssd.ssd_residual_norm_fwd(**dict(n, post_norm=False))
    with pytest.raises(ValueError, match="out"):
        ssd.ssd_residual_norm_fwd(**n, out=z(2, 6, 23))
    with pytest.raises(TypeError, match="residual_out"):
        ssd.ssd_residual_norm_fwd(**n, residual_out=z(2, 6, 24, dtype=f))
    with pytest.raises(ValueError, match="GPU"):      # one gate per sequence fits
        ssd.ssd_residual_norm_fwd(**dict(n, gate=z(2, 1, 24)))
    with pytest.raises(TypeError, match="residual"):
        ssd.ssd_residual_norm_fwd(**dict(n, residual=z(2, 6, 24, dtype=torch.float16)))
