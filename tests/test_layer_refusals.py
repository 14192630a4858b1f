"""The operators around the scan refuse calls that do not fit, on the host and
before any launch (no GPU needed: addresses below are never dereferenced)."""
import ctypes

import pytest
import torch

import mamba_ssd_scan_06_amd as ssd

OK, ERR_NULL, ERR_SHAPE, ERR_CHUNK, ERR_ALIGN, ERR_WORKSPACE, ERR_ALIAS, ERR_ARGS, ERR_HIP, ERR_UNSUPPORTED = range(10)
BASE, STEP = 1 << 40, 1 << 32
BF16, F32 = ssd.SSD_DTYPE_BF16, ssd.SSD_DTYPE_F32


class Call:
    """Arguments of one entry point at fake addresses; tests change some."""

    def __init__(self, names, order, shape, **scalars):
        self.p = {k: BASE + i * STEP for i, k in enumerate(names)}
        self.order, self.shape, self.scalars, self.dtype = order, shape, scalars, BF16

    def vals(self):
        for k in self.order:
            if k == "shape":
                yield None if self.shape is None else ctypes.byref(self.shape)
            elif k == "dtype":
                yield self.dtype
            elif k == "stream":
                yield None
            else:
                yield self.p[k] if k in self.p else self.scalars[k]

    def __call__(self):
        return getattr(ssd._load(), self.name)(*self.vals())


class Conv(Call):
    name = "ssd_causal_conv_fwd"

    def __init__(self, b=2, T=9, ch=(64, 16, 16), W=4, bs=1200, ts=120):
        super().__init__(["x", "weight", "bias", "init", "out0", "out1", "out2", "final", "idx", "at"],
                         ["x", "weight", "bias", "init", "act", "out0", "out1", "out2", "final", "idx", "at", "shape",
                          "dtype", "stream"],
                         ssd.ssd_conv_shape(b, T, (ctypes.c_int64 * 3)(*ch), W, bs, ts), act=1)


class Scan(Call):
    name = "ssd_selective_scan_fwd"

    def __init__(self, b=2, T=9, D=64, N=16, G=2, strides=(9 * 64, 64) * 3 + (9 * 64, 64) * 2):
        super().__init__(["u", "delta", "A", "B", "C", "D", "z", "bias", "init", "y", "final", "idx", "at", "ws"],
                         ["u", "delta", "A", "B", "C", "D", "z", "bias", "soft", "init", "y", "final", "idx", "at",
                          "shape", "dtype", "ws", "ws_bytes", "stream"],
                         ssd.ssd_selective_shape(b, T, D, N, G, *strides), soft=1, ws_bytes=1 << 30)


class Norm(Call):
    name = "ssd_gated_norm_fwd"

    def __init__(self, rows=4, dim=64, G=2, xs=64, zs=64, eps=1e-5, b=1, xb=256, zb=256):
        super().__init__(["x", "z", "weight", "out"],
                         ["x", "z", "weight", "out", "eps", "first", "shape", "dtype", "stream"],
                         ssd.ssd_norm_shape(b, rows, dim, G, xb, xs, zb, zs), eps=eps, first=0)


class Verify(Call):
    name = "ssd_verify_drafts"

    def __init__(self, b=2, K=3, V=100, strides=(400, 100, 300, 100)):
        super().__init__(["p", "q", "tok", "lens", "u", "n", "next", "tokens", "ws"],
                         ["p", "q", "tok", "lens", "u", "n", "next", "tokens", "shape", "dtype", "ws", "ws_bytes",
                          "stream"],
                         ssd.ssd_verify_shape(b, K, V, *strides), ws_bytes=1 << 30)


@pytest.mark.parametrize("make,status", [
    (lambda: Conv(b=-1), ERR_SHAPE), (lambda: Conv(T=-1), ERR_SHAPE), (lambda: Conv(ch=(0, 8, 8)), ERR_SHAPE),
    (lambda: Conv(ch=(8, -8, 8)), ERR_SHAPE), (lambda: Conv(W=1), ERR_UNSUPPORTED),
    (lambda: Conv(W=5), ERR_UNSUPPORTED), (lambda: Conv(ch=(1 << 20, 1, 0)), ERR_UNSUPPORTED),
    (lambda: Conv(b=65536), ERR_UNSUPPORTED), (lambda: Conv(T=1 << 31), ERR_UNSUPPORTED),
    (lambda: Conv(ts=-1), ERR_SHAPE), (lambda: Conv(bs=1 << 50), ERR_SHAPE), (lambda: Conv(bs=1 << 62), ERR_SHAPE),
    (lambda: Conv(b=65535, T=(1 << 31) - 1), ERR_SHAPE),
    (lambda: Scan(b=-1), ERR_SHAPE), (lambda: Scan(D=0), ERR_SHAPE), (lambda: Scan(G=3), ERR_SHAPE),
    (lambda: Scan(N=24), ERR_UNSUPPORTED), (lambda: Scan(N=128), ERR_UNSUPPORTED), (lambda: Scan(N=4), ERR_UNSUPPORTED),
    (lambda: Scan(b=65536), ERR_UNSUPPORTED), (lambda: Scan(D=(1 << 20) + 2), ERR_UNSUPPORTED),
    (lambda: Scan(T=1 << 31), ERR_UNSUPPORTED), (lambda: Scan(strides=(-1,) + (64,) * 9), ERR_SHAPE),
    (lambda: Scan(strides=(64,) * 9 + (1 << 60,)), ERR_SHAPE),
    (lambda: Norm(rows=-1), ERR_SHAPE), (lambda: Norm(dim=0), ERR_SHAPE), (lambda: Norm(G=3), ERR_SHAPE),
    (lambda: Norm(dim=(1 << 20) + 2), ERR_UNSUPPORTED), (lambda: Norm(rows=1 << 31), ERR_UNSUPPORTED),
    (lambda: Norm(b=1 << 20, rows=1 << 11), ERR_UNSUPPORTED), (lambda: Norm(b=-1), ERR_SHAPE),
    (lambda: Norm(b=1 << 62, rows=4), ERR_UNSUPPORTED),
    (lambda: Norm(xs=-64), ERR_SHAPE), (lambda: Norm(eps=-1.0), ERR_ARGS), (lambda: Norm(eps=float("nan")), ERR_ARGS),
    (lambda: Norm(eps=float("inf")), ERR_ARGS),
    (lambda: Verify(b=-1), ERR_SHAPE), (lambda: Verify(K=-1), ERR_SHAPE), (lambda: Verify(V=0), ERR_SHAPE),
    (lambda: Verify(b=65536), ERR_UNSUPPORTED), (lambda: Verify(V=1 << 31), ERR_UNSUPPORTED),
    (lambda: Verify(strides=(400, -1, 300, 100)), ERR_SHAPE),
])
def test_sizes_and_strides(make, status):
    assert make()() == status
    assert ssd.ssd_last_error()


@pytest.mark.parametrize("cls", [Conv, Scan, Norm, Verify])
def test_shape_and_dtype(cls):
    c = cls()
    c.dtype = 5
    assert c() == ERR_ARGS
    c = cls()
    c.shape = None
    assert c() == ERR_NULL


@pytest.mark.parametrize("cls,keys", [
    (Conv, ["x", "weight", "out0", "out1", "out2"]), (Scan, ["u", "delta", "A", "B", "C", "y"]), (Norm, ["x", "out"]),
    (Verify, ["p", "u", "n", "next", "tok"]),
])
def test_required_pointers(cls, keys):
    for k in keys:
        c = cls()
        c.p[k] = None
        assert c() == ERR_NULL, k


@pytest.mark.parametrize("cls,keys", [
    (Conv, [("x", 1), ("weight", 2), ("bias", 1), ("init", 1), ("out2", 1), ("final", 1), ("idx", 2), ("at", 1)]),
    (Scan, [("u", 1), ("delta", 1), ("A", 8), ("B", 1), ("D", 2), ("z", 1), ("init", 8), ("y", 1), ("final", 4),
            ("idx", 1), ("at", 8), ("ws", 8)]),
    (Norm, [("x", 1), ("z", 1), ("weight", 2), ("out", 1)]),
    (Verify, [("p", 1), ("q", 1), ("tok", 2), ("lens", 1), ("u", 2), ("n", 2), ("next", 2), ("tokens", 1), ("ws", 8)]),
])
def test_alignment(cls, keys):
    for k, off in keys:
        c = cls()
        c.p[k] += off
        assert c() == ERR_ALIGN, k


@pytest.mark.parametrize("cls,pairs", [
    (Conv, [("out0", "x"), ("out1", "out0"), ("final", "x"), ("at", "init"), ("at", "final"), ("out2", "weight"),
            ("final", "idx")]),
    (Scan, [("y", "u"), ("y", "delta"), ("y", "z"), ("final", "A"), ("at", "init"), ("at", "final"), ("y", "B"),
            ("final", "y")]),
    (Norm, [("out", "weight")]),
    (Verify, [("n", "p"), ("next", "n"), ("tokens", "tok"), ("tokens", "u"), ("n", "lens"), ("next", "q")]),
])
def test_overlaps(cls, pairs):
    for a, b in pairs:
        c = cls()
        c.p[a] = c.p[b]
        assert c() == ERR_ALIAS, (a, b)
    # One byte range into another, from below.
    c = Conv()
    c.p["final"] = c.p["init"] + 16                   # in place only where the state is the same
    assert c() == ERR_ALIAS
    c = Scan()
    c.p["final"] = c.p["init"] + 16
    assert c() == ERR_ALIAS
    c = Norm()
    c.p["out"] = c.p["x"] + 16
    assert c() == ERR_ALIAS
    # out is dense, x is not (also where both end at the same byte).
    for c in (Norm(xs=128), Norm(b=2, rows=3, xs=128, xb=64)):
        c.p["out"] = c.p["x"]
        assert c() == ERR_ALIAS


def test_index_pairs_activation_and_workspaces():
    for cls in (Conv, Scan):
        for k in ("idx", "at"):
            c = cls()
            c.p[k] = None
            assert c() == ERR_ARGS
    c = Conv()
    c.scalars["act"] = 2
    assert c() == ERR_ARGS
    c = Conv(ch=(64, 16, 0))
    assert c() == ERR_NULL                             # out2 without channels
    big = Scan(b=1, T=4096, D=64, G=1)
    need = ssd.ssd_selective_scan_workspace_bytes(big.shape, BF16)
    if need:
        big.scalars["ws_bytes"] = need - 1
        assert big() == ERR_WORKSPACE
        big.p["ws"] = None
        big.scalars["ws_bytes"] = need
        assert big() == ERR_WORKSPACE
        big.p["ws"] = big.p["y"]
        assert big() == ERR_ALIAS
    big = Verify(b=1, V=200000)
    need = ssd.ssd_verify_workspace_bytes(big.shape, F32)
    if need:
        big.dtype = F32
        big.scalars["ws_bytes"] = need - 1
        assert big() == ERR_WORKSPACE
        big.p["ws"] = None
        big.scalars["ws_bytes"] = need
        assert big() == ERR_WORKSPACE


def test_nothing_to_do():
    for c in (Conv(b=0), Scan(b=0), Norm(rows=0), Verify(b=0)):
        for k in c.p:
            c.p[k] = None
        assert c() == OK
    for c in (Conv(T=0), Scan(T=0)):
        c.p["final"] = c.p["idx"] = c.p["at"] = None
        assert c() == OK


def test_workspace_queries_of_invalid_shapes():
    assert ssd.ssd_selective_scan_workspace_bytes(Scan(N=24).shape, BF16) == 0 and ssd.ssd_last_error()
    assert ssd.ssd_verify_workspace_bytes(Verify(V=0).shape, BF16) == 0 and ssd.ssd_last_error()


# ------------------------------------------------ the binding's own checks
def z(*shape, dtype=torch.bfloat16):
    return torch.zeros(*shape, dtype=dtype)


f = torch.float32


def conv_args():
    return dict(x=z(2, 5, 24), weight=z(24, 4, dtype=f), bias=z(24, dtype=f), init_state=z(2, 3, 24),
                state_out_idx=z(2, dtype=torch.int32))


def scan_args():
    return dict(u=z(2, 5, 24), delta=z(2, 5, 24), A=z(24, 16, dtype=f), B=z(2, 5, 2, 16), C=z(2, 5, 2, 16),
                D=z(24, dtype=f), z=z(2, 5, 24), delta_bias=z(24, dtype=f), init_state=z(2, 24, 16, dtype=f),
                state_out_idx=z(2, dtype=torch.int32))


def norm_args():
    return dict(x=z(6, 24), z=z(6, 24), weight=z(24, dtype=f))


def verify_args():
    return dict(target_probs=z(2, 4, 50, dtype=f), draft_tokens=z(2, 3, dtype=torch.int32), uniforms=z(2, 4, dtype=f),
                draft_probs=z(2, 3, 50, dtype=f), draft_lens=z(2, dtype=torch.int32))


CALLS = {"conv": (ssd.ssd_causal_conv_fwd, conv_args), "scan": (ssd.ssd_selective_scan_fwd, scan_args),
         "norm": (ssd.ssd_gated_norm_fwd, norm_args), "verify": (ssd.ssd_verify_drafts, verify_args)}


@pytest.mark.parametrize("op,key", [(op, k) for op, (_, a) in CALLS.items() for k in a() if k not in
                                    ("x", "u", "target_probs")])
def test_binding_refuses_wrong_shape_type_and_layout(op, key):
    call, args = CALLS[op]
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
    call, args = CALLS[op]
    a = args()
    with pytest.raises(ValueError, match="GPU"):
        call(**a)
    first = next(iter(a))
    with pytest.raises(TypeError):
        call(**dict(a, **{first: a[first].half()}))
    with pytest.raises(ValueError):
        call(**dict(a, **{first: a[first].reshape(-1)}))


def test_binding_refuses_outputs_and_options():
    a = conv_args()
    for bad in ([24, 1], [], [0, 24], [8, 8, 4, 4], [30, -6]):
        with pytest.raises(ValueError, match="split"):
            ssd.ssd_causal_conv_fwd(**a, split=bad)
    with pytest.raises(ValueError, match="activation"):
        ssd.ssd_causal_conv_fwd(**a, activation="relu")
    with pytest.raises(ValueError, match="out"):
        ssd.ssd_causal_conv_fwd(**a, split=[16, 8], out=[z(2, 5, 16)])
    with pytest.raises(ValueError, match="out"):
        ssd.ssd_causal_conv_fwd(**a, split=[16, 8], out=[z(2, 5, 16), z(2, 5, 16)])
    with pytest.raises(ValueError, match="final_state"):
        ssd.ssd_causal_conv_fwd(**a, final_state=z(2, 4, 24))
    with pytest.raises(ValueError, match="state_out"):
        ssd.ssd_causal_conv_fwd(**dict(a, state_out_idx=None), state_out=z(2, 3, 24))
    s = scan_args()
    with pytest.raises(ValueError, match="y"):
        ssd.ssd_selective_scan_fwd(**s, y=z(2, 5, 23))
    with pytest.raises(ValueError, match="state_out"):
        ssd.ssd_selective_scan_fwd(**dict(s, state_out_idx=None), state_out=z(2, 24, 16, dtype=f))
    with pytest.raises(TypeError, match="workspace"):
        ssd.ssd_selective_scan_fwd(**s, workspace=z(100, dtype=f))
    n = norm_args()
    with pytest.raises(ValueError, match="out"):
        ssd.ssd_gated_norm_fwd(**n, out=z(6, 23))
    v = verify_args()
    with pytest.raises(TypeError, match="n_accepted"):
        ssd.ssd_verify_drafts(**v, n_accepted=z(2, dtype=torch.int64))
    with pytest.raises(ValueError, match="tokens"):
        ssd.ssd_verify_drafts(**v, tokens=z(2, 3, dtype=torch.int32))
