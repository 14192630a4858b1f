"""Python binding of libssd, the MI355X (gfx950) SSD chunked-scan forward and
the operators around it.

Argument marshalling only: every step of the computation runs in the HIP
kernels of ``libssd.so`` (built from ``csrc/`` by ``build.py``).  torch
supplies device memory and the current stream.  The functions carry the
names of the C entry points declared in ``include/ssd.h``; see there for the
operation, layouts, ownership and error behaviour.

There is no fallback: if the library is missing, every call raises.
"""
from __future__ import annotations

import ctypes
import os

__all__ = [
    "SsdError", "ssd_abi_version", "ssd_status_string", "ssd_last_error", "ssd_workspace_bytes",
    "ssd_get_workspace_layout", "ssd_select_path", "ssd_chunk_scan_fwd", "ssd_chunk_scan_fwd_ex",
    "ssd_chunk_scan_fwd_noalloc", "ssd_state_correction", "ssd_causal_conv_fwd", "ssd_selective_scan_fwd",
    "ssd_selective_scan_workspace_bytes", "ssd_gated_norm_fwd", "ssd_verify_drafts", "ssd_verify_workspace_bytes",
    "SSD_NOALLOC_SCRATCH_BYTES", "workspace_views", "library_path", "SSD_PATH_AUTO", "SSD_PATH_ONE_CHUNK", "SSD_PATH_SINGLE_PASS",
    "SSD_PATH_CHUNK_PARALLEL",
]

_PKG = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_PKG, "libssd.so")
_FAST_PATH = os.path.join(_PKG, "_fastcall.so")
_lib = None
# The short way of the operators around the scan for calls that fit as they
# are (csrc/fastcall.cpp): the same checks, allocations and C call without
# Python's share of their time.  It returns None for any other call, which the
# code here then makes or refuses.
_fast = None

SSD_DTYPE_F32 = 0
SSD_DTYPE_BF16 = 1
SSD_NOALLOC_SCRATCH_BYTES = 64 << 20
SSD_PATH_AUTO = 0
SSD_PATH_ONE_CHUNK = 1
SSD_PATH_SINGLE_PASS = 2
SSD_PATH_CHUNK_PARALLEL = 3
PATH_NAMES = {SSD_PATH_AUTO: "auto", SSD_PATH_ONE_CHUNK: "one_chunk", SSD_PATH_SINGLE_PASS: "single_pass",
              SSD_PATH_CHUNK_PARALLEL: "chunk_parallel"}
STATUS = {0: "SSD_OK", 1: "SSD_ERR_NULL", 2: "SSD_ERR_SHAPE", 3: "SSD_ERR_CHUNK", 4: "SSD_ERR_ALIGN",
          5: "SSD_ERR_WORKSPACE", 6: "SSD_ERR_ALIAS", 7: "SSD_ERR_ARGS", 8: "SSD_ERR_HIP",
          9: "SSD_ERR_UNSUPPORTED"}


class ssd_shape(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int64), ("seqlen", ctypes.c_int64), ("nheads", ctypes.c_int64),
                ("headdim", ctypes.c_int64), ("dstate", ctypes.c_int64), ("ngroups", ctypes.c_int64)]


class ssd_workspace_layout(ctypes.Structure):
    _fields_ = [("cumsum_offset", ctypes.c_size_t), ("ct_offset", ctypes.c_size_t),
                ("dt_decay_offset", ctypes.c_size_t), ("states_offset", ctypes.c_size_t),
                ("prev_offset", ctypes.c_size_t), ("hj_offset", ctypes.c_size_t),
                ("total_bytes", ctypes.c_size_t), ("nchunks", ctypes.c_int64)]


class ssd_conv_shape(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int64), ("seqlen", ctypes.c_int64), ("channels", ctypes.c_int64 * 3),
                ("width", ctypes.c_int64), ("x_batch_stride", ctypes.c_int64), ("x_token_stride", ctypes.c_int64)]


class ssd_selective_shape(ctypes.Structure):
    _fields_ = [(k, ctypes.c_int64) for k in (
        "batch", "seqlen", "channels", "dstate", "ngroups", "u_batch_stride", "u_token_stride",
        "delta_batch_stride", "delta_token_stride", "z_batch_stride", "z_token_stride",
        "B_batch_stride", "B_token_stride", "C_batch_stride", "C_token_stride")]


class ssd_norm_shape(ctypes.Structure):
    _fields_ = [(k, ctypes.c_int64) for k in (
        "batch", "seqlen", "dim", "ngroups", "x_batch_stride", "x_token_stride", "z_batch_stride", "z_token_stride")]


class ssd_verify_shape(ctypes.Structure):
    _fields_ = [(k, ctypes.c_int64) for k in ("batch", "drafts", "vocab", "target_batch_stride",
                                              "target_row_stride", "draft_batch_stride", "draft_row_stride")]


class SsdError(RuntimeError):
    def __init__(self, status: int, detail: str):
        self.status = status
        self.name = STATUS.get(status, str(status))
        super().__init__(f"{self.name}: {detail}")


def library_path() -> str:
    return _LIB_PATH


def _load():
    global _lib, _fast
    if _lib is not None:
        return _lib
    if not os.path.exists(_LIB_PATH):
        raise RuntimeError(f"{_LIB_PATH} is not built; run `python -m mamba_ssd_scan_06_amd.build`")
    # torch ships its own HIP runtime under the same soname; loading torch
    # first makes libssd bind to that one, so torch's streams and memory are
    # the library's too (one runtime per process).
    import torch  # noqa: F401
    lib = ctypes.CDLL(_LIB_PATH)
    vp, sz, i32 = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int
    shp = ctypes.POINTER(ssd_shape)
    lib.ssd_workspace_bytes.argtypes = [shp, i32, i32]
    lib.ssd_workspace_bytes.restype = sz
    lib.ssd_get_workspace_layout.argtypes = [shp, i32, i32, ctypes.POINTER(ssd_workspace_layout)]
    lib.ssd_get_workspace_layout.restype = i32
    lib.ssd_select_path.argtypes = [shp, i32, i32]
    lib.ssd_select_path.restype = i32
    lib.ssd_chunk_scan_fwd.argtypes = [vp, vp, vp, vp, vp, vp, vp, i32, vp, vp, vp, vp, shp, i32, vp, sz, vp]
    lib.ssd_chunk_scan_fwd.restype = i32
    lib.ssd_chunk_scan_fwd_ex.argtypes = [vp, vp, vp, vp, vp, vp, vp, i32, vp, vp, vp, vp, shp, i32, vp, sz, vp,
                                          i32, ctypes.POINTER(vp), i32, ctypes.POINTER(i32),
                                          ctypes.POINTER(ctypes.c_char_p)]
    lib.ssd_chunk_scan_fwd_ex.restype = i32
    lib.ssd_chunk_scan_fwd_noalloc.argtypes = [vp, vp, vp, vp, vp, vp, vp, i32, vp, vp, vp, vp, shp, i32, vp]
    lib.ssd_chunk_scan_fwd_noalloc.restype = i32
    lib.ssd_state_correction.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, shp, i32, vp]
    lib.ssd_state_correction.restype = i32
    lib.ssd_causal_conv_fwd.argtypes = [vp, vp, vp, vp, i32, vp, vp, vp, vp, vp, vp, ctypes.POINTER(ssd_conv_shape),
                                        i32, vp]
    lib.ssd_causal_conv_fwd.restype = i32
    sel = ctypes.POINTER(ssd_selective_shape)
    lib.ssd_selective_scan_fwd.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, i32, vp, vp, vp, vp, vp, sel, i32, vp, sz,
                                           vp]
    lib.ssd_selective_scan_fwd.restype = i32
    lib.ssd_selective_scan_workspace_bytes.argtypes = [sel, i32]
    lib.ssd_selective_scan_workspace_bytes.restype = sz
    lib.ssd_gated_norm_fwd.argtypes = [vp, vp, vp, vp, ctypes.c_float, i32, ctypes.POINTER(ssd_norm_shape), i32, vp]
    lib.ssd_gated_norm_fwd.restype = i32
    ver = ctypes.POINTER(ssd_verify_shape)
    lib.ssd_verify_drafts.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, ver, i32, vp, sz, vp]
    lib.ssd_verify_drafts.restype = i32
    lib.ssd_verify_workspace_bytes.argtypes = [ver, i32]
    lib.ssd_verify_workspace_bytes.restype = sz
    lib.ssd_status_string.argtypes = [i32]
    lib.ssd_status_string.restype = ctypes.c_char_p
    lib.ssd_last_error.argtypes = []
    lib.ssd_last_error.restype = ctypes.c_char_p
    lib.ssd_abi_version.argtypes = []
    lib.ssd_abi_version.restype = i32
    if os.path.exists(_FAST_PATH):
        import importlib.util

        spec = importlib.util.spec_from_file_location(__name__ + "._fastcall", _FAST_PATH)
        fast = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(fast)
        fast.bind(*(ctypes.cast(f, ctypes.c_void_p).value for f in (
            lib.ssd_causal_conv_fwd, lib.ssd_selective_scan_fwd, lib.ssd_selective_scan_workspace_bytes,
            lib.ssd_gated_norm_fwd, lib.ssd_verify_drafts, lib.ssd_verify_workspace_bytes)))
        fast.raw_stream = torch._C._cuda_getCurrentRawStream if torch.cuda.is_available() else None
        _fast = fast
    _lib = lib
    return lib


def ssd_abi_version() -> int:
    return int(_load().ssd_abi_version())


def ssd_status_string(status: int) -> str:
    return _load().ssd_status_string(status).decode()


def ssd_last_error() -> str:
    return _load().ssd_last_error().decode()


def _check(status: int):
    if status != 0:
        raise SsdError(status, ssd_last_error())


def make_shape(batch, seqlen, nheads, headdim, dstate, ngroups) -> ssd_shape:
    return ssd_shape(int(batch), int(seqlen), int(nheads), int(headdim), int(dstate), int(ngroups))


def ssd_workspace_bytes(shape: ssd_shape, chunk_size: int, dtype: int) -> int:
    return int(_load().ssd_workspace_bytes(ctypes.byref(shape), int(chunk_size), int(dtype)))


def ssd_get_workspace_layout(shape: ssd_shape, chunk_size: int, dtype: int) -> ssd_workspace_layout:
    out = ssd_workspace_layout()
    _check(_load().ssd_get_workspace_layout(ctypes.byref(shape), int(chunk_size), int(dtype), ctypes.byref(out)))
    return out


def ssd_select_path(shape: ssd_shape, chunk_size: int, dtype: int) -> int:
    path = int(_load().ssd_select_path(ctypes.byref(shape), int(chunk_size), int(dtype)))
    if path < 0:
        raise SsdError(7, ssd_last_error())
    return path


def _dtype_code(torch, t, name="x") -> int:
    if t.dtype == torch.bfloat16:
        return SSD_DTYPE_BF16
    if t.dtype == torch.float32:
        return SSD_DTYPE_F32
    raise TypeError(f"{name} must be bfloat16 or float32, got {t.dtype}")


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def ssd_chunk_scan_fwd(x, dt, A, B, C, D=None, init_state=None, chunk_size: int = 256, state_out_idx=None, *,
                       y=None, final_state=None, return_final_state: bool = True, state_out=None,
                       workspace=None, stream=None):
    """Run the SSD forward on torch device tensors.

    x [b,T,H,P] bf16|fp32, dt [b,T,H] fp32, A [H] fp32, B/C [b,T,G,N] like x,
    D [H] fp32 or None, init_state [b,H,P,N] fp32 or None, state_out_idx [b]
    int32 or None.  Outputs are allocated when not given; given ones must
    have the exact shape, dtype and device.  Returns (y, final_state or None,
    state_out or None).  Raises ValueError/TypeError for a tensor that does
    not fit the call (before anything runs) and SsdError on any status other
    than SSD_OK.
    """
    y, final_state, state_out, _ = _run(x, dt, A, B, C, D, init_state, chunk_size, state_out_idx, y, final_state,
                                        return_final_state, state_out, workspace, stream, SSD_PATH_AUTO, None)
    return y, final_state, state_out


def ssd_chunk_scan_fwd_ex(x, dt, A, B, C, D=None, init_state=None, chunk_size: int = 256, state_out_idx=None, *,
                          path: int = SSD_PATH_AUTO, marks=(), y=None, final_state=None,
                          return_final_state: bool = True, state_out=None, workspace=None, stream=None):
    """ssd_chunk_scan_fwd on a chosen path (SSD_PATH_*), recording the HIP
    events `marks` (raw hipEvent_t handles as ints): marks[0] before the
    first kernel, marks[k] after the k-th.  Returns (y, final_state,
    state_out, names of the kernels that marks[1:] end)."""
    return _run(x, dt, A, B, C, D, init_state, chunk_size, state_out_idx, y, final_state, return_final_state,
                state_out, workspace, stream, int(path), list(marks))


def ssd_chunk_scan_fwd_noalloc(x, dt, A, B, C, D=None, init_state=None, chunk_size: int = 256,
                               state_out_idx=None, *, y=None, final_state=None, return_final_state: bool = True,
                               state_out=None, stream=None):
    """ssd_chunk_scan_fwd through the entry point that allocates nothing: a
    workspace, when the call needs one, is the library's static device
    scratch (at most SSD_NOALLOC_SCRATCH_BYTES).  Pass y, final_state and
    state_out to allocate nothing here either; missing ones are allocated
    by torch before the call."""
    y, final_state, state_out, _ = _run(x, dt, A, B, C, D, init_state, chunk_size, state_out_idx, y, final_state,
                                        return_final_state, state_out, None, stream, SSD_PATH_AUTO, None,
                                        noalloc=True)
    return y, final_state, state_out


def ssd_state_correction(y, dt, A, C, h_in, shard_final=None, final_state=None, state_out_idx=None,
                         state_out=None, *, stream=None):
    """Sequence-shard correction in place (see ssd_state_correction in
    include/ssd.h): y [b,T,H,P] holds the shard's outputs from a zero initial
    state and becomes those from h_in [b,H,P,N]; final_state (may be
    shard_final itself) receives shard_final + exp(cs_{T-1}) h_in; state_out,
    given with state_out_idx, gains exp(cs_j) h_in.  dt, A, C as for the
    shard's forward.  Returns (y, final_state, state_out)."""
    import torch

    if y.dim() != 4 or C.dim() != 4:
        raise ValueError("y must be [b,T,H,P] and C [b,T,G,N]")
    b, T, H, P = y.shape
    G, N = C.shape[2], C.shape[3]
    code = _dtype_code(torch, y)
    dev = y.device
    state_shape = (b, H, P, N)
    _expect("y", y, y.shape, y.dtype, dev)
    _expect("C", C, (b, T, G, N), y.dtype, dev)
    _expect("dt", dt, (b, T, H), torch.float32, dev)
    _expect("A", A, (H,), torch.float32, dev)
    _expect("h_in", h_in, state_shape, torch.float32, dev)
    if shard_final is not None:
        _expect("shard_final", shard_final, state_shape, torch.float32, dev)
    if final_state is not None:
        _expect("final_state", final_state, state_shape, torch.float32, dev)
    if state_out_idx is not None:
        _expect("state_out_idx", state_out_idx, (b,), torch.int32, dev)
    if state_out is not None:
        _expect("state_out", state_out, state_shape, torch.float32, dev)
    if (state_out is None) != (state_out_idx is None):
        raise ValueError("state_out and state_out_idx go together")
    if not y.is_cuda:
        raise ValueError(f"tensors must be on a GPU device, y is on {dev}")
    lib = _load()
    if stream is None:
        stream = torch.cuda.current_stream(dev).cuda_stream
    _check(lib.ssd_state_correction(_ptr(y), _ptr(dt), _ptr(A), _ptr(C), _ptr(h_in), _ptr(shard_final),
                                    _ptr(final_state), _ptr(state_out_idx), _ptr(state_out),
                                    ctypes.byref(make_shape(b, T, H, P, N, G)), code,
                                    ctypes.c_void_p(stream) if stream else None))
    return y, final_state, state_out


def _expect(name, t, shape, dtype, device):
    """Checks one tensor argument; `shape` is the exact shape required."""
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, x on {device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _run(x, dt, A, B, C, D, init_state, chunk_size, state_out_idx, y, final_state, return_final_state, state_out,
         workspace, stream, path, marks, noalloc=False):
    import torch

    if x.dim() != 4 or B.dim() != 4:
        raise ValueError("x must be [b,T,H,P] and B, C [b,T,G,N]")
    b, T, H, P = x.shape
    G, N = B.shape[2], B.shape[3]
    code = _dtype_code(torch, x)
    dev = x.device
    state_shape = (b, H, P, N)
    _expect("x", x, x.shape, x.dtype, dev)
    _expect("B", B, (b, T, G, N), x.dtype, dev)
    _expect("C", C, (b, T, G, N), x.dtype, dev)
    _expect("dt", dt, (b, T, H), torch.float32, dev)
    _expect("A", A, (H,), torch.float32, dev)
    if D is not None:
        _expect("D", D, (H,), torch.float32, dev)
    if init_state is not None:
        _expect("init_state", init_state, state_shape, torch.float32, dev)
    if state_out_idx is not None:
        _expect("state_out_idx", state_out_idx, (b,), torch.int32, dev)
    elif state_out is not None:
        raise ValueError("state_out needs state_out_idx")
    if y is not None:
        _expect("y", y, x.shape, x.dtype, dev)
    if final_state is not None:
        _expect("final_state", final_state, state_shape, torch.float32, dev)
    if state_out is not None:
        _expect("state_out", state_out, state_shape, torch.float32, dev)
    if workspace is not None:
        if workspace.dim() != 1:
            raise ValueError("workspace must be a 1-D uint8 tensor")
        _expect("workspace", workspace, workspace.shape, torch.uint8, dev)
    if not x.is_cuda:
        raise ValueError(f"tensors must be on a GPU device, x is on {dev}")

    lib = _load()
    shape = make_shape(b, T, H, P, N, G)
    layout = ssd_get_workspace_layout(shape, chunk_size, code)  # raises the status of an invalid shape
    chosen = ssd_select_path(shape, chunk_size, code)
    run_path = path if path != SSD_PATH_AUTO and chosen != SSD_PATH_AUTO else chosen
    ws_bytes = layout.total_bytes if run_path == SSD_PATH_CHUNK_PARALLEL else 0
    if y is None:
        y = torch.empty_like(x)
    if final_state is None and return_final_state:
        final_state = torch.empty(state_shape, dtype=torch.float32, device=dev)
    if state_out_idx is not None and state_out is None:
        state_out = torch.empty(state_shape, dtype=torch.float32, device=dev)
    if workspace is None and ws_bytes > 0 and not noalloc:
        workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=dev)
    if stream is None:
        stream = torch.cuda.current_stream(dev).cuda_stream
    if noalloc:
        _check(lib.ssd_chunk_scan_fwd_noalloc(
            _ptr(x), _ptr(dt), _ptr(A), _ptr(B), _ptr(C), _ptr(D), _ptr(init_state), int(chunk_size), _ptr(y),
            _ptr(final_state), _ptr(state_out_idx), _ptr(state_out), ctypes.byref(shape), code,
            ctypes.c_void_p(stream) if stream else None))
        return y, final_state, state_out, None
    args = (_ptr(x), _ptr(dt), _ptr(A), _ptr(B), _ptr(C), _ptr(D), _ptr(init_state), int(chunk_size), _ptr(y),
            _ptr(final_state), _ptr(state_out_idx), _ptr(state_out), ctypes.byref(shape), code, _ptr(workspace),
            int(workspace.numel()) if workspace is not None else 0, ctypes.c_void_p(stream) if stream else None)
    if marks is None:
        _check(lib.ssd_chunk_scan_fwd(*args))
        return y, final_state, state_out, None
    n = len(marks)
    arr = (ctypes.c_void_p * max(n, 1))(*[ctypes.c_void_p(int(m)) for m in marks])
    names = (ctypes.c_char_p * max(n, 1))()
    count = ctypes.c_int(0)
    _check(lib.ssd_chunk_scan_fwd_ex(*args, int(path), arr, n, ctypes.byref(count), names))
    used = min(count.value, n - 1) if n > 0 else 0
    return y, final_state, state_out, [names[k].decode() for k in range(used)]


# ------------------------------------------------ operators around the scan
def _addr(t):
    return None if t is None else t.data_ptr()


def _dense(name, t, shape, dtype, device):
    """_expect at the cost of one condition for a tensor that fits (single
    tokens are bound by the time of the call itself)."""
    if t.shape != shape or t.dtype is not dtype or t.device != device or not t.is_contiguous():
        _expect(name, t, shape, dtype, device)


def _strided(name, t, shape, dtype, device, inner=1):
    """Checks a tensor argument whose leading dimensions may be strided and
    whose last `inner` dimensions are contiguous; returns its strides."""
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    st = t.stride()
    if st[-1] == 1 and (inner == 1 or st[-2] == shape[-1]):
        return st
    want = 1
    for k in range(1, inner + 1):
        if st[-k] != want and shape[-k] > 1 and t.numel() > 0:
            raise ValueError(f"{name} must be contiguous in its last {inner} dimension(s)" if inner > 1
                             else f"{name} must be contiguous in its last dimension")
        want *= shape[-k]
    return st


def _elsewhere(torch, t, stream):
    """Whether a call on tensor t has to leave the current device or stream."""
    return t.is_cuda and (stream is not None or t.device.index != torch.cuda.current_device())


def _scope(torch, t, stream):
    """What such a call runs inside: t's device and, where one is given,
    `stream` (a raw handle), so that tensors made by the call belong to the
    stream that uses them."""
    if stream is None:
        return torch.cuda.device(t.device)
    if stream == 0:
        return torch.cuda.stream(torch.cuda.default_stream(t.device))
    return torch.cuda.stream(torch.cuda.ExternalStream(stream, device=t.device))


def _raw_stream(torch, device):
    """The current stream's handle, without making a stream object of it
    (torch.cuda.current_stream takes 2 us, a fifth of a single token's call)."""
    return torch._C._cuda_getCurrentRawStream(device.index) or None


def ssd_causal_conv_fwd(x, weight, bias=None, init_state=None, state_out_idx=None, *, split=None, activation="silu",
                        out=None, final_state=None, return_final_state: bool = True, state_out=None, stream=None):
    """Depthwise causal convolution over tokens (see ssd_causal_conv_fwd in
    include/ssd.h).

    x [b,T,Ch] bf16|fp32 (batch and token strides free, e.g. a slice of a
    projection's output), weight [Ch,W] fp32 (W 2..4), bias [Ch] fp32 or None,
    init_state [b,W-1,Ch] like x or None, state_out_idx [b] int32 or None;
    activation "silu" or None.  With `split` (up to three sizes adding up to
    Ch) the outputs are that many dense tensors [b,T,size], else one.
    `out`, a tensor or with `split` a sequence of them, final_state (may be
    init_state itself) and state_out are allocated when not given.  Returns
    (out, final_state or None, state_out or None); out is a tuple with
    `split`.  Errors as for ssd_chunk_scan_fwd.
    """
    if _fast is not None and x.is_cuda and stream is None and out is None and state_out is None and (
            activation == "silu" or activation is None):
        r = _fast.conv(x, weight, bias, init_state, state_out_idx, split, activation is not None, final_state,
                       return_final_state, _fast.raw_stream(x.device.index))
        if r.__class__ is tuple:
            return r
        if r is not None:
            _check(r)
    import torch

    if x.dim() != 3 or weight.dim() != 2:
        raise ValueError("x must be [b,T,Ch] and weight [Ch,W]")
    if _elsewhere(torch, x, stream):
        with _scope(torch, x, stream):
            return ssd_causal_conv_fwd(x, weight, bias, init_state, state_out_idx, split=split, activation=activation,
                                       out=out, final_state=final_state, return_final_state=return_final_state,
                                       state_out=state_out)
    b, T, ch = x.shape
    w = weight.shape[1]
    code, dtype, dev = _dtype_code(torch, x), x.dtype, x.device
    st = _strided("x", x, x.shape, dtype, dev)
    _dense("weight", weight, (ch, w), torch.float32, dev)
    if activation not in (None, "silu"):
        raise ValueError(f"activation must be 'silu' or None, got {activation!r}")
    sizes = [ch] if split is None else [int(k) for k in split]
    if not 1 <= len(sizes) <= 3 or min(sizes) <= 0 or sum(sizes) != ch:
        raise ValueError(f"split must be one to three positive sizes adding up to {ch}, got {split}")
    held = (b, w - 1, ch)
    if bias is not None:
        _dense("bias", bias, (ch,), torch.float32, dev)
    if init_state is not None:
        _dense("init_state", init_state, held, dtype, dev)
    if state_out_idx is not None:
        _dense("state_out_idx", state_out_idx, (b,), torch.int32, dev)
    elif state_out is not None:
        raise ValueError("state_out needs state_out_idx")
    if out is None:
        outs = None
    else:
        outs = [out] if split is None else list(out)
        if len(outs) != len(sizes):
            raise ValueError(f"out must hold {len(sizes)} tensors, got {len(outs)}")
        for k, (o, n) in enumerate(zip(outs, sizes)):
            _dense("out" if split is None else f"out[{k}]", o, (b, T, n), dtype, dev)
    if final_state is not None:
        _dense("final_state", final_state, held, dtype, dev)
    if state_out is not None:
        _dense("state_out", state_out, held, dtype, dev)
    if not x.is_cuda:
        raise ValueError(f"tensors must be on a GPU device, x is on {dev}")
    lib = _load()
    if outs is None:
        outs = [x.new_empty((b, T, n)) for n in sizes]
    if final_state is None and return_final_state:
        final_state = x.new_empty(held)
    if state_out is None and state_out_idx is not None:
        state_out = x.new_empty(held)
    n = len(sizes)
    shape = ssd_conv_shape(b, T, (*sizes, 0, 0)[:3], w, st[0], st[1])
    _check(lib.ssd_causal_conv_fwd(_addr(x), _addr(weight), _addr(bias), _addr(init_state),
                                   1 if activation == "silu" else 0, outs[0].data_ptr(),
                                   outs[1].data_ptr() if n > 1 else None, outs[2].data_ptr() if n > 2 else None,
                                   _addr(final_state), _addr(state_out_idx), _addr(state_out), ctypes.byref(shape),
                                   code, _raw_stream(torch, dev)))
    return (outs[0] if split is None else tuple(outs)), final_state, state_out


def ssd_selective_scan_workspace_bytes(shape: ssd_selective_shape, dtype: int) -> int:
    return int(_load().ssd_selective_scan_workspace_bytes(ctypes.byref(shape), int(dtype)))


def ssd_selective_scan_fwd(u, delta, A, B, C, D=None, z=None, delta_bias=None, init_state=None, state_out_idx=None, *,
                           delta_softplus: bool = False, y=None, final_state=None, return_final_state: bool = True,
                           state_out=None, workspace=None, stream=None):
    """Selective scan with one decay per channel and state index (see
    ssd_selective_scan_fwd in include/ssd.h).

    u, delta, z [b,T,Dm] bf16|fp32 (batch and token strides free), A [Dm,N]
    fp32, B, C [b,T,G,N] like u (strides free by batch and token), D and
    delta_bias [Dm] fp32 or None, z None for no gate, init_state [b,Dm,N] fp32
    or None, state_out_idx [b] int32 or None.  Outputs and the workspace are
    allocated when not given; final_state may be init_state itself.  Returns
    (y, final_state or None, state_out or None).  Errors as for
    ssd_chunk_scan_fwd.
    """
    if _fast is not None and u.is_cuda and stream is None and y is None and state_out is None and workspace is None:
        r = _fast.scan(u, delta, A, B, C, D, z, delta_bias, init_state, state_out_idx, delta_softplus, final_state,
                       return_final_state, _fast.raw_stream(u.device.index))
        if r.__class__ is tuple:
            return r
        if r is not None:
            _check(r)
    import torch

    if u.dim() != 3 or A.dim() != 2 or B.dim() != 4:
        raise ValueError("u must be [b,T,Dm], A [Dm,N] and B, C [b,T,G,N]")
    if _elsewhere(torch, u, stream):
        with _scope(torch, u, stream):
            return ssd_selective_scan_fwd(u, delta, A, B, C, D, z, delta_bias, init_state, state_out_idx,
                                          delta_softplus=delta_softplus, y=y, final_state=final_state,
                                          return_final_state=return_final_state, state_out=state_out,
                                          workspace=workspace)
    f32 = torch.float32
    b, T, ch = u.shape
    G, N = B.shape[2], B.shape[3]
    code, dtype, dev = _dtype_code(torch, u, "u"), u.dtype, u.device
    su = _strided("u", u, u.shape, dtype, dev)
    sd = _strided("delta", delta, u.shape, dtype, dev)
    sz = _strided("z", z, u.shape, dtype, dev) if z is not None else (0, 0)
    sb = _strided("B", B, (b, T, G, N), dtype, dev, 2)
    sc = _strided("C", C, (b, T, G, N), dtype, dev, 2)
    _dense("A", A, (ch, N), f32, dev)
    if D is not None:
        _dense("D", D, (ch,), f32, dev)
    if delta_bias is not None:
        _dense("delta_bias", delta_bias, (ch,), f32, dev)
    state = (b, ch, N)
    if init_state is not None:
        _dense("init_state", init_state, state, f32, dev)
    if state_out_idx is not None:
        _dense("state_out_idx", state_out_idx, (b,), torch.int32, dev)
    elif state_out is not None:
        raise ValueError("state_out needs state_out_idx")
    if y is not None:
        _dense("y", y, u.shape, dtype, dev)
    if final_state is not None:
        _dense("final_state", final_state, state, f32, dev)
    if state_out is not None:
        _dense("state_out", state_out, state, f32, dev)
    if workspace is not None:
        _dense("workspace", workspace, (workspace.numel(),), torch.uint8, dev)
    if not u.is_cuda:
        raise ValueError(f"tensors must be on a GPU device, u is on {dev}")
    lib = _load()
    shape = ssd_selective_shape(b, T, ch, N, G, su[0], su[1], sd[0], sd[1], sz[0], sz[1], sb[0], sb[1], sc[0], sc[1])
    ref = ctypes.byref(shape)
    ws_bytes = 0
    if workspace is not None:
        ws_bytes = workspace.numel()
    else:
        ws_bytes = lib.ssd_selective_scan_workspace_bytes(ref, code)
        if ws_bytes > 0:
            workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=dev)
    if y is None:
        y = u.new_empty((b, T, ch))
    if final_state is None and return_final_state:
        final_state = A.new_empty(state)
    if state_out is None and state_out_idx is not None:
        state_out = A.new_empty(state)
    _check(lib.ssd_selective_scan_fwd(_addr(u), _addr(delta), _addr(A), _addr(B), _addr(C), _addr(D), _addr(z),
                                      _addr(delta_bias), 1 if delta_softplus else 0, _addr(init_state), _addr(y),
                                      _addr(final_state), _addr(state_out_idx), _addr(state_out), ref, code,
                                      _addr(workspace), ws_bytes, _raw_stream(torch, dev)))
    return y, final_state, state_out


def _two_levels(name, t, b, T):
    """The strides of t[..., :] seen as [b,T,dim], where b and T are the
    products of leading dimensions (b of all but the last of them)."""
    if t.dim() <= 3:
        return (0, t.stride(0) if t.dim() == 2 else 0) if t.dim() < 3 else t.stride()[:2]
    try:
        return t.view(b, T, t.shape[-1]).stride()[:2]
    except RuntimeError:
        raise ValueError(f"{name} of shape {tuple(t.shape)} and strides {t.stride()} cannot be viewed as "
                         f"[{b}, {T}, {t.shape[-1]}]") from None


def ssd_gated_norm_fwd(x, z=None, weight=None, *, ngroups: int = 1, eps: float = 1e-5, norm_before_gate: bool = False,
                       out=None, stream=None):
    """RMS norm with a gate (see ssd_gated_norm_fwd in include/ssd.h).

    x [dim], [T,dim], [b,T,dim] or more leading dimensions (those before the
    last two merge into one) bf16|fp32 and z like it or None, batch and token
    strides free (e.g. a slice of a projection's output); weight [dim] fp32 or
    None; each row is normalised in `ngroups` equal parts.  out (dense; may be x or
    z itself where that is dense) is allocated when not given, and returned.
    Errors as for ssd_chunk_scan_fwd.
    """
    if _fast is not None and x.is_cuda and stream is None and out is None:
        r = _fast.norm(x, z, weight, ngroups, eps, norm_before_gate, _fast.raw_stream(x.device.index))
        if r.__class__ is int:
            _check(r)
        if r is not None:
            return r
    import torch

    if x.dim() < 1:
        raise ValueError("x must be [..., dim]")
    if _elsewhere(torch, x, stream):
        with _scope(torch, x, stream):
            return ssd_gated_norm_fwd(x, z, weight, ngroups=ngroups, eps=eps, norm_before_gate=norm_before_gate,
                                      out=out)
    code, dtype, dev = _dtype_code(torch, x), x.dtype, x.device
    dim = x.shape[-1]
    _strided("x", x, x.shape, dtype, dev)
    if z is not None:
        _strided("z", z, x.shape, dtype, dev)
    if weight is not None:
        _dense("weight", weight, (dim,), torch.float32, dev)
    if out is not None:
        _dense("out", out, x.shape, dtype, dev)
    if not x.is_cuda:
        raise ValueError(f"tensors must be on a GPU device, x is on {dev}")
    lib = _load()
    if out is None:
        out = x.new_empty(x.shape)
    T = x.shape[-2] if x.dim() > 1 else 1
    b = x.numel() // (T * dim) if T * dim else 0
    sx = _two_levels("x", x, b, T)
    sz = _two_levels("z", z, b, T) if z is not None else (0, 0)
    shape = ssd_norm_shape(b, T, dim, ngroups, sx[0], sx[1], sz[0], sz[1])
    _check(lib.ssd_gated_norm_fwd(_addr(x), _addr(z), _addr(weight), _addr(out), eps, 1 if norm_before_gate else 0,
                                  ctypes.byref(shape), code, _raw_stream(torch, dev)))
    return out


def ssd_verify_workspace_bytes(shape: ssd_verify_shape, dtype: int) -> int:
    return int(_load().ssd_verify_workspace_bytes(ctypes.byref(shape), int(dtype)))


def ssd_verify_drafts(target_probs, draft_tokens, uniforms, draft_probs=None, draft_lens=None, *, n_accepted=None,
                      next_token=None, tokens=None, workspace=None, stream=None):
    """Verification of drafted tokens (see ssd_verify_drafts in
    include/ssd.h).

    target_probs [b,K+1,V] bf16|fp32 and draft_probs [b,K,V] like it (or None
    for looked-up drafts), batch and row strides free; draft_tokens [b,K]
    int32, uniforms [b,K+1] fp32 in [0,1), draft_lens [b] int32 or None.
    Outputs and the workspace are allocated when not given.  Returns
    (n_accepted [b], next_token [b], tokens [b,K+1]), all int32: the accepted
    drafts in `tokens` are followed by the next token, then -1.  n_accepted is
    also the state_out_idx of a scan over [last token, drafts].  Errors as for
    ssd_chunk_scan_fwd.
    """
    if _fast is not None and target_probs.is_cuda and stream is None and n_accepted is None and next_token is None \
            and tokens is None and workspace is None:
        r = _fast.verify(target_probs, draft_tokens, uniforms, draft_probs, draft_lens,
                         _fast.raw_stream(target_probs.device.index))
        if r.__class__ is tuple:
            return r
        if r is not None:
            _check(r)
    import torch

    if target_probs.dim() != 3 or target_probs.shape[1] < 1:
        raise ValueError("target_probs must be [b,K+1,V]")
    if _elsewhere(torch, target_probs, stream):
        with _scope(torch, target_probs, stream):
            return ssd_verify_drafts(target_probs, draft_tokens, uniforms, draft_probs, draft_lens,
                                     n_accepted=n_accepted, next_token=next_token, tokens=tokens,
                                     workspace=workspace)
    i32 = torch.int32
    b, rows, V = target_probs.shape
    K = rows - 1
    code, dtype, dev = _dtype_code(torch, target_probs, "target_probs"), target_probs.dtype, target_probs.device
    st = _strided("target_probs", target_probs, target_probs.shape, dtype, dev)
    sd = _strided("draft_probs", draft_probs, (b, K, V), dtype, dev) if draft_probs is not None else (0, 0)
    _dense("draft_tokens", draft_tokens, (b, K), i32, dev)
    _dense("uniforms", uniforms, (b, rows), torch.float32, dev)
    if draft_lens is not None:
        _dense("draft_lens", draft_lens, (b,), i32, dev)
    if n_accepted is not None:
        _dense("n_accepted", n_accepted, (b,), i32, dev)
    if next_token is not None:
        _dense("next_token", next_token, (b,), i32, dev)
    if tokens is not None:
        _dense("tokens", tokens, (b, rows), i32, dev)
    if workspace is not None:
        _dense("workspace", workspace, (workspace.numel(),), torch.uint8, dev)
    if not target_probs.is_cuda:
        raise ValueError(f"tensors must be on a GPU device, target_probs is on {dev}")
    lib = _load()
    shape = ssd_verify_shape(b, K, V, st[0], st[1], sd[0], sd[1])
    ref = ctypes.byref(shape)
    if workspace is not None:
        ws_bytes = workspace.numel()
    else:
        ws_bytes = lib.ssd_verify_workspace_bytes(ref, code)
        if ws_bytes > 0:
            workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=dev)
    if n_accepted is None:
        n_accepted = draft_tokens.new_empty(b)
    if next_token is None:
        next_token = draft_tokens.new_empty(b)
    if tokens is None:
        tokens = draft_tokens.new_empty((b, rows))
    _check(lib.ssd_verify_drafts(_addr(target_probs), _addr(draft_probs), _addr(draft_tokens), _addr(draft_lens),
                                 _addr(uniforms), _addr(n_accepted), _addr(next_token), _addr(tokens), ref, code,
                                 _addr(workspace), ws_bytes, _raw_stream(torch, dev)))
    return n_accepted, next_token, tokens


def workspace_views(workspace, shape: ssd_shape, chunk_size: int, dtype: int):
    """Views into the chunk-parallel path's workspace after a call, by the
    layout of include/ssd.h: cs, ct and dte [b,H,nc,Q] fp32, the chunk states
    from a zero start and the states entering each chunk (entry 0 only with
    init_state), both [b,nc,H,P,N] in the input dtype."""
    import torch

    lay = ssd_get_workspace_layout(shape, chunk_size, dtype)
    nc = lay.nchunks
    b, H, P, N = shape.batch, shape.nheads, shape.headdim, shape.dstate
    n_cs = b * H * nc * chunk_size
    n_st = b * nc * H * P * N
    tdt, esz = (torch.bfloat16, 2) if dtype == SSD_DTYPE_BF16 else (torch.float32, 4)

    def region(off, nbytes, dt, dims):
        return workspace[off:off + nbytes].view(dt).view(*dims)

    tab = (b, H, nc, chunk_size)
    return dict(cs=region(lay.cumsum_offset, 4 * n_cs, torch.float32, tab),
                ct=region(lay.ct_offset, 4 * n_cs, torch.float32, tab),
                dte=region(lay.dt_decay_offset, 4 * n_cs, torch.float32, tab),
                states=region(lay.states_offset, esz * n_st, tdt, (b, nc, H, P, N)),
                prev=region(lay.prev_offset, esz * n_st, tdt, (b, nc, H, P, N)))
