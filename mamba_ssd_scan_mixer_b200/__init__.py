"""Thin Python binding of libmamba2ssd.so, the B200 Mamba-2 mixer-core library.

Argument marshalling only: every step of the mixer runs in the library's CUDA
kernels.  PyTorch supplies device memory and the current stream.  There is no
CPU path: if the library is missing, importing the entry points raises.

Entry points (same names as the C ABI in include/mamba2ssd.h):
    mamba2_prefill_workspace_size(dims) -> int
    mamba2_conv_ssd_prefill(dims, params, xBC, z, dt_raw, y, conv_state, ssm_state,
                            states_in, workspace, stream=None)
    mamba2_ssd_step(dims, params, xBC, z, dt_raw, y, conv_state, ssm_state, stream=None)
Conveniences that allocate outputs and workspace with torch and call the above:
    prefill(...), step(...)

Beside the mixer core:
    gated_scan_prefill(...), gated_scan_step(...), gated_scan_backward(...)
        the gated linear recurrence (one fp32 state a channel, decays from the token)
    state_cache_store(...), state_cache_load(...)
        recurrent states in slots of a cache of 8-bit codes
"""
from __future__ import annotations

import ctypes
import os

__all__ = [
    "Mamba2Dims", "Mamba2Params", "Mamba2Error", "MAMBA2_F32", "MAMBA2_BF16", "lib",
    "library_path", "make_dims", "make_params", "mamba2_prefill_workspace_size",
    "mamba2_conv_ssd_prefill", "mamba2_conv_ssd_prefill_noalloc", "mamba2_ssd_step", "prefill",
    "step", "status_string", "mamba2_prefill_backward_workspace_size",
    "mamba2_conv_ssd_prefill_backward", "prefill_backward",
    "mamba2_prefill_host_workspace_size", "mamba2_conv_ssd_prefill_host", "prefill_host",
    "Mamba2GatedScanDims", "GATED_SCAN_CHUNK", "make_gated_scan_dims",
    "mamba2_gated_scan_workspace_size", "mamba2_gated_scan_backward_workspace_size",
    "gated_scan_checkpoints", "gated_scan_prefill", "gated_scan_step", "gated_scan_backward",
    "Mamba2StateCacheDims", "state_cache", "state_cache_store", "state_cache_load",
]

MAMBA2_F32, MAMBA2_BF16 = 0, 1
_PKG = os.path.dirname(os.path.abspath(__file__))
# MAMBA2SSD_LIBRARY selects another build of the library, e.g. the bounds-checked
# libmamba2ssd_checked.so (see build.py)
library_path = os.environ.get("MAMBA2SSD_LIBRARY") or os.path.join(_PKG, "libmamba2ssd.so")


class Mamba2Dims(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int64), ("seqlen", ctypes.c_int64),
                ("nheads", ctypes.c_int32), ("headdim", ctypes.c_int32),
                ("dstate", ctypes.c_int32), ("ngroups", ctypes.c_int32),
                ("d_conv", ctypes.c_int32), ("chunk_size", ctypes.c_int32),
                ("io_dtype", ctypes.c_int32), ("norm_before_gate", ctypes.c_int32),
                ("norm_eps", ctypes.c_float)]


class Mamba2Params(ctypes.Structure):
    _fields_ = [("conv_w", ctypes.c_void_p), ("conv_b", ctypes.c_void_p),
                ("dt_bias", ctypes.c_void_p), ("A", ctypes.c_void_p), ("D", ctypes.c_void_p),
                ("norm_w", ctypes.c_void_p)]


class Mamba2GatedScanDims(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int64), ("seqlen", ctypes.c_int64), ("width", ctypes.c_int32),
                ("io_dtype", ctypes.c_int32), ("decay_scale", ctypes.c_float)]


class Mamba2StateCacheDims(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int64), ("row", ctypes.c_int64), ("nslots", ctypes.c_int64),
                ("block", ctypes.c_int32), ("format", ctypes.c_int32),
                ("state_dtype", ctypes.c_int32)]


class Mamba2Error(RuntimeError):
    def __init__(self, status: int, where: str):
        super().__init__(f"{where}: {status_string(status)} (status {status})")
        self.status = status


_lib = None


def lib() -> ctypes.CDLL:
    """The loaded library; raises if it has not been built (no fallback)."""
    global _lib
    if _lib is None:
        if not os.path.exists(library_path):
            raise RuntimeError(
                f"{library_path} is missing: build it with "
                "`python -m mamba_ssd_scan_mixer_b200.build` (there is no CPU fallback)")
        L = ctypes.CDLL(library_path)
        vp, i64, i32, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_size_t
        pd, pp = ctypes.POINTER(Mamba2Dims), ctypes.POINTER(Mamba2Params)
        L.mamba2_status_string.restype = ctypes.c_char_p
        L.mamba2_status_string.argtypes = [ctypes.c_int]
        L.mamba2_version.restype = ctypes.c_int
        L.mamba2_version.argtypes = []
        L.mamba2_prefill_workspace_size.restype = sz
        L.mamba2_prefill_workspace_size.argtypes = [pd]
        L.mamba2_conv_ssd_prefill.restype = ctypes.c_int
        L.mamba2_conv_ssd_prefill.argtypes = [pd, pp, vp, i64, vp, i64, vp, i64, vp, vp, vp, i32,
                                              vp, sz, vp]
        L.mamba2_prefill_host_workspace_size.restype = sz
        L.mamba2_prefill_host_workspace_size.argtypes = [pd]
        L.mamba2_conv_ssd_prefill_host.restype = ctypes.c_int
        L.mamba2_conv_ssd_prefill_host.argtypes = [pd, pp, vp, i64, vp, i64, vp, i64, vp, vp, vp,
                                                   i32, vp, sz, vp]
        L.mamba2_prefill_varlen_workspace_size.restype = sz
        L.mamba2_prefill_varlen_workspace_size.argtypes = [pd]
        L.mamba2_conv_ssd_prefill_varlen.restype = ctypes.c_int
        L.mamba2_conv_ssd_prefill_varlen.argtypes = [pd, pp, vp, i64, vp, i64, vp, i64, vp, vp,
                                                     vp, vp, i32, vp, sz, vp]
        L.mamba2_conv_ssd_prefill_noalloc.restype = ctypes.c_int
        L.mamba2_conv_ssd_prefill_noalloc.argtypes = [pd, pp, vp, i64, vp, i64, vp, i64, vp, vp,
                                                      vp, i32, vp]
        L.mamba2_device_errors.restype = ctypes.c_int
        L.mamba2_device_errors.argtypes = [ctypes.POINTER(ctypes.c_uint)]
        L.mamba2_debug_stall_waits.restype = ctypes.c_int
        L.mamba2_debug_stall_waits.argtypes = [ctypes.c_int]
        L.mamba2_prefill_backward_workspace_size.restype = sz
        L.mamba2_prefill_backward_workspace_size.argtypes = [pd]
        L.mamba2_conv_ssd_prefill_backward.restype = ctypes.c_int
        L.mamba2_conv_ssd_prefill_backward.argtypes = ([pd, pp, vp, i64, vp, i64, vp, i64]
                                                       + [vp] * 15 + [vp, sz, vp])
        L.mamba2_ssd_step.restype = ctypes.c_int
        L.mamba2_ssd_step.argtypes = [pd, pp, vp, i64, vp, i64, vp, i64, vp, vp, vp, vp]
        pg, pc = ctypes.POINTER(Mamba2GatedScanDims), ctypes.POINTER(Mamba2StateCacheDims)
        for f in (L.mamba2_gated_scan_workspace_size, L.mamba2_gated_scan_backward_workspace_size,
                  L.mamba2_gated_scan_checkpoint_count):
            f.restype, f.argtypes = sz, [pg, ctypes.c_int]
        rows4 = [vp, i64] * 4
        L.mamba2_gated_scan_prefill.restype = ctypes.c_int
        L.mamba2_gated_scan_prefill.argtypes = [pg, vp, *rows4, vp, vp, vp, i32, vp, vp, sz, vp]
        L.mamba2_gated_scan_step.restype = ctypes.c_int
        L.mamba2_gated_scan_step.argtypes = [pg, vp, *rows4, vp, vp, vp]
        L.mamba2_gated_scan_backward.restype = ctypes.c_int
        L.mamba2_gated_scan_backward.argtypes = [pg, vp, *rows4] + [vp] * 12 + [sz, vp]
        L.mamba2_state_cache_store.restype = ctypes.c_int
        L.mamba2_state_cache_store.argtypes = [pc, vp, i64, vp, vp, vp, vp]
        L.mamba2_state_cache_load.restype = ctypes.c_int
        L.mamba2_state_cache_load.argtypes = [pc, vp, vp, vp, vp, i64, vp]
        _lib = L
    return _lib


def device_errors() -> int:
    """Synchronise the current device and return (and clear) the flags raised by
    kernels whose bounded waits ran out (0 = none)."""
    f = ctypes.c_uint(0)
    st = lib().mamba2_device_errors(ctypes.byref(f))
    if st != 0:
        raise Mamba2Error(st, "mamba2_device_errors")
    return int(f.value)


def debug_stall_waits(enable: bool) -> None:
    """Test aid: while enabled, every waiting kernel's first wait runs out (20 ms)
    and the kernel returns without doing its work, raising the flag that
    device_errors() reports (bit 0).  Synchronises the current device."""
    st = lib().mamba2_debug_stall_waits(int(bool(enable)))
    if st != 0:
        raise Mamba2Error(st, "mamba2_debug_stall_waits")


def status_string(status: int) -> str:
    return lib().mamba2_status_string(int(status)).decode()


def make_dims(batch, seqlen, nheads, headdim, dstate, ngroups, *, d_conv=4, chunk_size=256,
              io_dtype="bf16", norm_before_gate=False, norm_eps=1e-5) -> Mamba2Dims:
    io = {"f32": MAMBA2_F32, "bf16": MAMBA2_BF16}.get(io_dtype, io_dtype)
    return Mamba2Dims(int(batch), int(seqlen), int(nheads), int(headdim), int(dstate),
                      int(ngroups), int(d_conv), int(chunk_size), int(io),
                      int(bool(norm_before_gate)), float(norm_eps))


def dims_from_config(cfg, batch=None, seqlen=None) -> Mamba2Dims:
    return make_dims(cfg.batch if batch is None else batch,
                     cfg.seqlen if seqlen is None else seqlen, cfg.nheads, cfg.headdim,
                     cfg.dstate, cfg.ngroups, d_conv=cfg.d_conv, chunk_size=cfg.chunk_size,
                     io_dtype=cfg.io_dtype, norm_before_gate=cfg.norm_before_gate,
                     norm_eps=cfg.norm_eps)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def make_params(conv_w, conv_b, dt_bias, A, D, norm_w) -> Mamba2Params:
    """Pointers of fp32 device tensors; the caller keeps the tensors alive."""
    ts = (conv_w, conv_b, dt_bias, A, D, norm_w)
    for t in ts:
        import torch
        if not (t.is_cuda and t.dtype == torch.float32 and t.is_contiguous()):
            raise ValueError("parameters must be contiguous fp32 CUDA tensors")
    return Mamba2Params(*[t.data_ptr() for t in ts])


def _stream(stream):
    import torch
    if stream is None:
        return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    if hasattr(stream, "cuda_stream"):
        return ctypes.c_void_p(stream.cuda_stream)
    return ctypes.c_void_p(int(stream))


def _rows(t, name, width, batch, rows_per_batch):
    """Row stride (elements) of a [batch, rows, width]-shaped view with unit last stride."""
    if t.stride(-1) != 1:
        raise ValueError(f"{name}: last dimension must be contiguous")
    rs = t.stride(-2) if t.dim() >= 2 else width
    if (t.dim() == 3 and t.shape[0] > 1 and rows_per_batch > 0
            and t.stride(0) != rows_per_batch * rs):
        raise ValueError(f"{name}: batch stride must be rows * row stride")
    return rs


def mamba2_prefill_workspace_size(dims: Mamba2Dims) -> int:
    return int(lib().mamba2_prefill_workspace_size(ctypes.byref(dims)))


def mamba2_conv_ssd_prefill(dims, params, xBC, z, dt_raw, y, conv_state=None, ssm_state=None,
                            states_in=False, workspace=None, stream=None) -> None:
    """Enqueue one prefill on `stream` (default: torch's current stream).

    xBC [b, L, conv_dim], z [b, L, d_inner], dt_raw [b, L, H] (views with unit last
    stride; row strides are passed through); y [b, L, d_inner] contiguous;
    conv_state [b, conv_dim, 4] / ssm_state [b, H, P, N] fp32 or None;
    workspace: a CUDA byte tensor of mamba2_prefill_workspace_size(dims) bytes."""
    L = dims.seqlen
    lx = _rows(xBC, "xBC", None, dims.batch, L)
    lz = _rows(z, "z", None, dims.batch, L)
    ld = _rows(dt_raw, "dt_raw", None, dims.batch, L)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    st = lib().mamba2_conv_ssd_prefill(
        ctypes.byref(dims), ctypes.byref(params), _ptr(xBC), lx, _ptr(z), lz, _ptr(dt_raw), ld,
        _ptr(y), _ptr(conv_state), _ptr(ssm_state), int(bool(states_in)), _ptr(workspace),
        ws_bytes, _stream(stream))
    if st != 0:
        raise Mamba2Error(st, "mamba2_conv_ssd_prefill")


def mamba2_prefill_host_workspace_size(dims: Mamba2Dims) -> int:
    return int(lib().mamba2_prefill_host_workspace_size(ctypes.byref(dims)))


def mamba2_conv_ssd_prefill_host(dims, params, xBC, z, dt_raw, y, conv_state=None,
                                 ssm_state=None, states_in=False, workspace=None,
                                 stream=None) -> None:
    """Enqueue one prefill whose inputs, y and states are CPU tensors (page-locked
    for overlapped copies); layouts as mamba2_conv_ssd_prefill; workspace: a CUDA
    byte tensor of mamba2_prefill_host_workspace_size(dims) bytes.  Synchronise
    the stream before reading y or the states."""
    for name, t in (("xBC", xBC), ("z", z), ("dt_raw", dt_raw), ("y", y),
                    ("conv_state", conv_state), ("ssm_state", ssm_state)):
        if t is not None and t.is_cuda:
            raise ValueError(f"{name}: the host entry takes CPU tensors")
    L = dims.seqlen
    lx = _rows(xBC, "xBC", None, dims.batch, L)
    lz = _rows(z, "z", None, dims.batch, L)
    ld = _rows(dt_raw, "dt_raw", None, dims.batch, L)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    st = lib().mamba2_conv_ssd_prefill_host(
        ctypes.byref(dims), ctypes.byref(params), _ptr(xBC), lx, _ptr(z), lz, _ptr(dt_raw), ld,
        _ptr(y), _ptr(conv_state), _ptr(ssm_state), int(bool(states_in)), _ptr(workspace),
        ws_bytes, _stream(stream))
    if st != 0:
        raise Mamba2Error(st, "mamba2_conv_ssd_prefill_host")


def prefill_host(dims, params, xBC, z, dt_raw, conv_state=None, ssm_state=None,
                 states_in=False, workspace=None, y=None, stream=None, device=None):
    """Allocate y (page-locked) and the device workspace if not given, run a
    host-buffer prefill and wait for it.  Returns y [b, L, d_inner] on the CPU;
    the states, if given, are updated in place."""
    import torch
    dev = torch.device("cuda") if device is None else torch.device(device)
    if y is None:
        y = torch.empty(dims.batch, dims.seqlen, dims.nheads * dims.headdim, dtype=xBC.dtype,
                        pin_memory=True)
    if workspace is None:
        workspace = torch.empty(max(1, mamba2_prefill_host_workspace_size(dims)),
                                dtype=torch.uint8, device=dev)
    mamba2_conv_ssd_prefill_host(dims, params, xBC, z, dt_raw, y, conv_state, ssm_state,
                                 states_in, workspace, stream)
    torch.cuda.synchronize(dev)
    return y


def mamba2_prefill_varlen_workspace_size(dims: Mamba2Dims) -> int:
    return int(lib().mamba2_prefill_varlen_workspace_size(ctypes.byref(dims)))


def mamba2_conv_ssd_prefill_varlen(dims, params, xBC, z, dt_raw, cu_seqlens, y, conv_state=None,
                                   ssm_state=None, states_in=False, workspace=None,
                                   stream=None) -> None:
    """Enqueue one prefill of dims.batch sequences packed along the token axis
    (dims.seqlen = total tokens): xBC [T, conv_dim], z [T, d_inner], dt_raw [T, H]
    (unit last stride, row strides passed through), y [T, d_inner] contiguous;
    cu_seqlens: CUDA int32 [batch + 1] (0, running token counts, T); states per
    sequence; workspace of mamba2_prefill_varlen_workspace_size(dims) bytes."""
    lx = _rows(xBC, "xBC", None, 1, 0)
    lz = _rows(z, "z", None, 1, 0)
    ld = _rows(dt_raw, "dt_raw", None, 1, 0)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    st = lib().mamba2_conv_ssd_prefill_varlen(
        ctypes.byref(dims), ctypes.byref(params), _ptr(xBC), lx, _ptr(z), lz, _ptr(dt_raw), ld,
        _ptr(cu_seqlens), _ptr(y), _ptr(conv_state), _ptr(ssm_state), int(bool(states_in)),
        _ptr(workspace), ws_bytes, _stream(stream))
    if st != 0:
        raise Mamba2Error(st, "mamba2_conv_ssd_prefill_varlen")


def prefill_varlen(dims, params, xBC, z, dt_raw, cu_seqlens, conv_state=None, ssm_state=None,
                   states_in=False, workspace=None, y=None, stream=None):
    """Allocate y (and the workspace if not given) and run a packed-sequence prefill.
    Returns y [T, d_inner]; the states, if given, are updated in place."""
    import torch
    if y is None:
        y = torch.empty(dims.seqlen, dims.nheads * dims.headdim, dtype=xBC.dtype,
                        device=xBC.device)
    if workspace is None:
        workspace = torch.empty(max(1, mamba2_prefill_varlen_workspace_size(dims)),
                                dtype=torch.uint8, device=xBC.device)
    mamba2_conv_ssd_prefill_varlen(dims, params, xBC, z, dt_raw, cu_seqlens, y, conv_state,
                                   ssm_state, states_in, workspace, stream)
    return y


def mamba2_conv_ssd_prefill_noalloc(dims, params, xBC, z, dt_raw, y, conv_state=None,
                                    ssm_state=None, states_in=False, stream=None) -> None:
    """Prefill without a workspace, for callers that may not allocate device memory:
    the library's fixed device scratch array (MAMBA2_STATIC_SCRATCH_BYTES, 64 MiB)
    is used instead.  Larger problems raise Mamba2Error (workspace status).  Calls
    that overlap on the GPU share that array and race; serialise them."""
    L = dims.seqlen
    lx = _rows(xBC, "xBC", None, dims.batch, L)
    lz = _rows(z, "z", None, dims.batch, L)
    ld = _rows(dt_raw, "dt_raw", None, dims.batch, L)
    st = lib().mamba2_conv_ssd_prefill_noalloc(
        ctypes.byref(dims), ctypes.byref(params), _ptr(xBC), lx, _ptr(z), lz, _ptr(dt_raw), ld,
        _ptr(y), _ptr(conv_state), _ptr(ssm_state), int(bool(states_in)), _stream(stream))
    if st != 0:
        raise Mamba2Error(st, "mamba2_conv_ssd_prefill_noalloc")


def mamba2_ssd_step(dims, params, xBC, z, dt_raw, y, conv_state, ssm_state, stream=None) -> None:
    """Enqueue one decode step.  xBC [b, conv_dim], z [b, d_inner], dt_raw [b, H]
    (unit last stride); y [b, d_inner]; states updated in place."""
    st = lib().mamba2_ssd_step(
        ctypes.byref(dims), ctypes.byref(params), _ptr(xBC), xBC.stride(0), _ptr(z), z.stride(0),
        _ptr(dt_raw), dt_raw.stride(0), _ptr(y), _ptr(conv_state), _ptr(ssm_state),
        _stream(stream))
    if st != 0:
        raise Mamba2Error(st, "mamba2_ssd_step")


def prefill(dims, params, xBC, z, dt_raw, conv_state=None, ssm_state=None, states_in=False,
            workspace=None, y=None, stream=None):
    """Allocate y (and the workspace if not given) on xBC's device and run a prefill.
    Returns y; the states, if given, are updated in place."""
    import torch
    if y is None:
        y = torch.empty(dims.batch, dims.seqlen, dims.nheads * dims.headdim, dtype=xBC.dtype,
                        device=xBC.device)
    if workspace is None:
        workspace = torch.empty(max(1, mamba2_prefill_workspace_size(dims)), dtype=torch.uint8,
                                device=xBC.device)
    mamba2_conv_ssd_prefill(dims, params, xBC, z, dt_raw, y, conv_state, ssm_state, states_in,
                            workspace, stream)
    return y


def step(dims, params, xBC, z, dt_raw, conv_state, ssm_state, y=None, stream=None):
    """Allocate y and run one decode step; returns y."""
    import torch
    if y is None:
        y = torch.empty(dims.batch, dims.nheads * dims.headdim, dtype=xBC.dtype,
                        device=xBC.device)
    mamba2_ssd_step(dims, params, xBC, z, dt_raw, y, conv_state, ssm_state, stream)
    return y


def mamba2_prefill_backward_workspace_size(dims: Mamba2Dims) -> int:
    return int(lib().mamba2_prefill_backward_workspace_size(ctypes.byref(dims)))


def mamba2_conv_ssd_prefill_backward(dims, params, xBC, z, dt_raw, dy, grads, conv_state_in=None,
                                     ssm_state_in=None, d_ssm_state_out=None, workspace=None,
                                     stream=None) -> None:
    """Enqueue the prefill's backward pass on `stream`.

    xBC, z, dt_raw as for the prefill; dy [b, L, d_inner] contiguous; grads: a dict of
    output tensors "xBC", "z", "dt_raw" (io dtype, contiguous), "conv_w", "conv_b",
    "dt_bias", "A", "D", "norm_w" (fp32) and optionally "conv_state", "ssm_state" (the
    initial states' gradients); workspace: a CUDA byte tensor of
    mamba2_prefill_backward_workspace_size(dims) bytes."""
    L = dims.seqlen
    lx = _rows(xBC, "xBC", None, dims.batch, L)
    lz = _rows(z, "z", None, dims.batch, L)
    ld = _rows(dt_raw, "dt_raw", None, dims.batch, L)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    g = lambda k: _ptr(grads.get(k))
    st = lib().mamba2_conv_ssd_prefill_backward(
        ctypes.byref(dims), ctypes.byref(params), _ptr(xBC), lx, _ptr(z), lz, _ptr(dt_raw), ld,
        _ptr(conv_state_in), _ptr(ssm_state_in), _ptr(dy), _ptr(d_ssm_state_out), g("xBC"),
        g("z"), g("dt_raw"), g("conv_w"), g("conv_b"), g("dt_bias"), g("A"), g("D"), g("norm_w"),
        g("conv_state"), g("ssm_state"), _ptr(workspace), ws_bytes, _stream(stream))
    if st != 0:
        raise Mamba2Error(st, "mamba2_conv_ssd_prefill_backward")


def prefill_backward(dims, params, xBC, z, dt_raw, dy, conv_state_in=None, ssm_state_in=None,
                     d_ssm_state_out=None, workspace=None, stream=None):
    """Allocate the gradients (and the workspace if not given) and run the backward pass.
    Returns the dict of gradients (initial-state gradients when those states are given)."""
    import torch
    dev, dt = xBC.device, xBC.dtype
    b, L, H, P, N, G = (dims.batch, dims.seqlen, dims.nheads, dims.headdim, dims.dstate,
                        dims.ngroups)
    d_inner, conv_dim = H * P, H * P + 2 * G * N
    f32 = dict(dtype=torch.float32, device=dev)
    grads = {"xBC": torch.empty(b, L, conv_dim, dtype=dt, device=dev),
             "z": torch.empty(b, L, d_inner, dtype=dt, device=dev),
             "dt_raw": torch.empty(b, L, H, dtype=dt, device=dev),
             "conv_w": torch.empty(conv_dim, dims.d_conv, **f32),
             "conv_b": torch.empty(conv_dim, **f32), "dt_bias": torch.empty(H, **f32),
             "A": torch.empty(H, **f32), "D": torch.empty(H, **f32),
             "norm_w": torch.empty(d_inner, **f32)}
    if conv_state_in is not None:
        grads["conv_state"] = torch.empty_like(conv_state_in)
    if ssm_state_in is not None:
        grads["ssm_state"] = torch.empty_like(ssm_state_in)
    if workspace is None:
        workspace = torch.empty(max(1, mamba2_prefill_backward_workspace_size(dims)),
                                dtype=torch.uint8, device=dev)
    mamba2_conv_ssd_prefill_backward(dims, params, xBC, z, dt_raw, dy, grads, conv_state_in,
                                     ssm_state_in, d_ssm_state_out, workspace, stream)
    return grads


# ---------------------------------------------------------------- gated scan

#: Tokens of a checkpoint of the gated scan.
GATED_SCAN_CHUNK = 16


def make_gated_scan_dims(batch, seqlen, width, *, io_dtype="bf16",
                         decay_scale=8.0) -> Mamba2GatedScanDims:
    """Sizes of the gated scan.  Packed rows: batch = sequences, seqlen = all tokens."""
    io = {"f32": MAMBA2_F32, "bf16": MAMBA2_BF16}.get(io_dtype, io_dtype)
    return Mamba2GatedScanDims(int(batch), int(seqlen), int(width), int(io), float(decay_scale))


def mamba2_gated_scan_workspace_size(dims: Mamba2GatedScanDims, packed: bool = False) -> int:
    return int(lib().mamba2_gated_scan_workspace_size(ctypes.byref(dims), int(bool(packed))))


def mamba2_gated_scan_backward_workspace_size(dims: Mamba2GatedScanDims,
                                              packed: bool = False) -> int:
    return int(lib().mamba2_gated_scan_backward_workspace_size(ctypes.byref(dims),
                                                               int(bool(packed))))


def gated_scan_checkpoints(dims: Mamba2GatedScanDims, packed: bool = False, device="cuda"):
    """An fp32 tensor for the checkpoints of one prefill: [rows, ceil(L / 16), D]."""
    import torch
    rows = (1 if dims.seqlen > 0 else 0) if packed else dims.batch
    return torch.empty(rows, -(-dims.seqlen // GATED_SCAN_CHUNK), dims.width,
                       dtype=torch.float32, device=device)


def _need(t, name, shape, dtype, device, contiguous=True):
    if t.shape != shape or t.dtype != dtype or t.device != device:
        raise ValueError(f"{name}: {tuple(shape)} {dtype} on {device} expected, got "
                         f"{tuple(t.shape)} {t.dtype} on {t.device}")
    if contiguous and not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")


def _row_stride(t, name):
    """Elements from one token to the next of [..., tokens, D] rows that follow one another."""
    st, shape = t.stride(), t.shape
    if st[-1] != 1:
        raise ValueError(f"{name}: last dimension must be contiguous")
    if len(shape) == 2:
        return st[0] if shape[0] > 1 else max(st[0], shape[1])
    b, n = shape[0], shape[1]
    rs = st[1] if n > 1 else (st[0] if b > 1 else max(st[1], shape[2]))
    if b > 1 and n > 1 and st[0] != n * rs:
        raise ValueError(f"{name}: batch stride must be rows * row stride")
    return rs


def _gs_inputs(dims, shape, lam, x, r, g, z):
    """The shared inputs checked: their device, dtype and (pointer, row stride) arguments."""
    import torch
    f32, width = torch.float32, dims.width
    dt = torch.bfloat16 if dims.io_dtype == MAMBA2_BF16 else f32
    dev = x.device
    # (one expression for what is nearly always so; what is not is then told apart)
    if not (x.is_cuda and x.dtype is dt and r.dtype is dt and g.dtype is dt and lam.dtype is f32
            and x.shape == shape and r.shape == shape and g.shape == shape
            and r.device == dev and g.device == dev and lam.device == dev
            and lam.shape == (width,) and lam.is_contiguous()
            and dims.io_dtype in (MAMBA2_F32, MAMBA2_BF16)):
        if dims.io_dtype not in (MAMBA2_F32, MAMBA2_BF16):
            raise ValueError("io_dtype: f32 or bf16")
        if not x.is_cuda:
            raise ValueError(f"x: a CUDA tensor expected, got {dev}")
        _need(lam, "lam", (width,), f32, dev)
        for name, t in (("x", x), ("r", r), ("g", g)):
            _need(t, name, shape, dt, dev, False)
    if z is not None:
        _need(z, "z", shape, dt, dev, False)
    if len(shape) == 2 and shape[0] > 1:  # rows of tokens one after the other
        sx, sr, sg = x.stride(), r.stride(), g.stride()
        if sx[1] == 1 and sr[1] == 1 and sg[1] == 1 and z is None:
            return dev, dt, (x.data_ptr(), sx[0], r.data_ptr(), sr[0], g.data_ptr(), sg[0], None, 0)
    rows = (x.data_ptr(), _row_stride(x, "x"), r.data_ptr(), _row_stride(r, "r"),
            g.data_ptr(), _row_stride(g, "g"))
    return dev, dt, rows + ((None, 0) if z is None else (z.data_ptr(), _row_stride(z, "z")))


class _On:
    """A call's surroundings: the tensors' device current and, where the caller names a stream,
    that stream too, so that what the call allocates belongs to the stream it is used on."""

    __slots__ = ("other", "stream")

    def __init__(self, dev, stream):
        import torch
        self.other = None
        if stream is None:
            if torch.cuda.current_device() != dev.index:
                self.other = torch.cuda.device(dev)
            # (the raw handle: a Stream object takes longer to make than a small kernel)
            self.stream = torch._C._cuda_getCurrentRawStream(dev.index)
            return
        if not hasattr(stream, "cuda_stream"):
            stream = (torch.cuda.ExternalStream(int(stream), dev) if int(stream)
                      else torch.cuda.default_stream(dev))
        if stream.device != dev:
            raise ValueError(f"stream: one of {dev} expected, got one of {stream.device}")
        self.other = torch.cuda.stream(stream)
        self.stream = stream.cuda_stream

    def __enter__(self):
        if self.other is not None:
            self.other.__enter__()
        return self.stream

    def __exit__(self, *exc):
        if self.other is not None:
            self.other.__exit__(*exc)


def _addr(t):
    return None if t is None else t.data_ptr()


def _scratch(workspace, size, dev):
    """The caller's workspace, or a new one: (tensor, address, bytes)."""
    import torch
    if workspace is None:
        workspace = torch.empty(max(size, 1), dtype=torch.uint8, device=dev)
    elif workspace.device != dev or not workspace.is_contiguous():
        raise ValueError(f"workspace: a contiguous tensor on {dev} expected")
    return workspace, workspace.data_ptr(), workspace.numel() * workspace.element_size()


def _gs_optional(dims, packed, cu_seqlens, states, checkpoints, dev):
    import torch
    if packed:
        _need(cu_seqlens, "cu_seqlens", (dims.batch + 1,), torch.int32, dev)
    for name, t in states:
        if t is not None:
            _need(t, name, (dims.batch, dims.width), torch.float32, dev)
    if checkpoints is not None:
        rows = (1 if dims.seqlen > 0 else 0) if packed else dims.batch
        _need(checkpoints, "checkpoints", (rows, -(-dims.seqlen // GATED_SCAN_CHUNK), dims.width),
              torch.float32, dev)


def gated_scan_prefill(dims, lam, x, r, g, z=None, h_state=None, states_in=False, cu_seqlens=None,
                       checkpoints=None, workspace=None, y=None, stream=None):
    """The gated linear recurrence over dims.seqlen tokens (mamba2_gated_scan_prefill).

    x, r, g and z (optional output gate) [b, L, D], or [T, D] with cu_seqlens (CUDA int32
    [b + 1]); views with unit last stride, e.g. columns of one projection.  lam [D] fp32.
    h_state [b, D] fp32 (optional) holds the initial states when states_in is true and
    receives the final ones.  checkpoints: see gated_scan_checkpoints, for the backward
    pass.  Allocates y (and the workspace) if not given; returns y."""
    import torch
    packed = cu_seqlens is not None
    shape = (dims.seqlen, dims.width) if packed else (dims.batch, dims.seqlen, dims.width)
    dev, dt, rows = _gs_inputs(dims, shape, lam, x, r, g, z)
    _gs_optional(dims, packed, cu_seqlens, (("h_state", h_state),), checkpoints, dev)
    if y is not None:
        _need(y, "y", shape, dt, dev)
    with _On(dev, stream) as s:
        if y is None:
            y = torch.empty(*shape, dtype=dt, device=dev)
        ws, ws_at, ws_bytes = _scratch(workspace, mamba2_gated_scan_workspace_size(dims, packed),
                                       dev)
        st = lib().mamba2_gated_scan_prefill(
            ctypes.byref(dims), lam.data_ptr(), *rows, _addr(cu_seqlens), y.data_ptr(),
            _addr(h_state), int(bool(states_in)), _addr(checkpoints), ws_at, ws_bytes, s)
    if st != 0:
        raise Mamba2Error(st, "mamba2_gated_scan_prefill")
    return y


def gated_scan_step(dims, lam, x, r, g, h_state, z=None, y=None, stream=None):
    """One token of every sequence: x, r, g, z [b, D]; h_state [b, D] fp32 is updated in
    place.  Allocates y [b, D] if not given and returns it."""
    import torch
    shape = (dims.batch, dims.width)
    dev, dt, rows = _gs_inputs(dims, shape, lam, x, r, g, z)
    _need(h_state, "h_state", shape, torch.float32, dev)
    if y is not None:
        _need(y, "y", shape, dt, dev)
    if stream is None and torch.cuda.current_device() == dev.index:
        if y is None:
            y = torch.empty(*shape, dtype=dt, device=dev)
        st = lib().mamba2_gated_scan_step(ctypes.byref(dims), lam.data_ptr(), *rows, y.data_ptr(),
                                          h_state.data_ptr(),
                                          torch._C._cuda_getCurrentRawStream(dev.index))
    else:
        with _On(dev, stream) as s:
            if y is None:
                y = torch.empty(*shape, dtype=dt, device=dev)
            st = lib().mamba2_gated_scan_step(ctypes.byref(dims), lam.data_ptr(), *rows,
                                              y.data_ptr(), h_state.data_ptr(), s)
    if st != 0:
        raise Mamba2Error(st, "mamba2_gated_scan_step")
    return y


def gated_scan_backward(dims, lam, x, r, g, dy, z=None, h_state_in=None, d_h_state_out=None,
                        cu_seqlens=None, checkpoints=None, workspace=None, stream=None):
    """Gradients of sum(y dy) + sum(final state d_h_state_out) of gated_scan_prefill.

    Inputs as for the prefill; dy contiguous like y; h_state_in the state it began with (None:
    zero); checkpoints: those it wrote (None: the scan is run again).  Returns a dict "x",
    "r", "g", "lam", with z "z", and with h_state_in "h_state"."""
    import torch
    packed = cu_seqlens is not None
    shape = (dims.seqlen, dims.width) if packed else (dims.batch, dims.seqlen, dims.width)
    dev, dt, rows = _gs_inputs(dims, shape, lam, x, r, g, z)
    _need(dy, "dy", shape, dt, dev)
    _gs_optional(dims, packed, cu_seqlens,
                 (("h_state_in", h_state_in), ("d_h_state_out", d_h_state_out)), checkpoints, dev)
    with _On(dev, stream) as s:
        grads = {k: torch.empty(*shape, dtype=dt, device=dev)
                 for k in (("x", "r", "g") if z is None else ("x", "r", "g", "z"))}
        grads["lam"] = torch.empty(dims.width, dtype=torch.float32, device=dev)
        if h_state_in is not None:
            grads["h_state"] = torch.empty(dims.batch, dims.width, dtype=torch.float32, device=dev)
        ws, ws_at, ws_bytes = _scratch(
            workspace, mamba2_gated_scan_backward_workspace_size(dims, packed), dev)
        st = lib().mamba2_gated_scan_backward(
            ctypes.byref(dims), lam.data_ptr(), *rows, _addr(cu_seqlens), _addr(h_state_in),
            dy.data_ptr(), _addr(d_h_state_out), _addr(checkpoints), grads["x"].data_ptr(),
            grads["r"].data_ptr(), grads["g"].data_ptr(), _addr(grads.get("z")),
            grads["lam"].data_ptr(), _addr(grads.get("h_state")), ws_at, ws_bytes, s)
    if st != 0:
        raise Mamba2Error(st, "mamba2_gated_scan_backward")
    return grads


# ---------------------------------------------------------------- state cache

_CODES = ("int8", "e4m3")  # mamba2_code_format


def state_cache(nslots, row, block=64, codes="int8", device="cuda"):
    """An empty cache for `nslots` states of `row` values: (codes [nslots, row] int8 or
    float8_e4m3fn, scales [nslots, ceil(row / block)] uint8), all zero."""
    import torch
    if codes not in _CODES:
        raise ValueError("codes: int8 or e4m3")
    dt = torch.int8 if codes == "int8" else torch.float8_e4m3fn
    return (torch.zeros(nslots, row, dtype=dt, device=device),
            torch.zeros(nslots, -(-row // block), dtype=torch.uint8, device=device))


def _state_cache_args(state, slots, codes, scales, block):
    import torch
    dev, sdt, cdt = state.device, state.dtype, codes.dtype
    if not state.is_cuda:
        raise ValueError(f"state: a CUDA tensor expected, got {dev}")
    if state.dim() < 2 or (sdt is not torch.float32 and sdt is not torch.bfloat16):
        raise ValueError("state: [b, ...] of fp32 or bf16 expected")
    if codes.dim() != 2 or (cdt is not torch.int8 and cdt is not torch.float8_e4m3fn):
        raise ValueError("codes: [slots, row] of int8 or float8_e4m3fn expected")
    b, (nslots, row) = state.shape[0], codes.shape
    if state.numel() != b * row:
        raise ValueError(f"state: {row} values a row expected, got {tuple(state.shape)}")
    if not state.is_contiguous() and b and not state[0].is_contiguous():
        raise ValueError("state: each row's values must be contiguous")
    if block not in (32, 64, 128):
        raise ValueError("block: 32, 64 or 128")
    if not (slots.shape == (b,) and slots.dtype is torch.int32 and slots.device == dev
            and slots.is_contiguous() and codes.device == dev and codes.is_contiguous()
            and scales.dtype is torch.uint8 and scales.device == dev and scales.is_contiguous()
            and scales.shape == (nslots, -(-row // block))):
        _need(slots, "slots", (b,), torch.int32, dev)
        _need(codes, "codes", codes.shape, cdt, dev)
        _need(scales, "scales", (nslots, -(-row // block)), torch.uint8, dev)
    dims = Mamba2StateCacheDims(b, row, nslots, block, 0 if cdt is torch.int8 else 1,
                                MAMBA2_F32 if sdt is torch.float32 else MAMBA2_BF16)
    return dev, dims, state.stride(0) if b > 1 else row


def state_cache_store(state, slots, codes, scales, block=64, stream=None) -> None:
    """Write working states [b, ...] (fp32 or bf16) into slots (CUDA int32 [b]; negative:
    skipped; the last row of those that name one slot counts) of a cache (see state_cache)."""
    dev, dims, ld = _state_cache_args(state, slots, codes, scales, block)
    with _On(dev, stream) as s:
        st = lib().mamba2_state_cache_store(ctypes.byref(dims), state.data_ptr(), ld,
                                            slots.data_ptr(), codes.data_ptr(), scales.data_ptr(),
                                            s)
    if st != 0:
        raise Mamba2Error(st, "mamba2_state_cache_store")


def state_cache_load(codes, scales, slots, state, block=64, stream=None) -> None:
    """Read slots of a cache into working states [b, ...]; rows with a negative slot are left
    as they were."""
    dev, dims, ld = _state_cache_args(state, slots, codes, scales, block)
    with _On(dev, stream) as s:
        st = lib().mamba2_state_cache_load(ctypes.byref(dims), codes.data_ptr(),
                                           scales.data_ptr(), slots.data_ptr(), state.data_ptr(),
                                           ld, s)
    if st != 0:
        raise Mamba2Error(st, "mamba2_state_cache_load")
