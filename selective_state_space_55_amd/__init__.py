"""MI355X-native selective scan (Mamba): Python binding over libmamba_scan.so.

This module only marshals arguments: it checks torch tensors (device, dtype,
contiguity, shape), allocates outputs and the workspace with torch, and calls
the C ABI declared in include/mamba_scan.h.  Every step of the computation
runs in the library's HIP kernels.  If the library is not built, importing
works but every call raises; there is no fallback.

Streams: each call runs on its `stream` argument (a torch stream or a raw HIP
stream handle), or on the current stream when it is None.  Outputs and the
workspace a call allocates are allocated while that stream is current, so
torch's caching allocator hands their memory to no other stream's work before
the kernels are done with it.  Tensors the caller passes in (inputs, `out=`,
`workspace=`) are the caller's to keep alive and ordered with that stream.
"""
from __future__ import annotations

import ctypes
import functools
import inspect
import os
from typing import Optional, Tuple

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
# MAMBA_SCAN_LIBRARY names another build of the same library (a sanitizer or
# debug build); by default the in-tree build is loaded
LIB_PATH = os.environ.get("MAMBA_SCAN_LIBRARY") or os.path.join(_HERE, "lib", "libmamba_scan.so")

F32, BF16 = 0, 1
STATUS = {
    0: "MAMBA_SCAN_OK", 1: "MAMBA_SCAN_ERR_NULL", 2: "MAMBA_SCAN_ERR_SHAPE", 3: "MAMBA_SCAN_ERR_DTYPE",
    4: "MAMBA_SCAN_ERR_ALIGN", 5: "MAMBA_SCAN_ERR_UNSUPPORTED", 6: "MAMBA_SCAN_ERR_WORKSPACE",
    7: "MAMBA_SCAN_ERR_HIP",
}
EXPORTED = (
    "mamba_scan_fwd", "mamba_scan_fwd_ex", "mamba_scan_fwd_noalloc", "mamba_scan_fwd_workspace_size",
    "mamba_scan_fwd_workspace_size_ex",
    "mamba_scan_fwd_conv",
    "mamba_scan_fwd_varlen", "mamba_scan_fwd_varlen_workspace_size", "mamba_scan_step", "mamba_scan_bwd",
    "mamba_scan_bwd_workspace_size", "mamba_conv1d_fwd", "mamba_ssd_fwd", "mamba_scan_status_str",
    "mamba_scan_abi_version", "mamba_ssd_conv_fwd_varlen", "mamba_ssd_fwd_varlen",
    "mamba_ssd_fwd_varlen_workspace_size", "mamba_ssd_step",
)
EXPORTED_NORM = ("mamba_rms_norm_fwd", "mamba_rms_norm_bwd", "mamba_rms_norm_bwd_workspace_size")

_lib = None


class MambaScanError(RuntimeError):
    def __init__(self, fn: str, code: int, msg: str):
        super().__init__(f"{fn} failed: {STATUS.get(code, code)} ({msg})")
        self.code = code


def load_library():
    """Loads libmamba_scan.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is not built; run `python -m selective_state_space_55_amd.build`")
    lib = ctypes.CDLL(LIB_PATH)
    P, I64, I, SZ = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t
    lib.mamba_scan_fwd.restype = I
    lib.mamba_scan_fwd.argtypes = [P] * 11 + [I64] * 4 + [I, I, P, SZ, P]
    lib.mamba_scan_fwd_noalloc.restype = I
    lib.mamba_scan_fwd_noalloc.argtypes = [P] * 11 + [I64] * 4 + [I, I, P]
    lib.mamba_scan_fwd_ex.restype = I
    lib.mamba_scan_fwd_ex.argtypes = [P] * 11 + [I64] * 4 + [I, I, I64, I, P, SZ, P]
    lib.mamba_scan_fwd_workspace_size.restype = SZ
    lib.mamba_scan_fwd_workspace_size.argtypes = [I64] * 4 + [I]
    lib.mamba_scan_fwd_conv.restype = I
    lib.mamba_scan_fwd_conv.argtypes = [P] * 16 + [I64] * 4 + [I, I, P, SZ, P]
    lib.mamba_scan_fwd_workspace_size_ex.restype = SZ
    lib.mamba_scan_fwd_workspace_size_ex.argtypes = [I64] * 4 + [I, I64, I]
    lib.mamba_scan_step.restype = I
    lib.mamba_scan_step.argtypes = [P] * 9 + [I, P] + [I64] * 3 + [I, P]
    lib.mamba_scan_bwd.restype = I
    lib.mamba_scan_bwd.argtypes = [P] * 20 + [I64] * 4 + [I, I, P, SZ, P]
    lib.mamba_scan_bwd_workspace_size.restype = SZ
    lib.mamba_scan_bwd_workspace_size.argtypes = [I64] * 4 + [I]
    lib.mamba_scan_fwd_varlen.restype = I
    lib.mamba_scan_fwd_varlen.argtypes = [P] * 12 + [I64] * 4 + [I, I, P, SZ, P]
    lib.mamba_scan_fwd_varlen_workspace_size.restype = SZ
    lib.mamba_scan_fwd_varlen_workspace_size.argtypes = [I64] * 4 + [I]
    lib.mamba_ssd_fwd.restype = I
    lib.mamba_ssd_fwd.argtypes = [P] * 11 + [I64] * 5 + [I, I, P]
    lib.mamba_conv1d_fwd.restype = I
    lib.mamba_conv1d_fwd.argtypes = [P] * 6 + [I64] * 4 + [I, I, P]
    lib.mamba_ssd_conv_fwd_varlen.restype = I
    lib.mamba_ssd_conv_fwd_varlen.argtypes = [P] * 8 + [I64] * 6 + [I, I, P]
    lib.mamba_ssd_fwd_varlen.restype = I
    lib.mamba_ssd_fwd_varlen.argtypes = [P] * 13 + [I64] * 13 + [I, I, P, SZ, P]
    lib.mamba_ssd_fwd_varlen_workspace_size.restype = SZ
    lib.mamba_ssd_fwd_varlen_workspace_size.argtypes = [I64] * 7
    lib.mamba_ssd_step.restype = I
    lib.mamba_ssd_step.argtypes = [P] * 13 + [I64] * 10 + [I, I, P]
    lib.mamba_rms_norm_fwd.restype = I
    lib.mamba_rms_norm_fwd.argtypes = [P] * 3 + [ctypes.c_float] + [P] * 4 + [I64] * 2 + [I, I, I, P]
    lib.mamba_rms_norm_bwd.restype = I
    lib.mamba_rms_norm_bwd.argtypes = [P] * 8 + [I64] * 2 + [I, I, P, SZ, P]
    lib.mamba_rms_norm_bwd_workspace_size.restype = SZ
    lib.mamba_rms_norm_bwd_workspace_size.argtypes = [I64] * 2
    lib.mamba_scan_status_str.restype = ctypes.c_char_p
    lib.mamba_scan_status_str.argtypes = [I]
    lib.mamba_scan_abi_version.restype = I
    lib.mamba_scan_abi_version.argtypes = []
    _lib = lib
    return lib


def abi_version() -> int:
    return int(load_library().mamba_scan_abi_version())


def status_str(code: int) -> str:
    return load_library().mamba_scan_status_str(int(code)).decode()


def _check(fn: str, code: int) -> None:
    if code != 0:
        raise MambaScanError(fn, code, status_str(code))


def _io_dtype(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return F32
    if t.dtype == torch.bfloat16:
        return BF16
    raise ValueError(f"io tensors must be float32 or bfloat16, got {t.dtype}")


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _req(name: str, t: Optional[torch.Tensor], shape, dtype, device) -> Optional[torch.Tensor]:
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if t.dtype != dtype:
        raise ValueError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


FLAG_SOFTPLUS, FLAG_EULER = 1, 2


def _flags(softplus: bool, discretization: str) -> int:
    if discretization not in ("zoh", "euler"):
        raise ValueError(f"discretization must be 'zoh' or 'euler', got {discretization!r}")
    return (FLAG_SOFTPLUS if softplus else 0) | (FLAG_EULER if discretization == "euler" else 0)


def _stream(device: torch.device, stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream(device)
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _on_stream(fn):
    """Runs fn with its `stream` argument made the current stream, so that the outputs and workspace fn
    allocates belong to the stream its kernels are enqueued on (a raw handle is wrapped as an
    ExternalStream of the first argument's device)."""

    @functools.wraps(fn)
    def run(*args, stream=None, **kwargs):
        if stream is None:
            return fn(*args, stream=None, **kwargs)
        t0 = args[0] if args else None
        dev = t0.device if isinstance(t0, torch.Tensor) else torch.device("cuda", torch.cuda.current_device())
        if not isinstance(stream, torch.cuda.Stream):
            stream = torch.cuda.ExternalStream(int(stream), device=dev)
        with torch.cuda.stream(stream):
            return fn(*args, stream=stream, **kwargs)

    return run


def fwd_workspace_size(batch: int, dim: int, dstate: int, seqlen: int, io_dtype: int = BF16, nchunks: int = 0,
                       states_per_wave: int = 0) -> int:
    n = load_library().mamba_scan_fwd_workspace_size_ex(batch, dim, dstate, seqlen, io_dtype, nchunks,
                                                        states_per_wave)
    if n == ctypes.c_size_t(-1).value:
        raise ValueError("mamba_scan_fwd_workspace_size: sizes rejected")
    return int(n)


@_on_stream
def scan_fwd(u: torch.Tensor, delta: torch.Tensor, A_log: torch.Tensor, B: torch.Tensor, C: torch.Tensor,
             D: Optional[torch.Tensor] = None, z: Optional[torch.Tensor] = None,
             delta_bias: Optional[torch.Tensor] = None, initial_state: Optional[torch.Tensor] = None,
             delta_softplus: bool = True, return_final_state: bool = False, *,
             out: Optional[torch.Tensor] = None, final_state: Optional[torch.Tensor] = None,
             workspace: Optional[torch.Tensor] = None, nchunks: int = 0, states_per_wave: int = 0,
             discretization: str = "zoh", stream=None):
    """Selective-scan forward (discretization "zoh", or "euler" for Bbar u = Delta B u).  u, delta, z: (batch, dim, L); B, C: (batch, dstate, L) in the io dtype
    (float32 or bfloat16); A_log (dim, dstate), D, delta_bias (dim,), initial_state (batch, dim, dstate)
    in float32.  Returns y (batch, dim, L), or (y, final_state) if return_final_state."""
    lib = load_library()
    if u.dim() != 3:
        raise ValueError("u must be (batch, dim, L)")
    batch, dim, L = u.shape
    dev = u.device
    if dev.type != "cuda":
        raise ValueError("scan_fwd needs device tensors (HIP)")
    io = _io_dtype(u)
    iot = u.dtype
    dstate = A_log.shape[-1] if A_log.dim() == 2 else -1
    _req("u", u, (batch, dim, L), iot, dev)
    _req("delta", delta, (batch, dim, L), iot, dev)
    _req("A_log", A_log, (dim, dstate), torch.float32, dev)
    _req("B", B, (batch, dstate, L), iot, dev)
    _req("C", C, (batch, dstate, L), iot, dev)
    _req("D", D, (dim,), torch.float32, dev)
    _req("z", z, (batch, dim, L), iot, dev)
    _req("delta_bias", delta_bias, (dim,), torch.float32, dev)
    _req("initial_state", initial_state, (batch, dim, dstate), torch.float32, dev)
    y = out if out is not None else torch.empty((batch, dim, L), dtype=iot, device=dev)
    _req("out", y, (batch, dim, L), iot, dev)
    fs = final_state
    if fs is None and return_final_state:
        fs = torch.empty((batch, dim, dstate), dtype=torch.float32, device=dev)
    _req("final_state", fs, (batch, dim, dstate), torch.float32, dev)
    need = fwd_workspace_size(batch, dim, dstate, L, io, nchunks, states_per_wave)
    ws = workspace
    if ws is None and need > 0:
        ws = torch.empty(need + 256, dtype=torch.uint8, device=dev)
    ws_ptr, ws_bytes = None, 0
    if ws is not None:
        base = ws.data_ptr()
        off = (-base) % 256
        ws_ptr, ws_bytes = ctypes.c_void_p(base + off), max(0, ws.numel() * ws.element_size() - off)
    rc = lib.mamba_scan_fwd_ex(_ptr(u), _ptr(delta), _ptr(A_log), _ptr(B), _ptr(C), _ptr(D), _ptr(z),
                               _ptr(delta_bias), _ptr(initial_state), _ptr(fs), _ptr(y), batch, dim, dstate, L, io,
                               _flags(delta_softplus, discretization), int(nchunks), int(states_per_wave), ws_ptr,
                               ws_bytes,
                               _stream(dev, stream))
    _check("mamba_scan_fwd", rc)
    return (y, fs) if return_final_state else y


NOALLOC_SCRATCH_BYTES = 64 << 20   # MAMBA_SCAN_NOALLOC_SCRATCH_BYTES


@_on_stream
def scan_fwd_noalloc(u: torch.Tensor, delta: torch.Tensor, A_log: torch.Tensor, B: torch.Tensor, C: torch.Tensor,
                     out: torch.Tensor, D: Optional[torch.Tensor] = None, z: Optional[torch.Tensor] = None,
                     delta_bias: Optional[torch.Tensor] = None, initial_state: Optional[torch.Tensor] = None,
                     final_state: Optional[torch.Tensor] = None, delta_softplus: bool = True,
                     discretization: str = "zoh", stream=None) -> torch.Tensor:
    """scan_fwd through mamba_scan_fwd_noalloc: the caller passes every output (out: y, and optionally
    final_state) and nothing is allocated, by this function or the library (the chunk carry lives in
    the library's static per-GPU scratch).  Calls that overlap in time on one GPU race on that scratch.
    Returns out."""
    lib = load_library()
    if u.dim() != 3:
        raise ValueError("u must be (batch, dim, L)")
    batch, dim, L = u.shape
    dev = u.device
    if dev.type != "cuda":
        raise ValueError("scan_fwd_noalloc needs device tensors (HIP)")
    io = _io_dtype(u)
    iot = u.dtype
    dstate = A_log.shape[-1] if A_log.dim() == 2 else -1
    for name, t, shape, dt in (("u", u, (batch, dim, L), iot), ("delta", delta, (batch, dim, L), iot),
                               ("A_log", A_log, (dim, dstate), torch.float32), ("B", B, (batch, dstate, L), iot),
                               ("C", C, (batch, dstate, L), iot), ("D", D, (dim,), torch.float32),
                               ("z", z, (batch, dim, L), iot), ("delta_bias", delta_bias, (dim,), torch.float32),
                               ("initial_state", initial_state, (batch, dim, dstate), torch.float32),
                               ("out", out, (batch, dim, L), iot),
                               ("final_state", final_state, (batch, dim, dstate), torch.float32)):
        _req(name, t, shape, dt, dev)
    if out is None:
        raise ValueError("scan_fwd_noalloc needs out (y)")
    rc = lib.mamba_scan_fwd_noalloc(_ptr(u), _ptr(delta), _ptr(A_log), _ptr(B), _ptr(C), _ptr(D), _ptr(z),
                                    _ptr(delta_bias), _ptr(initial_state), _ptr(final_state), _ptr(out), batch, dim,
                                    dstate, L, io, _flags(delta_softplus, discretization), _stream(dev, stream))
    _check("mamba_scan_fwd_noalloc", rc)
    return out


@_on_stream
def scan_fwd_conv(x: torch.Tensor, conv_weight: torch.Tensor, delta: torch.Tensor, A_log: torch.Tensor,
                  B: torch.Tensor, C: torch.Tensor, D: Optional[torch.Tensor] = None, z: Optional[torch.Tensor] = None,
                  delta_bias: Optional[torch.Tensor] = None, conv_bias: Optional[torch.Tensor] = None,
                  conv_state: Optional[torch.Tensor] = None, initial_state: Optional[torch.Tensor] = None,
                  delta_softplus: bool = True, return_final_state: bool = False, return_conv_state: bool = False,
                  return_u: bool = False, *, out: Optional[torch.Tensor] = None,
                  final_state: Optional[torch.Tensor] = None, conv_state_out: Optional[torch.Tensor] = None,
                  u_out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                  discretization: str = "zoh", stream=None):
    """Causal depthwise conv1d (4 taps) + SiLU fused into the forward scan: u = SiLU(conv(x)) is formed
    on chip.  x, delta, z: (batch, dim, L) and B, C: (batch, dstate <= 16, L) in the io dtype;
    conv_weight (dim, 4), conv_bias (dim,), A_log (dim, dstate), D, delta_bias (dim,) float32;
    conv_state (batch, dim, 3) in the io dtype.  Returns y, followed by the final state, the final
    conv state and u for each of return_final_state, return_conv_state, return_u that is set."""
    lib = load_library()
    if x.dim() != 3:
        raise ValueError("x must be (batch, dim, L)")
    batch, dim, L = x.shape
    dev = x.device
    if dev.type != "cuda":
        raise ValueError("scan_fwd_conv needs device tensors (HIP)")
    io = _io_dtype(x)
    iot = x.dtype
    dstate = A_log.shape[-1] if A_log.dim() == 2 else -1
    _req("x", x, (batch, dim, L), iot, dev)
    _req("conv_weight", conv_weight, (dim, 4), torch.float32, dev)
    _req("conv_bias", conv_bias, (dim,), torch.float32, dev)
    _req("conv_state", conv_state, (batch, dim, 3), iot, dev)
    _req("delta", delta, (batch, dim, L), iot, dev)
    _req("A_log", A_log, (dim, dstate), torch.float32, dev)
    _req("B", B, (batch, dstate, L), iot, dev)
    _req("C", C, (batch, dstate, L), iot, dev)
    _req("D", D, (dim,), torch.float32, dev)
    _req("z", z, (batch, dim, L), iot, dev)
    _req("delta_bias", delta_bias, (dim,), torch.float32, dev)
    _req("initial_state", initial_state, (batch, dim, dstate), torch.float32, dev)
    y = out if out is not None else torch.empty((batch, dim, L), dtype=iot, device=dev)
    _req("out", y, (batch, dim, L), iot, dev)
    fs = final_state
    if fs is None and return_final_state:
        fs = torch.empty((batch, dim, dstate), dtype=torch.float32, device=dev)
    _req("final_state", fs, (batch, dim, dstate), torch.float32, dev)
    cso = conv_state_out
    if cso is None and return_conv_state:
        cso = torch.empty((batch, dim, 3), dtype=iot, device=dev)
    _req("conv_state_out", cso, (batch, dim, 3), iot, dev)
    uo = u_out
    if uo is None and return_u:
        uo = torch.empty((batch, dim, L), dtype=iot, device=dev)
    _req("u_out", uo, (batch, dim, L), iot, dev)
    need = fwd_workspace_size(batch, dim, dstate, L, io)
    ws = workspace
    if ws is None and need > 0:
        ws = torch.empty(need + 256, dtype=torch.uint8, device=dev)
    ws_ptr, ws_bytes = None, 0
    if ws is not None:
        base = ws.data_ptr()
        off = (-base) % 256
        ws_ptr, ws_bytes = ctypes.c_void_p(base + off), max(0, ws.numel() * ws.element_size() - off)
    rc = lib.mamba_scan_fwd_conv(_ptr(x), _ptr(conv_weight), _ptr(conv_bias), _ptr(conv_state), _ptr(cso),
                                 _ptr(delta), _ptr(A_log), _ptr(B), _ptr(C), _ptr(D), _ptr(z), _ptr(delta_bias),
                                 _ptr(initial_state), _ptr(fs), _ptr(uo), _ptr(y), batch, dim, dstate, L, io,
                                 _flags(delta_softplus, discretization), ws_ptr, ws_bytes, _stream(dev, stream))
    _check("mamba_scan_fwd_conv", rc)
    res = [y]
    if return_final_state:
        res.append(fs)
    if return_conv_state:
        res.append(cso)
    if return_u:
        res.append(uo)
    return res[0] if len(res) == 1 else tuple(res)


def fwd_varlen_workspace_size(nseq: int, dim: int, dstate: int, total_len: int, io_dtype: int = BF16) -> int:
    n = load_library().mamba_scan_fwd_varlen_workspace_size(nseq, dim, dstate, total_len, io_dtype)
    if n == ctypes.c_size_t(-1).value:
        raise ValueError("mamba_scan_fwd_varlen_workspace_size: sizes rejected")
    return int(n)


@_on_stream
def scan_fwd_varlen(u: torch.Tensor, delta: torch.Tensor, A_log: torch.Tensor, B: torch.Tensor, C: torch.Tensor,
                    cu_seqlens: torch.Tensor, D: Optional[torch.Tensor] = None, z: Optional[torch.Tensor] = None,
                    delta_bias: Optional[torch.Tensor] = None, initial_states: Optional[torch.Tensor] = None,
                    delta_softplus: bool = True, return_final_states: bool = False, *,
                    out: Optional[torch.Tensor] = None, final_states: Optional[torch.Tensor] = None,
                    workspace: Optional[torch.Tensor] = None, discretization: str = "zoh", stream=None):
    """Variable-length batch: nseq sequences packed along time.  u, delta, z: (dim, total); B, C:
    (dstate, total) in the io dtype; cu_seqlens (nseq + 1,) int64 on the device; initial_states
    (nseq, dim, dstate) float32.  Returns y (dim, total), or (y, final_states)."""
    lib = load_library()
    if u.dim() != 2:
        raise ValueError("u must be (dim, total)")
    dim, total = u.shape
    dev = u.device
    if dev.type != "cuda":
        raise ValueError("scan_fwd_varlen needs device tensors (HIP)")
    io = _io_dtype(u)
    iot = u.dtype
    dstate = A_log.shape[-1] if A_log.dim() == 2 else -1
    if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 2:
        raise ValueError("cu_seqlens must be (nseq + 1,)")
    nseq = cu_seqlens.numel() - 1
    _req("cu_seqlens", cu_seqlens, (nseq + 1,), torch.int64, dev)
    _req("u", u, (dim, total), iot, dev)
    _req("delta", delta, (dim, total), iot, dev)
    _req("A_log", A_log, (dim, dstate), torch.float32, dev)
    _req("B", B, (dstate, total), iot, dev)
    _req("C", C, (dstate, total), iot, dev)
    _req("D", D, (dim,), torch.float32, dev)
    _req("z", z, (dim, total), iot, dev)
    _req("delta_bias", delta_bias, (dim,), torch.float32, dev)
    _req("initial_states", initial_states, (nseq, dim, dstate), torch.float32, dev)
    y = out if out is not None else torch.empty((dim, total), dtype=iot, device=dev)
    _req("out", y, (dim, total), iot, dev)
    fs = final_states
    if fs is None and return_final_states:
        fs = torch.empty((nseq, dim, dstate), dtype=torch.float32, device=dev)
    _req("final_states", fs, (nseq, dim, dstate), torch.float32, dev)
    need = fwd_varlen_workspace_size(nseq, dim, dstate, total, io)
    ws = workspace
    if ws is None and need > 0:
        ws = torch.empty(need + 256, dtype=torch.uint8, device=dev)
    ws_ptr, ws_bytes = None, 0
    if ws is not None:
        base = ws.data_ptr()
        off = (-base) % 256
        ws_ptr, ws_bytes = ctypes.c_void_p(base + off), max(0, ws.numel() * ws.element_size() - off)
    rc = lib.mamba_scan_fwd_varlen(_ptr(u), _ptr(delta), _ptr(A_log), _ptr(B), _ptr(C), _ptr(D), _ptr(z),
                                   _ptr(delta_bias), _ptr(cu_seqlens), _ptr(initial_states), _ptr(fs), _ptr(y),
                                   nseq, dim, dstate, total, io, _flags(delta_softplus, discretization), ws_ptr,
                                   ws_bytes, _stream(dev, stream))
    _check("mamba_scan_fwd_varlen", rc)
    return (y, fs) if return_final_states else y


@_on_stream
def scan_step(state: torch.Tensor, x: torch.Tensor, dt: torch.Tensor, A_log: torch.Tensor, B: torch.Tensor,
              C: torch.Tensor, D: Optional[torch.Tensor] = None, z: Optional[torch.Tensor] = None,
              dt_bias: Optional[torch.Tensor] = None, dt_softplus: bool = True, *,
              out: Optional[torch.Tensor] = None, discretization: str = "zoh", stream=None) -> torch.Tensor:
    """One recurrent step (discretization as in scan_fwd).  state (batch, dim, dstate) float32 is updated IN PLACE; x, dt, z (batch, dim)
    and B, C (batch, dstate) in the io dtype.  Returns y (batch, dim)."""
    lib = load_library()
    if state.dim() != 3:
        raise ValueError("state must be (batch, dim, dstate)")
    batch, dim, dstate = state.shape
    dev = state.device
    if dev.type != "cuda":
        raise ValueError("scan_step needs device tensors (HIP)")
    io = _io_dtype(x)
    iot = x.dtype
    _req("state", state, (batch, dim, dstate), torch.float32, dev)
    _req("x", x, (batch, dim), iot, dev)
    _req("dt", dt, (batch, dim), iot, dev)
    _req("A_log", A_log, (dim, dstate), torch.float32, dev)
    _req("B", B, (batch, dstate), iot, dev)
    _req("C", C, (batch, dstate), iot, dev)
    _req("D", D, (dim,), torch.float32, dev)
    _req("z", z, (batch, dim), iot, dev)
    _req("dt_bias", dt_bias, (dim,), torch.float32, dev)
    y = out if out is not None else torch.empty((batch, dim), dtype=iot, device=dev)
    _req("out", y, (batch, dim), iot, dev)
    rc = lib.mamba_scan_step(_ptr(state), _ptr(x), _ptr(dt), _ptr(A_log), _ptr(B), _ptr(C), _ptr(D), _ptr(z),
                             _ptr(dt_bias), _flags(dt_softplus, discretization), _ptr(y), batch, dim, dstate, io,
                             _stream(dev, stream))
    _check("mamba_scan_step", rc)
    return y


def bwd_workspace_size(batch: int, dim: int, dstate: int, seqlen: int, io_dtype: int = BF16) -> int:
    n = load_library().mamba_scan_bwd_workspace_size(batch, dim, dstate, seqlen, io_dtype)
    if n == ctypes.c_size_t(-1).value:
        raise ValueError("mamba_scan_bwd_workspace_size: sizes rejected")
    return int(n)


@_on_stream
def scan_bwd(u: torch.Tensor, delta: torch.Tensor, A_log: torch.Tensor, B: torch.Tensor, C: torch.Tensor,
             dy: torch.Tensor, D: Optional[torch.Tensor] = None, z: Optional[torch.Tensor] = None,
             delta_bias: Optional[torch.Tensor] = None, initial_state: Optional[torch.Tensor] = None,
             d_final_state: Optional[torch.Tensor] = None, delta_softplus: bool = True, *,
             workspace: Optional[torch.Tensor] = None, discretization: str = "zoh", stream=None) -> dict:
    """Selective-scan backward.  Inputs as in scan_fwd plus dy (batch, dim, L) in the io dtype and
    d_final_state (batch, dim, dstate) float32.  Returns a dict of gradients: du, ddelta, dz, dB, dC in
    the io dtype; dA_log, dD, ddelta_bias, d_initial_state in float32 (dD, dz, ddelta_bias and
    d_initial_state only when D, z, delta_bias and initial_state are given)."""
    lib = load_library()
    if u.dim() != 3:
        raise ValueError("u must be (batch, dim, L)")
    batch, dim, L = u.shape
    dev = u.device
    if dev.type != "cuda":
        raise ValueError("scan_bwd needs device tensors (HIP)")
    io = _io_dtype(u)
    iot = u.dtype
    dstate = A_log.shape[-1] if A_log.dim() == 2 else -1
    _req("u", u, (batch, dim, L), iot, dev)
    _req("delta", delta, (batch, dim, L), iot, dev)
    _req("A_log", A_log, (dim, dstate), torch.float32, dev)
    _req("B", B, (batch, dstate, L), iot, dev)
    _req("C", C, (batch, dstate, L), iot, dev)
    _req("dy", dy, (batch, dim, L), iot, dev)
    _req("D", D, (dim,), torch.float32, dev)
    _req("z", z, (batch, dim, L), iot, dev)
    _req("delta_bias", delta_bias, (dim,), torch.float32, dev)
    _req("initial_state", initial_state, (batch, dim, dstate), torch.float32, dev)
    _req("d_final_state", d_final_state, (batch, dim, dstate), torch.float32, dev)
    f32 = torch.float32
    g = {"du": torch.empty((batch, dim, L), dtype=iot, device=dev),
         "ddelta": torch.empty((batch, dim, L), dtype=iot, device=dev),
         "dA_log": torch.empty((dim, dstate), dtype=f32, device=dev),
         "dB": torch.empty((batch, dstate, L), dtype=iot, device=dev),
         "dC": torch.empty((batch, dstate, L), dtype=iot, device=dev),
         "dD": torch.empty((dim,), dtype=f32, device=dev) if D is not None else None,
         "dz": torch.empty((batch, dim, L), dtype=iot, device=dev) if z is not None else None,
         "ddelta_bias": torch.empty((dim,), dtype=f32, device=dev) if delta_bias is not None else None,
         "d_initial_state": torch.empty((batch, dim, dstate), dtype=f32, device=dev)
         if initial_state is not None else None}
    need = bwd_workspace_size(batch, dim, dstate, L, io)
    ws = workspace
    if ws is None and need > 0:
        ws = torch.empty(need + 256, dtype=torch.uint8, device=dev)
    ws_ptr, ws_bytes = None, 0
    if ws is not None:
        base = ws.data_ptr()
        off = (-base) % 256
        ws_ptr, ws_bytes = ctypes.c_void_p(base + off), max(0, ws.numel() * ws.element_size() - off)
    rc = lib.mamba_scan_bwd(_ptr(u), _ptr(delta), _ptr(A_log), _ptr(B), _ptr(C), _ptr(D), _ptr(z),
                            _ptr(delta_bias), _ptr(initial_state), _ptr(dy), _ptr(d_final_state), _ptr(g["du"]),
                            _ptr(g["ddelta"]), _ptr(g["dA_log"]), _ptr(g["dB"]), _ptr(g["dC"]), _ptr(g["dD"]),
                            _ptr(g["dz"]), _ptr(g["ddelta_bias"]), _ptr(g["d_initial_state"]), batch, dim, dstate,
                            L, io, _flags(delta_softplus, discretization), ws_ptr, ws_bytes, _stream(dev, stream))
    _check("mamba_scan_bwd", rc)
    return g


@_on_stream
def conv1d_fwd(x: torch.Tensor, weight: torch.Tensor, bias: Optional[torch.Tensor] = None,
               conv_state: Optional[torch.Tensor] = None, silu: bool = True, return_state: bool = False, *,
               out: Optional[torch.Tensor] = None, state_out: Optional[torch.Tensor] = None, stream=None):
    """Causal depthwise conv1d (+ SiLU).  x (batch, dim, L) in the io dtype, weight (dim, K) float32 with
    K <= 4, bias (dim,) float32, conv_state (batch, dim, K-1) in the io dtype (inputs before x, oldest
    first).  Returns u (batch, dim, L), or (u, final conv state) if return_state (state_out may be
    conv_state itself, for an in-place update)."""
    lib = load_library()
    if x.dim() != 3:
        raise ValueError("x must be (batch, dim, L)")
    batch, dim, L = x.shape
    dev = x.device
    if dev.type != "cuda":
        raise ValueError("conv1d_fwd needs device tensors (HIP)")
    io = _io_dtype(x)
    iot = x.dtype
    K = weight.shape[-1] if weight.dim() == 2 else -1
    _req("weight", weight, (dim, K), torch.float32, dev)
    _req("bias", bias, (dim,), torch.float32, dev)
    _req("conv_state", conv_state, (batch, dim, K - 1), iot, dev)
    u = out if out is not None else torch.empty((batch, dim, L), dtype=iot, device=dev)
    _req("out", u, (batch, dim, L), iot, dev)
    so = state_out
    if so is None and return_state:
        so = torch.empty((batch, dim, K - 1), dtype=iot, device=dev)
    _req("state_out", so, (batch, dim, K - 1), iot, dev)
    rc = lib.mamba_conv1d_fwd(_ptr(x), _ptr(weight), _ptr(bias), _ptr(conv_state), _ptr(so), _ptr(u), batch, dim,
                              L, K, io, int(bool(silu)), _stream(dev, stream))
    _check("mamba_conv1d_fwd", rc)
    return (u, so) if return_state else u


@_on_stream
def ssd_fwd(x: torch.Tensor, dt: torch.Tensor, A_log: torch.Tensor, B: torch.Tensor, C: torch.Tensor,
            D: Optional[torch.Tensor] = None, z: Optional[torch.Tensor] = None,
            dt_bias: Optional[torch.Tensor] = None, initial_state: Optional[torch.Tensor] = None,
            dt_softplus: bool = True, return_final_state: bool = False, *, out: Optional[torch.Tensor] = None,
            final_state: Optional[torch.Tensor] = None, discretization: str = "zoh", stream=None):
    """Multi-head SSM with a scalar decay per head (state-space-duality form).  x, z: (batch, L, H, P);
    dt: (batch, L, H); B, C: (batch, L, N) in bfloat16; A_log, D, dt_bias: (H,) float32;
    initial_state (batch, H, P, N) float32.  Returns y (batch, L, H, P), or (y, final_state)."""
    lib = load_library()
    if x.dim() != 4:
        raise ValueError("x must be (batch, L, H, P)")
    batch, L, H, P = x.shape
    dev = x.device
    if dev.type != "cuda":
        raise ValueError("ssd_fwd needs device tensors (HIP)")
    io = _io_dtype(x)
    iot = x.dtype
    N = B.shape[-1] if B.dim() == 3 else -1
    _req("x", x, (batch, L, H, P), iot, dev)
    _req("dt", dt, (batch, L, H), iot, dev)
    _req("A_log", A_log, (H,), torch.float32, dev)
    _req("B", B, (batch, L, N), iot, dev)
    _req("C", C, (batch, L, N), iot, dev)
    _req("D", D, (H,), torch.float32, dev)
    _req("z", z, (batch, L, H, P), iot, dev)
    _req("dt_bias", dt_bias, (H,), torch.float32, dev)
    _req("initial_state", initial_state, (batch, H, P, N), torch.float32, dev)
    y = out if out is not None else torch.empty((batch, L, H, P), dtype=iot, device=dev)
    _req("out", y, (batch, L, H, P), iot, dev)
    fs = final_state
    if fs is None and return_final_state:
        fs = torch.empty((batch, H, P, N), dtype=torch.float32, device=dev)
    _req("final_state", fs, (batch, H, P, N), torch.float32, dev)
    rc = lib.mamba_ssd_fwd(_ptr(x), _ptr(dt), _ptr(A_log), _ptr(B), _ptr(C), _ptr(D), _ptr(z), _ptr(dt_bias),
                           _ptr(initial_state), _ptr(fs), _ptr(y), batch, L, H, P, N, io,
                           _flags(dt_softplus, discretization), _stream(dev, stream))
    _check("mamba_ssd_fwd", rc)
    return (y, fs) if return_final_state else y


def _entry(fn):
    """Runs fn with the device of its first parameter, passed by place or by name, current (the library launches on
    the current device) and with its `stream` argument, if any, made the current stream, as _on_stream does."""
    on_stream = _on_stream(fn)
    first = next(iter(inspect.signature(fn).parameters))

    @functools.wraps(fn)
    def run(*args, **kwargs):
        t0 = args[0] if args else kwargs.get(first)
        dev = t0.get_device() if isinstance(t0, torch.Tensor) and t0.is_cuda else -1
        if dev < 0 or dev == torch.cuda.current_device():
            return fn(*args, **kwargs) if kwargs.get("stream") is None else on_stream(*args, **kwargs)
        with torch.cuda.device(dev):
            return fn(*args, **kwargs) if kwargs.get("stream") is None else on_stream(*args, **kwargs)

    return run


def _need(name: str, t, shape, dtype, device) -> Optional[int]:
    """_req of a contiguous tensor (or None), fast where it passes; returns its address (None)."""
    if t is None:
        return None
    if not (isinstance(t, torch.Tensor) and t.shape == shape and t.dtype == dtype and t.device == device and t.is_contiguous()):
        _req(name, t, shape, dtype, device)
    return t.data_ptr()


def _token_stride(name: str, t: torch.Tensor, shape, dtype, device) -> int:
    """Checks a tensor of tokens whose rows are contiguous but may lie apart; returns the elements between them."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.shape != shape or t.dtype != dtype or t.device != device:
        _req(name, t, shape, dtype, device)
    st = t.stride()
    if not (st[-1] == 1 and (len(st) == 2 or st[1] == shape[2])) and shape[0] and not t[0].is_contiguous():
        raise ValueError(f"{name}: the elements of a token must be contiguous")
    if shape[0] > 1:
        return st[0]
    width = shape[1] if len(shape) == 2 else shape[1] * shape[2]
    return -(-width // 8) * 8


def _overlap(a: int, a_bytes: int, b: int, b_bytes: int) -> bool:
    """Whether two ranges of memory share a byte."""
    return a < b + b_bytes and b < a + a_bytes and a_bytes > 0 and b_bytes > 0


def _current_handle(index: int) -> int:
    return torch.cuda.current_stream(index).cuda_stream


# the same without the Stream object, where torch has it (0.1 against 1.9 us a call)
_current_handle = getattr(torch._C, "_cuda_getCurrentRawStream", _current_handle)


def _handle(device: torch.device, stream) -> int:
    """The HIP stream of a call: its stream argument (already current) or the current stream."""
    if stream is None:
        return _current_handle(device.index)
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _scratch(need: int, workspace: Optional[torch.Tensor], device):
    """(tensor to keep alive, 256-byte aligned address, bytes) of a call's workspace."""
    ws = workspace
    if ws is None:
        if need == 0:
            return None, None, 0
        ws = torch.empty(need + 256, dtype=torch.uint8, device=device)
    elif ws.device != device:
        raise ValueError(f"workspace is on {ws.device}, expected {device}")
    elif not ws.is_contiguous():
        raise ValueError("workspace must be contiguous")
    base = ws.data_ptr()
    off = (-base) % 256
    return ws, base + off, max(0, ws.numel() * ws.element_size() - off)


@_entry
def ssd_conv_fwd_varlen(x: torch.Tensor, weight: torch.Tensor, cu_seqlens: torch.Tensor,
                        bias: Optional[torch.Tensor] = None, conv_state: Optional[torch.Tensor] = None,
                        slots: Optional[torch.Tensor] = None, positions: Optional[torch.Tensor] = None,
                        silu: bool = True, *, out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """The SSD layer's causal depthwise conv (+ SiLU) over packed sequences, token-major.  x (total, width)
    in the io dtype (its rows may lie apart, as a slice of a projection's output), weight (width, K) float32
    with K 2 to 4, bias (width,) float32, cu_seqlens (nseq + 1,) int64 on the device.  conv_state
    (nslots, K, width) in the io dtype is updated IN PLACE: sequence s reads and writes ring slots[s]
    (outside [0, nslots): starts from zeros, keeps nothing), positions[s] tokens (0: a new request) behind
    it, both (nseq,) int64.  No slot may be named twice.  Returns u (total, width); rows outside every
    sequence are not written."""
    lib = load_library()
    if x.dim() != 2:
        raise ValueError("x must be (total, width)")
    total, width = x.shape
    dev = x.device
    if dev.type != "cuda":
        raise ValueError("ssd_conv_fwd_varlen needs device tensors (HIP)")
    io, iot = _io_dtype(x), x.dtype
    if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 2:
        raise ValueError("cu_seqlens must be (nseq + 1,)")
    nseq = cu_seqlens.numel() - 1
    K = weight.shape[-1] if weight.dim() == 2 else -1
    xs = _token_stride("x", x, (total, width), iot, dev)
    f32, i64 = torch.float32, torch.int64
    nslots = 0
    if conv_state is not None:
        nslots = conv_state.shape[0] if conv_state.dim() == 3 else -1
        if slots is None or positions is None:
            raise ValueError("conv_state needs slots and positions")
    if out is not None and total:
        e = x.element_size()
        at, end = out.data_ptr(), total * width * e
        if _overlap(at, end, x.data_ptr(), ((total - 1) * xs + width) * e):
            raise ValueError("out must not overlap x, whose earlier tokens later ones read")
        if conv_state is not None and _overlap(at, end, conv_state.data_ptr(), conv_state.numel() * e):
            raise ValueError("out must not overlap conv_state")
    u = out if out is not None else torch.empty((total, width), dtype=iot, device=dev)
    rc = lib.mamba_ssd_conv_fwd_varlen(
        x.data_ptr(), _need("weight", weight, (width, K), f32, dev), _need("bias", bias, (width,), f32, dev),
        _need("cu_seqlens", cu_seqlens, (nseq + 1,), i64, dev),
        _need("conv_state", conv_state, (nslots, K, width), iot, dev), _need("slots", slots, (nseq,), i64, dev),
        _need("positions", positions, (nseq,), i64, dev), _need("out", u, (total, width), iot, dev), nseq, total, width,
        K, xs, nslots, io, 1 if silu else 0, _handle(dev, stream))
    _check("mamba_ssd_conv_fwd_varlen", rc)
    return u


def ssd_fwd_varlen_workspace_size(nseq: int, total_len: int, nheads: int, headdim: int, dstate: int,
                                  ngroups: int = 1, max_seqlen: int = 0) -> int:
    n = load_library().mamba_ssd_fwd_varlen_workspace_size(nseq, total_len, nheads, headdim, dstate, ngroups, max_seqlen)
    if n == ctypes.c_size_t(-1).value:
        raise ValueError("mamba_ssd_fwd_varlen_workspace_size: sizes rejected")
    return int(n)


@_entry
def ssd_fwd_varlen(x: torch.Tensor, dt: torch.Tensor, A_log: torch.Tensor, B: torch.Tensor, C: torch.Tensor,
                   cu_seqlens: torch.Tensor, D: Optional[torch.Tensor] = None, z: Optional[torch.Tensor] = None,
                   dt_bias: Optional[torch.Tensor] = None, state: Optional[torch.Tensor] = None,
                   slots: Optional[torch.Tensor] = None, positions: Optional[torch.Tensor] = None,
                   dt_softplus: bool = True, *, max_seqlen: int = 0, out: Optional[torch.Tensor] = None,
                   workspace: Optional[torch.Tensor] = None, discretization: str = "zoh", stream=None) -> torch.Tensor:
    """ssd_fwd over packed sequences.  x, z (total, H, P), dt (total, H), B, C (total, G, N) in bfloat16, heads in
    G groups that share B and C; tokens may lie apart (slices of a wider row), each contiguous; x, B, C and
    z 16-byte aligned.  cu_seqlens (nseq + 1,) int64 on the device.  state (nslots, H, P, N) float32 is
    updated IN PLACE by slot, as conv_state in ssd_conv_fwd_varlen.  max_seqlen, the longest sequence's length where
    the host knows it, only serves the choice of launches.  Returns y (total, H, P); rows outside every
    sequence are not written.  out may be x or z itself (contiguous), and overlap no other argument."""
    lib = load_library()
    if x.dim() != 3:
        raise ValueError("x must be (total, H, P)")
    total, H, P = x.shape
    dev = x.device
    if dev.type != "cuda":
        raise ValueError("ssd_fwd_varlen needs device tensors (HIP)")
    io, iot = _io_dtype(x), x.dtype
    if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 2:
        raise ValueError("cu_seqlens must be (nseq + 1,)")
    nseq = cu_seqlens.numel() - 1
    if B.dim() != 3:
        raise ValueError("B must be (total, G, N)")
    G, N = B.shape[1:]
    f32 = torch.float32
    xs = _token_stride("x", x, (total, H, P), iot, dev)
    ds = _token_stride("dt", dt, (total, H), iot, dev)
    bs = _token_stride("B", B, (total, G, N), iot, dev)
    cs = _token_stride("C", C, (total, G, N), iot, dev)
    zs = 0 if z is None else _token_stride("z", z, (total, H, P), iot, dev)
    i64 = torch.int64
    nslots = 0
    if state is not None:
        nslots = state.shape[0] if state.dim() == 4 else -1
        if slots is None or positions is None:
            raise ValueError("state needs slots and positions")
    if out is not None and total:
        at, end = out.data_ptr(), total * H * P * 2
        px, pz, far = x.data_ptr(), 0 if z is None else z.data_ptr(), total - 1
        if (at != px or xs != H * P) and _overlap(at, end, px, (far * xs + H * P) * 2) or \
                z is not None and (at != pz or zs != H * P) and _overlap(at, end, pz, (far * zs + H * P) * 2) or \
                _overlap(at, end, dt.data_ptr(), (far * ds + H) * 2) or \
                _overlap(at, end, B.data_ptr(), (far * bs + G * N) * 2) or \
                _overlap(at, end, C.data_ptr(), (far * cs + G * N) * 2) or \
                state is not None and _overlap(at, end, state.data_ptr(), state.numel() * 4):
            raise ValueError("out overlaps an argument that other workgroups read (x or z itself may be out)")
    y = out if out is not None else torch.empty((total, H, P), dtype=iot, device=dev)
    ws, ws_ptr, ws_bytes = _scratch(ssd_fwd_varlen_workspace_size(nseq, total, H, P, N, G, max_seqlen), workspace, dev)
    rc = lib.mamba_ssd_fwd_varlen(
        x.data_ptr(), dt.data_ptr(), _need("A_log", A_log, (H,), f32, dev), B.data_ptr(), C.data_ptr(),
        _need("D", D, (H,), f32, dev), None if z is None else z.data_ptr(), _need("dt_bias", dt_bias, (H,), f32, dev),
        _need("cu_seqlens", cu_seqlens, (nseq + 1,), i64, dev), _need("state", state, (nslots, H, P, N), f32, dev),
        _need("slots", slots, (nseq,), i64, dev), _need("positions", positions, (nseq,), i64, dev),
        _need("out", y, (total, H, P), iot, dev), nseq, total, H, P, N, G, max_seqlen, nslots,
        xs, ds, bs, cs, zs, io,
        _flags(dt_softplus, discretization), ws_ptr, ws_bytes, _handle(dev, stream))
    _check("mamba_ssd_fwd_varlen", rc)
    return y


@_entry
def ssd_step(xbc: torch.Tensor, dt: torch.Tensor, A_log: torch.Tensor, conv_weight: torch.Tensor,
             conv_state: torch.Tensor, state: torch.Tensor, positions: torch.Tensor,
             slots: Optional[torch.Tensor] = None, D: Optional[torch.Tensor] = None, z: Optional[torch.Tensor] = None,
             dt_bias: Optional[torch.Tensor] = None, conv_bias: Optional[torch.Tensor] = None,
             dt_softplus: bool = True, *, out: Optional[torch.Tensor] = None, discretization: str = "zoh",
             stream=None) -> torch.Tensor:
    """One token per request: the conv + SiLU of its x | B | C channels (xbc (batch, H P + 2 G N)), the SSM
    update and readout, the D skip and the gate, in one launch.  dt (batch, H) and z (batch, H, P) as xbc in
    the io dtype (float32 or bfloat16; rows may lie apart).  conv_state (nslots, K, width) in the io dtype and
    state (nslots, H, P, N) float32 are updated IN PLACE at slots[i] (default: i); a row whose slot is
    outside [0, nslots) is padding and its y is not written.  positions (batch,): tokens each request has
    behind it (0: a new one).  No slot may be named twice.  Returns y (batch, H, P); out may be z itself
    (contiguous), and overlap no other argument."""
    lib = load_library()
    if xbc.dim() != 2 or state.dim() != 4:
        raise ValueError("xbc must be (batch, width) and state (nslots, H, P, N)")
    batch, width = xbc.shape
    nslots, H, P, N = state.shape
    dev = xbc.device
    if dev.type != "cuda":
        raise ValueError("ssd_step needs device tensors (HIP)")
    io, iot = _io_dtype(xbc), xbc.dtype
    K = conv_weight.shape[-1] if conv_weight.dim() == 2 else -1
    G, rest = divmod(width - H * P, 2 * N)
    if rest or G < 1:
        raise ValueError(f"xbc has {width} channels, expected {H * P} + 2 G {N}")
    f32 = torch.float32
    xs = _token_stride("xbc", xbc, (batch, width), iot, dev)
    ds = _token_stride("dt", dt, (batch, H), iot, dev)
    zs = 0 if z is None else _token_stride("z", z, (batch, H, P), iot, dev)
    if slots is None and batch > nslots:
        raise ValueError(f"{batch} rows without slots, but {nslots} pool entries")
    if positions is None:
        raise ValueError("ssd_step needs positions")
    if out is not None and batch:
        e = xbc.element_size()
        at, end, far, pz = out.data_ptr(), batch * H * P * e, batch - 1, 0 if z is None else z.data_ptr()
        if _overlap(at, end, xbc.data_ptr(), (far * xs + width) * e) or _overlap(at, end, dt.data_ptr(), (far * ds + H) * e) or \
                z is not None and (at != pz or far and zs != H * P) and _overlap(at, end, pz, (far * zs + H * P) * e) or \
                _overlap(at, end, conv_state.data_ptr(), nslots * K * width * e) or \
                _overlap(at, end, state.data_ptr(), state.numel() * 4):
            raise ValueError("out overlaps an argument that other workgroups read (z itself may be out)")
    y = out if out is not None else torch.empty((batch, H, P), dtype=iot, device=dev)
    i64 = torch.int64
    rc = lib.mamba_ssd_step(
        xbc.data_ptr(), dt.data_ptr(), _need("A_log", A_log, (H,), f32, dev),
        _need("conv_weight", conv_weight, (width, K), f32, dev), _need("conv_bias", conv_bias, (width,), f32, dev),
        _need("conv_state", conv_state, (nslots, K, width), iot, dev), _need("state", state, (nslots, H, P, N), f32, dev),
        _need("slots", slots, (batch,), i64, dev), _need("positions", positions, (batch,), i64, dev),
        _need("D", D, (H,), f32, dev), None if z is None else z.data_ptr(), _need("dt_bias", dt_bias, (H,), f32, dev),
        _need("out", y, (batch, H, P), iot, dev), batch, H, P, N, G, K, nslots, xs, ds, zs, io,
        _flags(dt_softplus, discretization), _handle(dev, stream))
    _check("mamba_ssd_step", rc)
    return y


_NORM_OUT = {None: 0, "row": 1, "mx": 2}   # MAMBA_NORM_OUT_*


@_entry
def rms_norm_fwd(x: torch.Tensor, weight: torch.Tensor, residual: Optional[torch.Tensor] = None, *, eps: float = 1e-5,
                 quant: Optional[str] = None, return_rstd: bool = False, out: Optional[torch.Tensor] = None,
                 scales: Optional[torch.Tensor] = None, residual_out: Optional[torch.Tensor] = None, stream=None):
    """Root-mean-square norm of r = x + residual over the last axis: y = r rstd weight.  x (..., dim) in the io
    dtype, weight (dim,) float32, residual (..., dim) in the io dtype or float32.  quant None: y in the io
    dtype; "row": y in float8_e4m3fn with one float32 scale per row (shape x.shape[:-1]); "mx": y in
    float8_e4m3fn with one float8_e8m0fnu scale per 32 columns.  Returns y, followed by the scales (quant), r in
    the residual's dtype (residual given) and rstd float32 (return_rstd).  out and residual_out may each be x or
    residual itself where the dtype is the same; outputs overlap nothing else."""
    lib = load_library()
    if x.dim() < 1 or x.shape[-1] < 1:
        raise ValueError("x must be (..., dim)")
    shape, dim, dev = x.shape, x.shape[-1], x.device
    rows = x.numel() // dim
    if dev.type != "cuda":
        raise ValueError("rms_norm_fwd needs device tensors (HIP)")
    if quant not in _NORM_OUT:
        raise ValueError(f"quant must be None, 'row' or 'mx', got {quant!r}")
    given = out is not None or residual_out is not None or scales is not None
    io, iot = _io_dtype(x), x.dtype
    rio = io
    ro = residual_out
    if residual is not None:
        rio = _io_dtype(residual)
        if rio != io and rio != F32:
            raise ValueError("residual must have x's dtype or float32")
        rt = residual.dtype
        if ro is None:
            ro = torch.empty_like(residual)
    elif ro is not None:
        raise ValueError("residual_out needs residual")
    if residual is None:
        rt = iot
    if quant is None:
        if scales is not None:
            raise ValueError("scales needs quant")
        yt = st = iot
        ss = shape
    else:
        yt = torch.float8_e4m3fn
        st = torch.float32 if quant == "row" else torch.float8_e8m0fnu
        ss = shape[:-1] if quant == "row" else shape[:-1] + ((dim + 31) // 32,)
        if scales is None:
            scales = torch.empty(ss, dtype=st, device=dev)
    y = out if out is not None else torch.empty_like(x) if quant is None else torch.empty(shape, dtype=yt, device=dev)
    if given and rows:
        ins = [t for t in (x, residual) if t is not None]
        outs = [t for t in (y, ro, scales) if t is not None]
        for i, t in enumerate(outs):
            at, end = t.data_ptr(), t.numel() * t.element_size()
            if any(_overlap(at, end, o.data_ptr(), o.numel() * o.element_size()) for o in outs[:i] + [weight]) or \
                    any(_overlap(at, end, o.data_ptr(), o.numel() * o.element_size()) for o in ins
                        if t is scales or t.dtype != o.dtype or at != o.data_ptr()):
                raise ValueError("an output overlaps another argument (x or residual itself may be out or residual_out)")
    rstd = torch.empty(shape[:-1], dtype=torch.float32, device=dev) if return_rstd else None
    rc = lib.mamba_rms_norm_fwd(
        _need("x", x, shape, iot, dev), _need("residual", residual, shape, rt, dev),
        _need("weight", weight, (dim,), torch.float32, dev), eps, _need("residual_out", ro, shape, rt, dev),
        _need("out", y, shape, yt, dev), _need("scales", scales, ss, st, dev), None if rstd is None else rstd.data_ptr(),
        rows, dim, io, rio, _NORM_OUT[quant], _handle(dev, stream))
    _check("mamba_rms_norm_fwd", rc)
    res = [y]
    if quant is not None:
        res.append(scales)
    if residual is not None:
        res.append(ro)
    if return_rstd:
        res.append(rstd)
    return res[0] if len(res) == 1 else tuple(res)


def rms_norm_bwd_workspace_size(rows: int, dim: int) -> int:
    n = load_library().mamba_rms_norm_bwd_workspace_size(rows, dim)
    if n == ctypes.c_size_t(-1).value:
        raise ValueError("mamba_rms_norm_bwd_workspace_size: sizes rejected")
    return int(n)


@_entry
def rms_norm_bwd(dy: torch.Tensor, r: torch.Tensor, weight: torch.Tensor, rstd: torch.Tensor,
                 d_residual: Optional[torch.Tensor] = None, return_dresidual: bool = False, *,
                 workspace: Optional[torch.Tensor] = None, stream=None) -> dict:
    """Gradient of rms_norm_fwd.  dy (..., dim) in the io dtype; r, what was normed (residual_out, or x where there
    was no residual), in the io dtype or float32; rstd float32 from the forward; d_residual, the gradient that
    reaches r from the residual stream, in r's dtype.  Returns a dict: dx in the io dtype, dweight float32, and
    with d_residual or return_dresidual also dresidual, the gradient of r, in r's dtype (dx itself where that is the io
    dtype; for a float32 residual of a bfloat16 layer dx alone is the gradient cut to 8 bits)."""
    lib = load_library()
    if dy.dim() < 1 or dy.shape[-1] < 1:
        raise ValueError("dy must be (..., dim)")
    shape, dim, dev = dy.shape, dy.shape[-1], dy.device
    rows = dy.numel() // dim
    if dev.type != "cuda":
        raise ValueError("rms_norm_bwd needs device tensors (HIP)")
    io, iot = _io_dtype(dy), dy.dtype
    rio = _io_dtype(r)
    if rio != io and rio != F32:
        raise ValueError("r must have dy's dtype or float32")
    f32, rt = torch.float32, r.dtype
    dx = torch.empty_like(dy)
    return_dresidual = return_dresidual or d_residual is not None
    apart = return_dresidual and rio != io
    dres = torch.empty_like(r) if apart else None
    dw = torch.empty_like(weight)
    ws, ws_ptr, ws_bytes = _scratch(rms_norm_bwd_workspace_size(rows, dim), workspace, dev)
    rc = lib.mamba_rms_norm_bwd(
        _need("dy", dy, shape, iot, dev), _need("r", r, shape, rt, dev), _need("weight", weight, (dim,), f32, dev),
        _need("rstd", rstd, shape[:-1], f32, dev), _need("d_residual", d_residual, shape, rt, dev), dx.data_ptr(),
        None if dres is None else dres.data_ptr(), dw.data_ptr(), rows, dim, io, rio, ws_ptr, ws_bytes, _handle(dev, stream))
    _check("mamba_rms_norm_bwd", rc)
    g = {"dx": dx, "dweight": dw}
    if return_dresidual:
        g["dresidual"] = dres if apart else dx
    return g
