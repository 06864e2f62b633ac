"""B200-native selective scan (S6): thin Python binding over libmss.so.

Argument marshalling only.  Every step of the forward pass and of the decode
update runs in the CUDA kernels of libmss.so; PyTorch supplies device memory
and streams.  There is no fallback: if the library is missing or a tensor is
not on a CUDA device, the call raises.

    y, last_state = scan_fwd(u, delta, A, B, C, D=D, z=z, delta_bias=bias)
    y = state_update(state, u, delta, A, B, C, D=D, z=z, delta_bias=bias)

Layouts (C-contiguous): u, delta, z, y [batch, dim, L]; B, C [batch, N, L];
A [dim, N] float32; D, delta_bias [dim] float32; last_state [batch, dim, N]
float32.  Decode: state [batch, dim, N] float32 (updated in place); u, delta,
z, y [batch, dim]; B, C [batch, N].  u, delta, z, B, C share one dtype,
float32 or bfloat16, which is also the dtype of y.

The gated linear recurrence (glr_fwd, glr_fwd_save, glr_bwd, glr_update) and
the residual add and norm (norm_fwd, norm_bwd) take token-major tensors,
[batch, L, dim] and [..., dim].
"""
from __future__ import annotations

import ctypes
import functools
import os
import threading

import torch

__all__ = ["scan_fwd", "scan_fwd_host", "scan_fwd_conv", "scan_bwd", "ssd_fwd", "bwd_workspace_size", "state_update", "state_update_conv",
           "glr_fwd", "glr_fwd_save", "glr_bwd", "glr_bwd_workspace_size", "glr_update",
           "norm_fwd", "norm_bwd", "norm_bwd_workspace_size",
           "get_device_error", "probe_pipe_rates", "selftest_timeout",
           "library_path", "workspace_size",
           "FLAG_GENERAL_A", "FLAG_SIMPLE", "FLAG_NO_SPLIT", "FLAG_ZOH_INPUT", "FLAG_SELFTEST_TIMEOUT",
           "ERR_DEVICE_TIMEOUT", "ERR_FLAGS", "ERR_OFFSETS", "SSD_FLAG_WARP_MMA", "MssError", "load_library"]

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_HERE, "libmss.so")

DTYPE_F32 = 0
DTYPE_BF16 = 1
FLAG_GENERAL_A = 0x1
FLAG_SIMPLE = 0x2
FLAG_NO_SPLIT = 0x4
FLAG_ZOH_INPUT = 0x8  # zero-order-hold input matrix (e^{Delta A} - 1)/A * B instead of Delta * B
FLAG_SELFTEST_TIMEOUT = 0x10  # the tiled kernel's bounded wait gives up on purpose (failure-path tests)
FLAG_SAVED_STATES = 0x20  # scan_bwd: the workspace holds the states scan_fwd_save stored
FLAG_PAIR_LANES = 0x40  # forward: the two-lanes-per-channel kernel where the four-lane one would run (fp32 io; bf16 io on grids of at most 384 units of 16 channels)
ERR_PATH = -12
ERR_FLAGS = -8
SSD_FLAG_WARP_MMA = 0x1  # ssd_fwd: the warp-level (mma.sync) kernels instead of the tcgen05 one
ERR_DEVICE_TIMEOUT = -7
ERR_OFFSETS = -13  # get_device_error: packed offsets decrease or leave the tokens
NORM_FLAG_RMS = 0x1

_lib = None
_lock = threading.Lock()


class MssError(RuntimeError):
    def __init__(self, code: int, what: str):
        self.code = code
        super().__init__(f"{what} failed: {_strerror(code)} (code {code})")


def library_path() -> str:
    return _LIB_PATH


def load_library():
    """Load libmss.so (built in-tree by __graft_entry__.build() or
    ``python -m selective_state_space_mss_b200.build``)."""
    global _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(_LIB_PATH):
                raise RuntimeError(
                    f"{_LIB_PATH} is not built; run `python -m selective_state_space_mss_b200.build`")
            lib = ctypes.CDLL(_LIB_PATH)
            vp, fp, i64, i, u32 = (ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64,
                                   ctypes.c_int, ctypes.c_uint)
            lib.mss_scan_fwd_ex.argtypes = [vp, vp, fp, vp, vp, fp, vp, fp, i, vp, fp,
                                            i64, i64, i64, i64, i, u32, vp]
            lib.mss_scan_fwd_ex.restype = i
            lib.mss_scan_fwd.argtypes = [vp, vp, fp, vp, vp, fp, vp, fp, i, vp, fp,
                                         i64, i64, i64, i64, i, vp]
            lib.mss_scan_fwd.restype = i
            lib.mss_scan_fwd_ex2.argtypes = [vp, vp, fp, vp, vp, fp, vp, fp, i, fp, vp, fp,
                                             i64, i64, i64, i64, i, u32, vp, i64, vp]
            lib.mss_scan_fwd_ex2.restype = i
            lib.mss_scan_fwd_save.argtypes = [vp, vp, fp, vp, vp, fp, vp, fp, i, fp, vp, fp,
                                              i64, i64, i64, i64, i, u32, vp, i64, vp, i64, vp]
            lib.mss_scan_fwd_save.restype = i
            lib.mss_scan_fwd_workspace_size.argtypes = [i64, i64, i64, i64, i, u32]
            lib.mss_scan_fwd_workspace_size.restype = i64
            lib.mss_state_update.argtypes = [fp, vp, vp, fp, vp, vp, fp, vp, fp, i, vp,
                                             i64, i64, i64, i, vp]
            lib.mss_state_update.restype = i
            lib.mss_state_update_ex.argtypes = [fp, vp, vp, fp, vp, vp, fp, vp, fp, i, vp,
                                                i64, i64, i64, i, u32, vp]
            lib.mss_state_update_ex.restype = i
            lib.mss_scan_bwd.argtypes = [vp, vp, fp, vp, vp, fp, vp, fp, i, fp, vp, fp,
                                         vp, vp, vp, fp, fp, fp, fp, fp, fp, i64, i64, i64, i64, i, u32, vp, i64, vp]
            lib.mss_scan_bwd.restype = i
            lib.mss_scan_bwd_workspace_size.argtypes = [i64, i64, i64, i64, i, u32]
            lib.mss_scan_bwd_workspace_size.restype = i64
            lib.mss_ssd_fwd.argtypes = [vp, vp, fp, vp, vp, fp, vp, fp, i, fp, vp, fp,
                                        i64, i64, i64, i64, i64, i64, i, vp]
            lib.mss_ssd_fwd.restype = i
            lib.mss_ssd_fwd_ex.argtypes = [vp, vp, fp, vp, vp, fp, vp, fp, i, fp, vp, fp,
                                           i64, i64, i64, i64, i64, i64, i, vp, i64, vp]
            lib.mss_ssd_fwd_ex.restype = i
            lib.mss_ssd_fwd_workspace_size.argtypes = [i64, i64, i64, i64, i64, i64]
            lib.mss_ssd_fwd_workspace_size.restype = i64
            lib.mss_ssd_fwd_ex2.argtypes = [vp, vp, fp, vp, vp, fp, vp, fp, i, fp, vp, fp,
                                            i64, i64, i64, i64, i64, i64, i, u32, vp, i64, vp]
            lib.mss_ssd_fwd_ex2.restype = i
            lib.mss_ssd_fwd_workspace_size_ex.argtypes = [i64, i64, i64, i64, i64, i64, u32]
            lib.mss_ssd_fwd_workspace_size_ex.restype = i64
            lib.mss_scan_fwd_conv.argtypes = [vp, fp, fp, i, vp, vp, vp, fp, vp, vp, fp, vp, fp, i, fp, vp, fp,
                                              i64, i64, i64, i64, i, u32, vp, i64, vp]
            lib.mss_scan_fwd_conv.restype = i
            lib.mss_state_update_conv.argtypes = [fp, vp, vp, fp, fp, i, vp, fp, vp, vp, fp, vp, fp, i, vp,
                                                  i64, i64, i64, i, u32, vp]
            lib.mss_state_update_conv.restype = i
            lib.mss_scan_fwd_host.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, i, vp, vp, vp,
                                              i64, i64, i64, i64, i, u32, vp, i64, vp]
            lib.mss_scan_fwd_host.restype = i
            lib.mss_scan_fwd_host_workspace_size.argtypes = [i64, i64, i64, i64, i, i, i, i, i, i]
            lib.mss_scan_fwd_host_workspace_size.restype = i64
            lib.mss_glr_fwd.argtypes = [vp, vp, vp, fp, fp, vp, i64, vp, fp, fp, i64, i64, i64, i64, i, vp]
            lib.mss_glr_fwd.restype = i
            lib.mss_glr_states_size.argtypes = [i64, i64, i64]
            lib.mss_glr_states_size.restype = i64
            lib.mss_glr_bwd.argtypes = [vp, vp, vp, fp, fp, vp, i64, fp, i64, vp, fp, vp, vp, vp, fp, fp,
                                        i64, i64, i64, i, vp, i64, vp]
            lib.mss_glr_bwd.restype = i
            lib.mss_glr_bwd_workspace_size.argtypes = [i64, i64, i64, i]
            lib.mss_glr_bwd_workspace_size.restype = i64
            lib.mss_glr_update.argtypes = [fp, fp, vp, vp, vp, fp, vp, i64, i64, i, vp]
            lib.mss_glr_update.restype = i
            lib.mss_norm_fwd.argtypes = [vp, vp, fp, fp, ctypes.c_float, vp, vp, fp, fp, i64, i64, i, i, u32, vp]
            lib.mss_norm_fwd.restype = i
            lib.mss_norm_bwd.argtypes = [vp, fp, fp, fp, vp, vp, vp, vp, fp, fp, i64, i64, i, i, vp, i64, vp]
            lib.mss_norm_bwd.restype = i
            lib.mss_norm_bwd_workspace_size.argtypes = [i64, i64]
            lib.mss_norm_bwd_workspace_size.restype = i64
            lib.mss_selftest_timeout.argtypes = [i]
            lib.mss_selftest_timeout.restype = i
            lib.mss_get_device_error.argtypes = [vp]
            lib.mss_get_device_error.restype = i
            lib.mss_strerror.argtypes = [i]
            lib.mss_strerror.restype = ctypes.c_char_p
            lib.mss_version.argtypes = []
            lib.mss_version.restype = i
            lib.mss_probe_pipe_rates.argtypes = [ctypes.POINTER(ctypes.c_double), i, vp]
            lib.mss_probe_pipe_rates.restype = i
            _lib = lib
    return _lib


def _strerror(code: int) -> str:
    return load_library().mss_strerror(int(code)).decode()


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _check(t, name, shape, dtype, device, optional=False):
    if t is None:
        if optional:
            return
        raise ValueError(f"{name} is required")
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if t.dtype != dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _io_dtype(t):
    if t.dtype == torch.float32:
        return DTYPE_F32
    if t.dtype == torch.bfloat16:
        return DTYPE_BF16
    raise TypeError(f"unsupported dtype {t.dtype}: use torch.float32 or torch.bfloat16")


def _stream_handle(stream, device):
    s = torch.cuda.current_stream(device) if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def workspace_size(batch, dim, dstate, seqlen, dtype=torch.bfloat16, flags=0, device=None) -> int:
    """Bytes of workspace the forward pass would use to split the sequence
    on `device` (0: no split)."""
    code = DTYPE_BF16 if dtype == torch.bfloat16 else DTYPE_F32
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    with torch.cuda.device(dev):
        n = int(load_library().mss_scan_fwd_workspace_size(batch, dim, dstate, seqlen, code, int(flags)))
    if n < 0:
        raise MssError(n, "mss_scan_fwd_workspace_size")
    return n


def scan_fwd(u, delta, A, B, C, D=None, z=None, delta_bias=None, softplus=True,
             y=None, last_state=None, want_last_state=True, initial_state=None,
             workspace="auto", flags=0, stream=None):
    """Selective-scan forward pass (mss_scan_fwd_ex2).  Returns (y, last_state);
    last_state is None when want_last_state is False and none was given.

    initial_state: [batch, dim, N] float32 state before the first token (None:
    zero).  flags: FLAG_* bits; FLAG_ZOH_INPUT selects the zero-order-hold
    input matrix.  workspace: "auto" (the size the library asks for, allocated from
    PyTorch's caching allocator), None (no sequence split), or a uint8 CUDA
    tensor the call may use."""
    y, last_state, _ = _scan_fwd(u, delta, A, B, C, D, z, delta_bias, softplus, y, last_state, want_last_state,
                                 initial_state, workspace, flags, stream, None)
    return y, last_state


def scan_fwd_save(u, delta, A, B, C, D=None, z=None, delta_bias=None, softplus=True,
                  y=None, last_state=None, want_last_state=True, initial_state=None,
                  workspace="auto", states="auto", flags=0, stream=None):
    """The forward pass of a training step (mss_scan_fwd_save): scan_fwd that
    also stores the states scan_bwd needs.  Returns (y, last_state, states);
    pass `states` to scan_bwd(saved_states=...) with the same inputs and flags.
    states: "auto" (allocated here) or a uint8 CUDA tensor of at least
    bwd_workspace_size(...) bytes.  Raises MssError(ERR_PATH) for calls the
    tiled kernels do not take (then use scan_fwd and scan_bwd without it)."""
    return _scan_fwd(u, delta, A, B, C, D, z, delta_bias, softplus, y, last_state, want_last_state,
                     initial_state, workspace, flags, stream, states)


def _scan_fwd(u, delta, A, B, C, D, z, delta_bias, softplus, y, last_state, want_last_state, initial_state,
              workspace, flags, stream, states):
    if not isinstance(u, torch.Tensor) or u.device.type != "cuda":
        raise ValueError("u must be a CUDA tensor (there is no CPU path)")
    if u.dim() != 3:
        raise ValueError("u must be [batch, dim, L]")
    batch, dim, L = u.shape
    dev, dt = u.device, u.dtype
    code = _io_dtype(u)
    if A.dim() != 2:
        raise ValueError("A must be [dim, N]")
    N = A.shape[1]
    _check(u, "u", (batch, dim, L), dt, dev)
    _check(delta, "delta", (batch, dim, L), dt, dev)
    _check(A, "A", (dim, N), torch.float32, dev)
    _check(B, "B", (batch, N, L), dt, dev)
    _check(C, "C", (batch, N, L), dt, dev)
    _check(D, "D", (dim,), torch.float32, dev, optional=True)
    _check(z, "z", (batch, dim, L), dt, dev, optional=True)
    _check(delta_bias, "delta_bias", (dim,), torch.float32, dev, optional=True)
    _check(initial_state, "initial_state", (batch, dim, N), torch.float32, dev, optional=True)
    if y is None:
        y = torch.empty((batch, dim, L), dtype=dt, device=dev)
    _check(y, "y", (batch, dim, L), dt, dev)
    if last_state is None and want_last_state:
        last_state = torch.empty((batch, dim, N), dtype=torch.float32, device=dev)
    _check(last_state, "last_state", (batch, dim, N), torch.float32, dev, optional=True)
    if isinstance(workspace, str):
        if workspace != "auto":
            raise ValueError("workspace must be 'auto', None or a uint8 CUDA tensor")
        nbytes = workspace_size(batch, dim, N, L, dt, flags, dev)
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=dev) if nbytes > 0 else None
    if workspace is not None:
        _check(workspace, "workspace", (workspace.numel(),), torch.uint8, dev)
    if states is None:
        rc = load_library().mss_scan_fwd_ex2(
            _ptr(u), _ptr(delta), _ptr(A), _ptr(B), _ptr(C), _ptr(D), _ptr(z), _ptr(delta_bias),
            int(bool(softplus)), _ptr(initial_state), _ptr(y), _ptr(last_state), batch, dim, N, L, code,
            int(flags), _ptr(workspace), 0 if workspace is None else workspace.numel(),
            _stream_handle(stream, dev))
        if rc != 0:
            raise MssError(rc, "mss_scan_fwd")
        return y, last_state, None
    if isinstance(states, str):
        if states != "auto":
            raise ValueError("states must be 'auto' or a uint8 CUDA tensor")
        states = torch.empty(max(bwd_workspace_size(batch, dim, N, L, dt, flags), 16), dtype=torch.uint8,
                             device=dev)
    _check(states, "states", (states.numel(),), torch.uint8, dev)
    rc = load_library().mss_scan_fwd_save(
        _ptr(u), _ptr(delta), _ptr(A), _ptr(B), _ptr(C), _ptr(D), _ptr(z), _ptr(delta_bias),
        int(bool(softplus)), _ptr(initial_state), _ptr(y), _ptr(last_state), batch, dim, N, L, code,
        int(flags), _ptr(workspace), 0 if workspace is None else workspace.numel(), _ptr(states),
        states.numel(), _stream_handle(stream, dev))
    if rc != 0:
        raise MssError(rc, "mss_scan_fwd_save")
    return y, last_state, states


def scan_fwd_host(u, delta, A, B, C, D=None, z=None, delta_bias=None, softplus=True,
                  y=None, last_state=None, want_last_state=True, initial_state=None,
                  workspace="auto", flags=0, device=None, stream=None):
    """The forward pass over CPU tensors (mss_scan_fwd_host): the library
    copies the inputs to `device` piece by piece through a device workspace,
    runs the kernels and copies y and last_state back, overlapping the copies
    of different pieces with each other and with the kernels.  Inputs and
    outputs are CPU tensors in the layouts of scan_fwd.  Pinned memory is
    needed for the overlap, and outputs created here are pinned.  The call is
    asynchronous on `stream` (default: the current stream of `device`), so
    the outputs are complete only after that stream has been synchronised.
    Returns (y, last_state)."""
    if not isinstance(u, torch.Tensor) or u.device.type != "cpu":
        raise ValueError("u must be a CPU tensor (scan_fwd takes CUDA tensors)")
    if u.dim() != 3 or A.dim() != 2:
        raise ValueError("u must be [batch, dim, L] and A [dim, N]")
    batch, dim, L = u.shape
    N = A.shape[1]
    cpu, dt = torch.device("cpu"), u.dtype
    code = _io_dtype(u)
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    for t, name, shape, typ, opt in ((u, "u", (batch, dim, L), dt, False), (delta, "delta", (batch, dim, L), dt, False),
                                     (A, "A", (dim, N), torch.float32, False), (B, "B", (batch, N, L), dt, False),
                                     (C, "C", (batch, N, L), dt, False), (D, "D", (dim,), torch.float32, True),
                                     (z, "z", (batch, dim, L), dt, True),
                                     (delta_bias, "delta_bias", (dim,), torch.float32, True),
                                     (initial_state, "initial_state", (batch, dim, N), torch.float32, True)):
        _check(t, name, shape, typ, cpu, optional=opt)
    if y is None:
        y = torch.empty((batch, dim, L), dtype=dt, pin_memory=True)
    _check(y, "y", (batch, dim, L), dt, cpu)
    if last_state is None and want_last_state:
        last_state = torch.empty((batch, dim, N), dtype=torch.float32, pin_memory=True)
    _check(last_state, "last_state", (batch, dim, N), torch.float32, cpu, optional=True)
    lib = load_library()
    with torch.cuda.device(dev):
        if isinstance(workspace, str):
            if workspace != "auto":
                raise ValueError("workspace must be 'auto' or a uint8 CUDA tensor")
            nbytes = int(lib.mss_scan_fwd_host_workspace_size(
                batch, dim, N, L, code, int(z is not None), int(D is not None), int(delta_bias is not None),
                int(initial_state is not None), int(last_state is not None)))
            if nbytes < 0:
                raise MssError(nbytes, "mss_scan_fwd_host_workspace_size")
            workspace = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=dev)
        _check(workspace, "workspace", (workspace.numel(),), torch.uint8, dev)
        rc = lib.mss_scan_fwd_host(
            _ptr(u), _ptr(delta), _ptr(A), _ptr(B), _ptr(C), _ptr(D), _ptr(z), _ptr(delta_bias),
            int(bool(softplus)), _ptr(initial_state), _ptr(y), _ptr(last_state), batch, dim, N, L, code,
            int(flags), _ptr(workspace), workspace.numel(), _stream_handle(stream, dev))
    if rc != 0:
        raise MssError(rc, "mss_scan_fwd_host")
    return y, last_state


def scan_fwd_conv(x, conv_w, delta, A, B, C, conv_b=None, conv_state=None, D=None, z=None,
                  delta_bias=None, softplus=True, y=None, last_state=None, want_last_state=True,
                  conv_state_out=None, want_conv_state=True, initial_state=None, workspace="auto",
                  flags=0, stream=None):
    """Forward pass with the causal convolution and SiLU in front
    (mss_scan_fwd_conv): u = silu(conv_b + causal conv of x with conv_w).
    Returns (y, last_state, conv_state_out); each state is None when not
    wanted and not given.

    x: [batch, dim, L]; conv_w: [dim, K] float32 (K = 1..4); conv_b: [dim]
    float32; conv_state: [batch, dim, K-1] in x's dtype (None: zeros).  Other
    arguments as scan_fwd."""
    if not isinstance(x, torch.Tensor) or x.device.type != "cuda":
        raise ValueError("x must be a CUDA tensor (there is no CPU path)")
    if x.dim() != 3:
        raise ValueError("x must be [batch, dim, L]")
    batch, dim, L = x.shape
    dev, dt = x.device, x.dtype
    code = _io_dtype(x)
    if A.dim() != 2 or conv_w.dim() != 2:
        raise ValueError("A must be [dim, N] and conv_w [dim, K]")
    N, K = A.shape[1], conv_w.shape[1]
    _check(x, "x", (batch, dim, L), dt, dev)
    _check(conv_w, "conv_w", (dim, K), torch.float32, dev)
    _check(conv_b, "conv_b", (dim,), torch.float32, dev, optional=True)
    _check(conv_state, "conv_state", (batch, dim, K - 1), dt, dev, optional=True)
    _check(delta, "delta", (batch, dim, L), dt, dev)
    _check(A, "A", (dim, N), torch.float32, dev)
    _check(B, "B", (batch, N, L), dt, dev)
    _check(C, "C", (batch, N, L), dt, dev)
    _check(D, "D", (dim,), torch.float32, dev, optional=True)
    _check(z, "z", (batch, dim, L), dt, dev, optional=True)
    _check(delta_bias, "delta_bias", (dim,), torch.float32, dev, optional=True)
    _check(initial_state, "initial_state", (batch, dim, N), torch.float32, dev, optional=True)
    if y is None:
        y = torch.empty((batch, dim, L), dtype=dt, device=dev)
    _check(y, "y", (batch, dim, L), dt, dev)
    if last_state is None and want_last_state:
        last_state = torch.empty((batch, dim, N), dtype=torch.float32, device=dev)
    _check(last_state, "last_state", (batch, dim, N), torch.float32, dev, optional=True)
    if conv_state_out is None and want_conv_state:
        conv_state_out = torch.empty((batch, dim, K - 1), dtype=dt, device=dev)
    _check(conv_state_out, "conv_state_out", (batch, dim, K - 1), dt, dev, optional=True)
    if isinstance(workspace, str):
        if workspace != "auto":
            raise ValueError("workspace must be 'auto', None or a uint8 CUDA tensor")
        nbytes = workspace_size(batch, dim, N, L, dt, flags, dev)
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=dev) if nbytes > 0 else None
    if workspace is not None:
        _check(workspace, "workspace", (workspace.numel(),), torch.uint8, dev)
    rc = load_library().mss_scan_fwd_conv(
        _ptr(x), _ptr(conv_w), _ptr(conv_b), int(K), _ptr(conv_state), _ptr(conv_state_out),
        _ptr(delta), _ptr(A), _ptr(B), _ptr(C), _ptr(D), _ptr(z), _ptr(delta_bias), int(bool(softplus)),
        _ptr(initial_state), _ptr(y), _ptr(last_state), batch, dim, N, L, code, int(flags),
        _ptr(workspace), 0 if workspace is None else workspace.numel(), _stream_handle(stream, dev))
    if rc != 0:
        raise MssError(rc, "mss_scan_fwd_conv")
    return y, last_state, conv_state_out


def ssd_fwd(x, dt, A, B, C, D=None, z=None, dt_bias=None, softplus=True, initial_state=None, y=None,
            last_state=None, want_last_state=True, workspace="auto", flags=0, stream=None):
    """Structured-state-space-duality forward pass (mss_ssd_fwd_ex2).  x, z:
    [batch, L, H, P] bf16; dt: [batch, L, H] bf16; A, D, dt_bias: [H]
    float32; B, C: [batch, L, G, N] bf16; initial_state: [batch, H, N, P]
    float32.  workspace: "auto" (what mss_ssd_fwd_workspace_size_ex asks for,
    from PyTorch's allocator: every chunk in parallel where that beats one CTA
    per head -- for N = 128 also only the few pairs past the tcgen05 kernel's
    last full wave -- else nothing), None (one CTA per head walks its chunks)
    or a uint8 CUDA tensor.  flags: 0 (the tcgen05 kernel for N = 128, unless a
    workspace is given and the chunk-parallel passes are faster for so few
    (batch, head) pairs) or SSD_FLAG_WARP_MMA (the warp-level kernels).
    Returns (y, last_state)."""
    if not isinstance(x, torch.Tensor) or x.device.type != "cuda":
        raise ValueError("x must be a CUDA tensor (there is no CPU path)")
    if x.dim() != 4 or B.dim() != 4:
        raise ValueError("x must be [batch, L, H, P] and B [batch, L, G, N]")
    batch, L, H, P = x.shape
    G, N = B.shape[2], B.shape[3]
    dev, dt_ = x.device, x.dtype
    code = _io_dtype(x)
    for t, name, shape, typ, opt in ((x, "x", (batch, L, H, P), dt_, False), (dt, "dt", (batch, L, H), dt_, False),
                                     (A, "A", (H,), torch.float32, False), (B, "B", (batch, L, G, N), dt_, False),
                                     (C, "C", (batch, L, G, N), dt_, False), (D, "D", (H,), torch.float32, True),
                                     (z, "z", (batch, L, H, P), dt_, True),
                                     (dt_bias, "dt_bias", (H,), torch.float32, True),
                                     (initial_state, "initial_state", (batch, H, N, P), torch.float32, True)):
        _check(t, name, shape, typ, dev, optional=opt)
    if y is None:
        y = torch.empty((batch, L, H, P), dtype=dt_, device=dev)
    _check(y, "y", (batch, L, H, P), dt_, dev)
    if last_state is None and want_last_state:
        last_state = torch.empty((batch, H, N, P), dtype=torch.float32, device=dev)
    _check(last_state, "last_state", (batch, H, N, P), torch.float32, dev, optional=True)
    if isinstance(workspace, str):
        if workspace != "auto":
            raise ValueError("workspace must be 'auto', None or a uint8 CUDA tensor")
        nbytes = int(load_library().mss_ssd_fwd_workspace_size_ex(batch, L, H, P, G, N, int(flags)))
        if nbytes < 0:
            raise MssError(nbytes, "mss_ssd_fwd_workspace_size_ex")
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=dev) if nbytes > 0 else None
    if workspace is not None:
        _check(workspace, "workspace", (workspace.numel(),), torch.uint8, dev)
    rc = load_library().mss_ssd_fwd_ex2(
        _ptr(x), _ptr(dt), _ptr(A), _ptr(B), _ptr(C), _ptr(D), _ptr(z), _ptr(dt_bias), int(bool(softplus)),
        _ptr(initial_state), _ptr(y), _ptr(last_state), batch, L, H, P, G, N, code, int(flags), _ptr(workspace),
        0 if workspace is None else workspace.numel(), _stream_handle(stream, dev))
    if rc != 0:
        raise MssError(rc, "mss_ssd_fwd")
    return y, last_state


def bwd_workspace_size(batch, dim, dstate, seqlen, dtype=torch.bfloat16, flags=0) -> int:
    """Bytes of workspace scan_bwd needs (16-byte aligned tensors)."""
    code = DTYPE_BF16 if dtype == torch.bfloat16 else DTYPE_F32
    n = int(load_library().mss_scan_bwd_workspace_size(batch, dim, dstate, seqlen, code, int(flags)))
    if n < 0:
        raise MssError(n, "mss_scan_bwd_workspace_size")
    return n


def scan_bwd(u, delta, A, B, C, dy, D=None, z=None, delta_bias=None, softplus=True, initial_state=None,
             dlast=None, flags=0, workspace="auto", want_dinit=True, out=None, stream=None, saved_states=None):
    """Backward pass of scan_fwd (mss_scan_bwd).  dy: [batch, dim, L] (the io
    dtype), dlast: [batch, dim, N] float32 or None.  Returns a dict with du,
    ddelta, dz (None without z) in the io dtype, dA [dim, N], dB, dC
    [batch, N, L], dD, dbias [dim] and dinit [batch, dim, N] in float32.
    out: optional dict of caller-owned output tensors under those names (the
    rest are allocated).  saved_states: the states scan_fwd_save returned for
    these inputs and flags; the call then skips its checkpoint pass (the
    tensor is its workspace)."""
    if saved_states is not None:
        flags = int(flags) | FLAG_SAVED_STATES
        workspace = saved_states
    if not isinstance(u, torch.Tensor) or u.device.type != "cuda":
        raise ValueError("u must be a CUDA tensor (there is no CPU path)")
    batch, dim, L = u.shape
    dev, dt = u.device, u.dtype
    code = _io_dtype(u)
    N = A.shape[1]
    for t, name, shape, typ, opt in ((u, "u", (batch, dim, L), dt, False), (delta, "delta", (batch, dim, L), dt, False),
                                     (A, "A", (dim, N), torch.float32, False), (B, "B", (batch, N, L), dt, False),
                                     (C, "C", (batch, N, L), dt, False), (dy, "dy", (batch, dim, L), dt, False),
                                     (D, "D", (dim,), torch.float32, True), (z, "z", (batch, dim, L), dt, True),
                                     (delta_bias, "delta_bias", (dim,), torch.float32, True),
                                     (initial_state, "initial_state", (batch, dim, N), torch.float32, True),
                                     (dlast, "dlast", (batch, dim, N), torch.float32, True)):
        _check(t, name, shape, typ, dev, optional=opt)
    f32 = dict(dtype=torch.float32, device=dev)
    ret = dict(du=torch.empty((batch, dim, L), dtype=dt, device=dev),
               ddelta=torch.empty((batch, dim, L), dtype=dt, device=dev),
               dz=torch.empty((batch, dim, L), dtype=dt, device=dev) if z is not None else None,
               dA=torch.empty((dim, N), **f32), dB=torch.empty((batch, N, L), **f32),
               dC=torch.empty((batch, N, L), **f32), dD=torch.empty((dim,), **f32),
               dbias=torch.empty((dim,), **f32),
               dinit=torch.empty((batch, dim, N), **f32) if want_dinit else None)
    for k, t in (out or {}).items():
        if k not in ret or ret[k] is None:
            raise ValueError(f"out[{k!r}]: no such output here")
        _check(t, k, tuple(ret[k].shape), ret[k].dtype, dev)
        ret[k] = t
    if isinstance(workspace, str):
        if workspace != "auto":
            raise ValueError("workspace must be 'auto', None or a uint8 CUDA tensor")
        nbytes = bwd_workspace_size(batch, dim, N, L, dt, flags)
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=dev) if nbytes > 0 else None
    if workspace is not None:
        _check(workspace, "workspace", (workspace.numel(),), torch.uint8, dev)
    rc = load_library().mss_scan_bwd(
        _ptr(u), _ptr(delta), _ptr(A), _ptr(B), _ptr(C), _ptr(D), _ptr(z), _ptr(delta_bias), int(bool(softplus)),
        _ptr(initial_state), _ptr(dy), _ptr(dlast), _ptr(ret["du"]), _ptr(ret["ddelta"]), _ptr(ret["dz"]),
        _ptr(ret["dA"]), _ptr(ret["dB"]), _ptr(ret["dC"]), _ptr(ret["dD"]), _ptr(ret["dbias"]), _ptr(ret["dinit"]),
        batch, dim, N, L, code, int(flags), _ptr(workspace), 0 if workspace is None else workspace.numel(),
        _stream_handle(stream, dev))
    if rc != 0:
        raise MssError(rc, "mss_scan_bwd")
    return ret


def state_update_conv(state, conv_state, x, conv_w, delta, A, B, C, conv_b=None, D=None, z=None,
                      delta_bias=None, softplus=True, y=None, flags=0, stream=None):
    """One decode token with the causal convolution in front
    (mss_state_update_conv); `state` and `conv_state` ([batch, dim, K-1] in
    x's dtype, None when K = 1) are updated in place.  Returns y [batch, dim]."""
    if not isinstance(state, torch.Tensor) or state.device.type != "cuda":
        raise ValueError("state must be a CUDA tensor (there is no CPU path)")
    if state.dim() != 3:
        raise ValueError("state must be [batch, dim, N]")
    batch, dim, N = state.shape
    dev, dt = state.device, x.dtype
    code = _io_dtype(x)
    if conv_w.dim() != 2:
        raise ValueError("conv_w must be [dim, K]")
    K = conv_w.shape[1]
    _check(state, "state", (batch, dim, N), torch.float32, dev)
    _check(conv_state, "conv_state", (batch, dim, K - 1), dt, dev, optional=K == 1)
    _check(x, "x", (batch, dim), dt, dev)
    _check(conv_w, "conv_w", (dim, K), torch.float32, dev)
    _check(conv_b, "conv_b", (dim,), torch.float32, dev, optional=True)
    _check(delta, "delta", (batch, dim), dt, dev)
    _check(A, "A", (dim, N), torch.float32, dev)
    _check(B, "B", (batch, N), dt, dev)
    _check(C, "C", (batch, N), dt, dev)
    _check(D, "D", (dim,), torch.float32, dev, optional=True)
    _check(z, "z", (batch, dim), dt, dev, optional=True)
    _check(delta_bias, "delta_bias", (dim,), torch.float32, dev, optional=True)
    if y is None:
        y = torch.empty((batch, dim), dtype=dt, device=dev)
    _check(y, "y", (batch, dim), dt, dev)
    rc = load_library().mss_state_update_conv(
        _ptr(state), _ptr(conv_state), _ptr(x), _ptr(conv_w), _ptr(conv_b), int(K), _ptr(delta), _ptr(A),
        _ptr(B), _ptr(C), _ptr(D), _ptr(z), _ptr(delta_bias), int(bool(softplus)), _ptr(y), batch, dim, N,
        code, int(flags), _stream_handle(stream, dev))
    if rc != 0:
        raise MssError(rc, "mss_state_update_conv")
    return y


def state_update(state, u, delta, A, B, C, D=None, z=None, delta_bias=None, softplus=True,
                 y=None, flags=0, stream=None):
    """One decode token (mss_state_update_ex); `state` is updated in place.
    Returns y [batch, dim].  flags: 0 or FLAG_ZOH_INPUT."""
    if not isinstance(state, torch.Tensor) or state.device.type != "cuda":
        raise ValueError("state must be a CUDA tensor (there is no CPU path)")
    if state.dim() != 3:
        raise ValueError("state must be [batch, dim, N]")
    batch, dim, N = state.shape
    dev, dt = state.device, u.dtype
    code = _io_dtype(u)
    _check(state, "state", (batch, dim, N), torch.float32, dev)
    _check(u, "u", (batch, dim), dt, dev)
    _check(delta, "delta", (batch, dim), dt, dev)
    _check(A, "A", (dim, N), torch.float32, dev)
    _check(B, "B", (batch, N), dt, dev)
    _check(C, "C", (batch, N), dt, dev)
    _check(D, "D", (dim,), torch.float32, dev, optional=True)
    _check(z, "z", (batch, dim), dt, dev, optional=True)
    _check(delta_bias, "delta_bias", (dim,), torch.float32, dev, optional=True)
    if y is None:
        y = torch.empty((batch, dim), dtype=dt, device=dev)
    _check(y, "y", (batch, dim), dt, dev)
    rc = load_library().mss_state_update_ex(
        _ptr(state), _ptr(u), _ptr(delta), _ptr(A), _ptr(B), _ptr(C), _ptr(D), _ptr(z),
        _ptr(delta_bias), int(bool(softplus)), _ptr(y), batch, dim, N, code, int(flags),
        _stream_handle(stream, dev))
    if rc != 0:
        raise MssError(rc, "mss_state_update")
    return y


def _addr(t):
    return t.data_ptr() if t is not None else None


def _expect(t, name, shape, dtype, device):
    """_check of a required tensor; the usual case costs one expression."""
    try:
        if t.dtype is dtype and t.shape == shape and t.device == device and t.is_contiguous():
            return
    except AttributeError:
        pass
    _check(t, name, shape, dtype, device)


def _new(like, shape, dtype, stream):
    """An output or workspace on the device of `like` for a call on `stream`:
    allocated there, so that the allocator hands its memory on only in that
    stream's order."""
    if stream is None:
        if dtype is like.dtype and shape == like.shape:
            return torch.empty_like(like)
        return like.new_empty(shape, dtype=dtype)
    with torch.cuda.stream(stream):
        return like.new_empty(shape, dtype=dtype)


_raw_stream = torch._C._cuda_getCurrentRawStream if hasattr(torch._C, "_cuda_getCurrentRawStream") else (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _on_device(device, stream, name, *args):
    """The library's function `name` on these arguments and the stream's
    handle, with `device` current; raises for a status other than 0."""
    fn = getattr(_lib or load_library(), name)
    if device.index == torch.cuda.current_device():
        rc = fn(*args, _raw_stream(device.index) if stream is None else stream.cuda_stream)
    else:
        with torch.cuda.device(device):
            rc = fn(*args, _raw_stream(device.index) if stream is None else stream.cuda_stream)
    if rc != 0:
        raise MssError(rc, name)


def _cuda_input(t, name, dims, layout):
    if not isinstance(t, torch.Tensor) or t.device.type != "cuda":
        raise ValueError(f"{name} must be a CUDA tensor (there is no CPU path)")
    if t.dim() != dims:
        raise ValueError(f"{name} must be {layout}")


def _glr_checks(x, gate, z, gate_bias, initial_state, seq_offsets):
    """Shared checks of the recurrence's calls over sequences: (batch, L, dim,
    number of states, sequences)."""
    _cuda_input(x, "x", 3, "[batch, L, dim]")
    shape, dt, dev = x.shape, x.dtype, x.device
    batch, L, dim = shape
    if not x.is_contiguous():
        _expect(x, "x", shape, dt, dev)
    _expect(gate, "gate", shape, dt, dev)
    if z is not None:
        _expect(z, "z", shape, dt, dev)
    if gate_bias is not None:
        _expect(gate_bias, "gate_bias", (dim,), torch.float32, dev)
    nseq, states = 0, batch
    if seq_offsets is not None:
        if batch != 1 or not isinstance(seq_offsets, torch.Tensor) or seq_offsets.dim() != 1 or seq_offsets.numel() < 1:
            raise ValueError("seq_offsets must be a tensor [nseq + 1] and x [1, tokens, dim]")
        nseq = states = seq_offsets.numel() - 1
        _expect(seq_offsets, "seq_offsets", (nseq + 1,), torch.int32, dev)
    if initial_state is not None:
        _expect(initial_state, "initial_state", (states, dim), torch.float32, dev)
    return batch, L, dim, states, nseq


def glr_fwd(x, gate, z=None, gate_bias=None, initial_state=None, seq_offsets=None, y=None, last_state=None,
            want_last_state=True, stream=None):
    """Gated linear recurrence (mss_glr_fwd): with f = sigmoid(gate + gate_bias),
    h_t = f_t h_{t-1} + (1 - f_t) x_t and y_t = h_t silu(z_t).  Returns
    (y, last_state); last_state is None when want_last_state is False and none
    was given.

    x, gate, z: [batch, L, dim], float32 or bfloat16; gate_bias: [dim] float32;
    initial_state, last_state: [batch, dim] float32.  seq_offsets: packed
    sequences, int32 [nseq + 1] on the GPU with x [1, tokens, dim] -- sequence
    i is tokens seq_offsets[i] .. seq_offsets[i+1] - 1, the states are [nseq, dim],
    and rows of y outside the sequences are left as they were (unwritten when y
    is allocated here)."""
    return _glr_fwd(x, gate, z, gate_bias, initial_state, seq_offsets, y, last_state, want_last_state, None, stream)[:2]


def glr_fwd_save(x, gate, z=None, gate_bias=None, initial_state=None, seq_offsets=None, y=None, last_state=None,
                 want_last_state=True, states="auto", stream=None):
    """glr_fwd of a training step: also stores the state before every 64th
    token.  Returns (y, last_state, states); pass `states` to
    glr_bwd(saved_states=...).  states: "auto" (allocated here) or a float32
    CUDA tensor of [batch, ceil(L / 64), dim]."""
    return _glr_fwd(x, gate, z, gate_bias, initial_state, seq_offsets, y, last_state, want_last_state, states, stream)


def _glr_fwd(x, gate, z, gate_bias, initial_state, seq_offsets, y, last_state, want_last_state, states, stream,
             want_y=True):
    batch, L, dim, nstates, nseq = _glr_checks(x, gate, z, gate_bias, initial_state, seq_offsets)
    dt, dev = x.dtype, x.device
    code = _io_dtype(x)
    if y is not None:
        _expect(y, "y", (batch, L, dim), dt, dev)
    elif want_y:
        y = _new(x, (batch, L, dim), dt, stream)
    if last_state is not None:
        _expect(last_state, "last_state", (nstates, dim), torch.float32, dev)
    elif want_last_state:
        last_state = _new(x, (nstates, dim), torch.float32, stream)
    if states is not None:
        saved = (batch, (L + 63) // 64, dim)
        if isinstance(states, str):
            if states != "auto":
                raise ValueError("states must be 'auto' or a float32 CUDA tensor")
            states = _new(x, saved, torch.float32, stream)
        _expect(states, "states", saved, torch.float32, dev)
    _on_device(dev, stream, "mss_glr_fwd", _addr(x), _addr(gate), _addr(z), _addr(gate_bias),
               _addr(initial_state), _addr(seq_offsets), nseq, _addr(y), _addr(last_state), _addr(states),
               0 if states is None else states.numel() * 4, batch, L, dim, code)
    return y, last_state, states


def glr_bwd(x, gate, dy, z=None, gate_bias=None, initial_state=None, seq_offsets=None, dlast=None,
            saved_states=None, want_dbias=True, want_dinit=True, out=None, workspace="auto", stream=None):
    """Backward pass of glr_fwd (mss_glr_bwd).  dy: as x; dlast: as last_state,
    or None.  Returns a dict with dx, dgate, dz (None without z) as x, dbias
    [dim] and dinit (as initial_state) in float32, None where not wanted.
    saved_states: what glr_fwd_save returned for these inputs; without it a
    forward pass that writes only these states runs first.  out: optional
    dict of caller-owned output tensors under those names (with seq_offsets their
    rows outside the sequences are left as they were).  workspace: "auto" or a
    uint8 CUDA tensor of at least glr_bwd_workspace_size(...) bytes."""
    batch, L, dim, nstates, nseq = _glr_checks(x, gate, z, gate_bias, initial_state, seq_offsets)
    dt, dev = x.dtype, x.device
    code = _io_dtype(x)
    _expect(dy, "dy", (batch, L, dim), dt, dev)
    if dlast is not None:
        _expect(dlast, "dlast", (nstates, dim), torch.float32, dev)
    shape, f32 = x.shape, torch.float32
    ret = _outputs(out, x, stream, ("dx", shape, dt), ("dgate", shape, dt), ("dz", shape if z is not None else None, dt),
                   ("dbias", (dim,) if want_dbias else None, f32), ("dinit", (nstates, dim) if want_dinit else None, f32))
    if saved_states is None:
        saved_states = _glr_fwd(x, gate, None, gate_bias, initial_state, seq_offsets, None, None, False, "auto",
                                stream, want_y=False)[2]
    else:
        _expect(saved_states, "saved_states", (batch, (L + 63) // 64, dim), torch.float32, dev)
    if isinstance(workspace, str):
        if workspace != "auto":
            raise ValueError("workspace must be 'auto', None or a uint8 CUDA tensor")
        nbytes = glr_bwd_workspace_size(batch, L, dim, dt) if want_dbias else 0
        workspace = _new(x, (nbytes,), torch.uint8, stream) if nbytes > 0 else None
    if workspace is not None:
        _expect(workspace, "workspace", (workspace.numel(),), torch.uint8, dev)
    _on_device(dev, stream, "mss_glr_bwd", _addr(x), _addr(gate), _addr(z), _addr(gate_bias),
               _addr(initial_state), _addr(seq_offsets), nseq, _addr(saved_states), saved_states.numel() * 4,
               _addr(dy), _addr(dlast), _addr(ret["dx"]), _addr(ret["dgate"]), _addr(ret["dz"]),
               _addr(ret["dbias"]), _addr(ret["dinit"]), batch, L, dim, code, _addr(workspace),
               0 if workspace is None else workspace.numel())
    return ret


def _outputs(out, like, stream, *wanted):
    """The output tensors of a backward pass by name: `wanted` are (name, shape or
    None, dtype), `out` holds the caller's own."""
    ret = {}
    for name, shape, dtype in wanted:
        if out and name in out and shape is not None:
            _expect(out[name], name, shape, dtype, like.device)
            ret[name] = out[name]
        else:
            ret[name] = None if shape is None else _new(like, shape, dtype, stream)
    for name in out or ():
        if ret.get(name) is None:
            raise ValueError(f"out[{name!r}]: no such output here")
    return ret


@functools.lru_cache(maxsize=256)
def _size(query, *sizes):
    """A size query of the library that depends on nothing but its arguments."""
    n = int(getattr(load_library(), query)(*sizes))
    if n < 0:
        raise MssError(n, query)
    return n


def glr_bwd_workspace_size(batch, seqlen, dim, dtype=torch.bfloat16) -> int:
    """Bytes of workspace glr_bwd needs for dbias (0: none)."""
    return _size("mss_glr_bwd_workspace_size", batch, seqlen, dim, DTYPE_BF16 if dtype == torch.bfloat16 else DTYPE_F32)


def glr_update(state, x, gate, z=None, gate_bias=None, y=None, state_out=None, stream=None):
    """One decode token of the gated linear recurrence (mss_glr_update).
    state: [batch, dim] float32, updated in place, or read only when state_out
    is given; x, gate, z: [batch, dim].  Returns y [batch, dim]."""
    _cuda_input(state, "state", 2, "[batch, dim]")
    shape, dev = state.shape, state.device
    if state.dtype is not torch.float32 or not state.is_contiguous():
        _expect(state, "state", shape, torch.float32, dev)
    if not isinstance(x, torch.Tensor):
        raise TypeError("x must be a torch.Tensor")
    dt = x.dtype
    code = _io_dtype(x)
    _expect(x, "x", shape, dt, dev)
    _expect(gate, "gate", shape, dt, dev)
    if z is not None:
        _expect(z, "z", shape, dt, dev)
    if gate_bias is not None:
        _expect(gate_bias, "gate_bias", shape[1:], torch.float32, dev)
    if state_out is not None:
        _expect(state_out, "state_out", shape, torch.float32, dev)
    if y is None:
        y = _new(x, shape, dt, stream)
    else:
        _expect(y, "y", shape, dt, dev)
    _on_device(dev, stream, "mss_glr_update", _addr(state), _addr(state_out), _addr(x), _addr(gate),
               _addr(z), _addr(gate_bias), _addr(y), shape[0], shape[1], code)
    return y


def norm_fwd(x, weight, bias=None, residual=None, eps=1e-5, rms=False, y=None, residual_out=None, want_stats=True,
             stream=None):
    """Residual add and layer norm (mss_norm_fwd): s = x + residual, y = the
    norm of s over the last dimension.  Returns (y, s, mean, rstd): s is None
    without residual and residual_out, mean None with rms=True (the
    root-mean-square form), mean and rstd None with want_stats=False.

    x: [..., dim] float32 or bfloat16; weight, bias: [dim] float32; residual,
    residual_out: [..., dim] float32 or x's type; mean, rstd: [...] float32 (NaN
    for rows without elements).  No output may be an input's memory, residual_out
    not residual's either."""
    if not isinstance(x, torch.Tensor) or x.device.type != "cuda":
        raise ValueError("x must be a CUDA tensor (there is no CPU path)")
    if x.dim() < 1:
        raise ValueError("x must be [..., dim]")
    shape, dt, dev = x.shape, x.dtype, x.device
    dim = shape[-1]
    rows = x.numel() // dim if dim else 0
    code = _io_dtype(x)
    if not x.is_contiguous():
        _expect(x, "x", shape, dt, dev)
    _expect(weight, "weight", (dim,), torch.float32, dev)
    if bias is not None:
        _expect(bias, "bias", (dim,), torch.float32, dev)
    rdt = residual.dtype if isinstance(residual, torch.Tensor) else dt
    if residual is not None:
        _expect(residual, "residual", shape, torch.float32 if rdt == torch.float32 else dt, dev)
    if residual_out is not None:
        if residual is None and isinstance(residual_out, torch.Tensor):
            rdt = torch.float32 if residual_out.dtype == torch.float32 else dt
        _expect(residual_out, "residual_out", shape, rdt, dev)
    elif residual is not None:
        residual_out = _new(x, shape, rdt, stream)
    if y is None:
        y = _new(x, shape, dt, stream)
    else:
        _expect(y, "y", shape, dt, dev)
    mean = _new(x, shape[:-1], torch.float32, stream) if want_stats and not rms else None
    rstd = _new(x, shape[:-1], torch.float32, stream) if want_stats else None
    _on_device(dev, stream, "mss_norm_fwd", _addr(x), _addr(residual), _addr(weight), _addr(bias),
               float(eps), _addr(y), _addr(residual_out), _addr(mean), _addr(rstd), rows, dim, code,
               DTYPE_F32 if rdt == torch.float32 else DTYPE_BF16, NORM_FLAG_RMS if rms else 0)
    if dim == 0 and want_stats:  # 0 / 0: the library writes nothing for rows without elements
        with torch.cuda.stream(stream):
            for v in (mean, rstd):
                if v is not None:
                    v.fill_(float("nan"))
    return y, residual_out, mean, rstd


def norm_bwd(s, weight, dy, rstd, mean=None, dresidual=None, want_dx=True, want_dweight=True, want_dbias=True,
             out=None, workspace="auto", stream=None):
    """Backward pass of norm_fwd (mss_norm_bwd).  s: the normalised input, i.e.
    norm_fwd's s, or its x when there was no residual; mean, rstd: as norm_fwd
    returned them (mean None: the root-mean-square form); dy: [..., dim];
    dresidual: the gradient of s from the layers above, in s's type.  Returns a
    dict: dx in dy's type (the gradient of norm_fwd's x), dresidual in s's type
    (the gradient of its residual; None when s has dy's type, where dx is both),
    dweight and dbias [dim] float32; None where not wanted.  out: optional dict
    of caller-owned output tensors under those names."""
    if not isinstance(s, torch.Tensor) or s.device.type != "cuda":
        raise ValueError("s must be a CUDA tensor (there is no CPU path)")
    if s.dim() < 1:
        raise ValueError("s must be [..., dim]")
    if not isinstance(dy, torch.Tensor):
        raise TypeError("dy must be a torch.Tensor")
    shape, dt, sdt, dev = s.shape, dy.dtype, s.dtype, s.device
    dim = shape[-1]
    rows = s.numel() // dim if dim else 0
    code, scode = _io_dtype(dy), _io_dtype(s)
    if not s.is_contiguous():
        _expect(s, "s", shape, sdt, dev)
    _expect(dy, "dy", shape, dt, dev)
    _expect(weight, "weight", (dim,), torch.float32, dev)
    _expect(rstd, "rstd", shape[:-1], torch.float32, dev)
    if mean is not None:
        _expect(mean, "mean", shape[:-1], torch.float32, dev)
    if dresidual is not None:
        _expect(dresidual, "dresidual", shape, sdt, dev)
    f32 = torch.float32
    ret = _outputs(out, s, stream, ("dx", shape if want_dx or sdt == dt else None, dt),
                   ("dresidual", shape if sdt != dt else None, sdt), ("dweight", (dim,) if want_dweight else None, f32),
                   ("dbias", (dim,) if want_dbias else None, f32))
    if isinstance(workspace, str):
        if workspace != "auto":
            raise ValueError("workspace must be 'auto', None or a uint8 CUDA tensor")
        nbytes = norm_bwd_workspace_size(rows, dim) if want_dweight or want_dbias else 0
        workspace = _new(s, (nbytes,), torch.uint8, stream) if nbytes > 0 else None
    if workspace is not None:
        _expect(workspace, "workspace", (workspace.numel(),), torch.uint8, dev)
    _on_device(dev, stream, "mss_norm_bwd", _addr(s), _addr(weight), _addr(mean), _addr(rstd), _addr(dy),
               _addr(dresidual), _addr(ret["dx"]), _addr(ret["dresidual"]), _addr(ret["dweight"]),
               _addr(ret["dbias"]), rows, dim, code, scode, _addr(workspace),
               0 if workspace is None else workspace.numel())
    return ret


def norm_bwd_workspace_size(rows, dim) -> int:
    """Bytes of workspace norm_bwd needs for dweight and dbias."""
    return _size("mss_norm_bwd_workspace_size", rows, dim)


PIPE_RATE_NAMES = ("ffma", "ffma2", "mufu_ex2", "shfl")


def probe_pipe_rates(stream=None, device=None) -> dict:
    """Measured throughput of the fp32 fma pipe (scalar and packed, lane
    operations), the multi-function unit (ex2 results) and warp shuffles
    (results), per SM and SM clock cycle, on the current device
    (mss_probe_pipe_rates)."""
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else device
    out = (ctypes.c_double * len(PIPE_RATE_NAMES))()
    rc = load_library().mss_probe_pipe_rates(out, len(PIPE_RATE_NAMES), _stream_handle(stream, dev))
    if rc != 0:
        raise MssError(rc, "mss_probe_pipe_rates")
    return {k: float(v) for k, v in zip(PIPE_RATE_NAMES, out)}


def selftest_timeout(on: bool) -> bool:
    """Self-test of the bounded waits of the recurrence and the norm
    (mss_selftest_timeout): while on, this thread's calls give up waiting after
    1 ms and set the device error status; their outputs are then unspecified.
    Returns the setting before."""
    return bool(load_library().mss_selftest_timeout(1 if on else 0))


def get_device_error(stream=None, device=None) -> int:
    """Synchronise the stream and return (and clear) the library's device
    error status: 0, or a negative mss_status code (ERR_DEVICE_TIMEOUT before
    ERR_OFFSETS, one a call)."""
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else device
    return int(load_library().mss_get_device_error(_stream_handle(stream, dev)))
