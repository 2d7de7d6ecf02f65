"""Python binding of libgka.so: argument marshalling only.

Every step of the layer runs in the library's CUDA kernels; this module checks
tensor shapes, dtypes and devices, hands raw device pointers and the current
CUDA stream to the C ABI (include/gka.h) and raises on a non-zero status.
There is no fallback: if the library is missing or a call fails, it raises.
"""
from __future__ import annotations

import ctypes
import functools
import struct
from pathlib import Path

import torch

_PKG = Path(__file__).resolve().parent
LIB_PATH = _PKG / "libgka.so"

GKA_F32, GKA_BF16 = 0, 1
_DT = {torch.float32: GKA_F32, torch.bfloat16: GKA_BF16}


class GkaError(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        msg = _lib().gka_status_string(status).decode()
        if status == -5:
            msg += f" (cudaError {_lib().gka_last_cuda_error()})"
        super().__init__(f"{fn}: {msg} [{status}]")


KERNEL_NAMES = ["chunk_delta", "state_scan", "chunk_norm", "chunk_solve", "decode_step",
                "chunk_solve_tc", "state_pass_tc", "bwd_solve", "bwd_delta", "adjoint_scan",
                "bwd_rows", "bwd_grads", "solver_study", "linear", "linear_grad", "block_rows"]
_KERNEL_COUNT = 16


class KernelTimes(ctypes.Structure):
    _fields_ = [("ms", ctypes.c_double * _KERNEL_COUNT), ("launches", ctypes.c_int * _KERNEL_COUNT)]


class WorkspaceLayout(ctypes.Structure):
    _fields_ = [("states_offset", ctypes.c_size_t), ("decay_offset", ctypes.c_size_t),
                ("norms_offset", ctypes.c_size_t), ("states_lp_offset", ctypes.c_size_t),
                ("total_bytes", ctypes.c_size_t)]


_L = None


def _lib():
    global _L
    if _L is None:
        if not LIB_PATH.exists():
            raise ImportError(f"{LIB_PATH} is missing: build it with "
                              "`python -m test_ridge_regression_b200.build`")
        lib = ctypes.CDLL(str(LIB_PATH))
        vp, i, f, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
        lib.gka_forward_workspace_bytes.argtypes = [i, i, i, i, i, i]
        lib.gka_forward_workspace_bytes.restype = sz
        lib.gka_forward_workspace_layout.argtypes = [i, i, i, i, i, i, ctypes.POINTER(WorkspaceLayout)]
        lib.gka_forward_workspace_layout.restype = i
        lib.gka_forward.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, f, i, i, vp, vp, sz, vp]
        lib.gka_forward.restype = i
        lib.gka_forward_gated.argtypes = [vp, vp, vp, vp, vp, vp, i, i, i, i, i, f, i, i, vp, vp,
                                          sz, vp]
        lib.gka_forward_gated.restype = i
        lib.gka_forward_static_scratch.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, f, i, i,
                                                   vp, vp]
        lib.gka_forward_host_workspace_bytes.argtypes = [i, i, i, i, i, i, i]
        lib.gka_forward_host_workspace_bytes.restype = sz
        lib.gka_forward_host.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, f, i, i, vp, i, vp,
                                         sz, vp]
        lib.gka_forward_host.restype = i
        lib.gka_forward_static_scratch.restype = i
        lib.gka_decode_step.argtypes = [vp, vp, vp, vp, vp, vp, i, i, i, i, f, i, vp]
        lib.gka_decode_step.restype = i
        lib.gka_decode_step_gated.argtypes = [vp, vp, vp, vp, vp, vp, vp, i, i, i, i, f, i, vp]
        lib.gka_decode_step_gated.restype = i
        lib.gka_backward_workspace_bytes.argtypes = [i, i, i, i, i, i]
        lib.gka_backward_workspace_bytes.restype = sz
        lib.gka_backward.argtypes = [vp] * 11 + [i, i, i, i, i, f, i, i, vp, sz, vp]
        lib.gka_backward.restype = i
        lib.gka_solver_study_workspace_bytes.argtypes = [i, i, i, i, i, i]
        lib.gka_solver_study_workspace_bytes.restype = sz
        lib.gka_solver_study.argtypes = [vp, vp, vp, vp, i, i, i, i, i, f, i, i, i, vp, vp, sz, vp]
        lib.gka_solver_study.restype = i
        for n in ("forward", "backward"):
            fn = getattr(lib, f"gka_linear_{n}_workspace_bytes")
            fn.argtypes, fn.restype = [i] * 5, sz
        lib.gka_linear_forward.argtypes = [vp] * 6 + [i] * 5 + [f, vp, vp, vp, sz, vp]
        lib.gka_linear_forward.restype = i
        lib.gka_linear_backward.argtypes = [vp] * 14 + [i] * 5 + [f, vp, sz, vp]
        lib.gka_linear_backward.restype = i
        lib.gka_linear_decode_step.argtypes = [vp] * 7 + [i] * 4 + [f, vp]
        lib.gka_linear_decode_step.restype = i
        rows = vp   # const gka_strided *: packed by _strided
        lib.gka_block_in_forward.argtypes = [rows] * 5 + [vp] * 8 + [i] * 6 + [f, vp]
        lib.gka_block_in_forward.restype = i
        lib.gka_block_in_backward_workspace_bytes.argtypes = [i] * 6
        lib.gka_block_in_backward_workspace_bytes.restype = sz
        lib.gka_block_in_backward.argtypes = [rows] * 4 + [vp] * 15 + [i] * 6 + [f, vp, sz, vp]
        lib.gka_block_in_backward.restype = i
        lib.gka_block_out_forward.argtypes = [vp, vp, rows, vp, vp, vp] + [i] * 5 + [f, vp]
        lib.gka_block_out_forward.restype = i
        lib.gka_block_out_backward_workspace_bytes.argtypes = [i] * 5
        lib.gka_block_out_backward_workspace_bytes.restype = sz
        lib.gka_block_out_backward.argtypes = ([vp, vp, rows] + [vp] * 8 + [i] * 5 +
                                               [f, vp, sz, vp])
        lib.gka_block_out_backward.restype = i
        lib.gka_selftest_timeout.argtypes = [vp]
        lib.gka_selftest_timeout.restype = i
        lib.gka_device_status.argtypes = [vp]
        lib.gka_device_status.restype = i
        lib.gka_last_cuda_error.argtypes = []
        lib.gka_last_cuda_error.restype = i
        lib.gka_status_string.argtypes = [i]
        lib.gka_status_string.restype = ctypes.c_char_p
        lib.gka_version.argtypes = []
        lib.gka_version.restype = i
        lib.gka_profiler_enable.argtypes = [i]
        lib.gka_profiler_enable.restype = i
        lib.gka_profiler_read.argtypes = [ctypes.POINTER(KernelTimes)]
        lib.gka_profiler_read.restype = i
        _L = lib
    return _L


def lib():
    """The loaded ctypes library (raises ImportError if it was not built)."""
    return _lib()


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _check(fn, rc):
    if rc != 0:
        raise GkaError(fn, rc)


def _dtype(t: torch.Tensor) -> int:
    if t.dtype not in _DT:
        raise TypeError(f"unsupported dtype {t.dtype}; use float32 or bfloat16")
    return _DT[t.dtype]


def _dev(*ts):
    for t in ts:
        if t is not None and (not t.is_cuda or not t.is_contiguous()):
            raise ValueError("tensors must be contiguous CUDA tensors")


def workspace_bytes(B, H, T, D, chunk, dtype=torch.bfloat16) -> int:
    return int(_lib().gka_forward_workspace_bytes(B, H, T, D, chunk, _DT[dtype]))


def workspace_layout(B, H, T, D, chunk, dtype=torch.bfloat16) -> WorkspaceLayout:
    out = WorkspaceLayout()
    _check("gka_forward_workspace_layout",
           _lib().gka_forward_workspace_layout(B, H, T, D, chunk, _DT[dtype], ctypes.byref(out)))
    return out


def alloc_workspace(B, H, T, D, chunk, dtype=torch.bfloat16, device=None) -> torch.Tensor:
    n = workspace_bytes(B, H, T, D, chunk, dtype)
    return torch.empty(max(n, 256), dtype=torch.uint8, device=device or "cuda")


def gka_forward(q, k, v, beta, a: float, r: int, chunk: int, *, o=None, final_state=None,
                workspace=None, stream=None):
    """Chunk-wise GKA forward (see include/gka.h).  q, k, v: [B, H, T, D] fp32 or
    bf16 CUDA tensors; beta: [B, H, T] fp32.  Returns o (same shape/dtype as v)."""
    _dev(q, k, v, beta, o, final_state, workspace)
    B, H, T, D = q.shape
    if k.shape != q.shape or v.shape != q.shape or beta.shape != (B, H, T):
        raise ValueError("shape mismatch")
    dt = _dtype(q)
    if k.dtype != q.dtype or v.dtype != q.dtype or beta.dtype != torch.float32:
        raise TypeError("q, k, v must share a dtype; beta must be float32")
    if o is None:
        o = torch.empty_like(v)
    if final_state is not None and (final_state.dtype != torch.float32 or
                                    final_state.shape != (B, H, 2, D, D)):
        raise ValueError("final_state must be float32 [B, H, 2, D, D]")
    if workspace is None:
        workspace = alloc_workspace(B, H, T, D, chunk, q.dtype, q.device)
    rc = _lib().gka_forward(_ptr(q), _ptr(k), _ptr(v), _ptr(beta), _ptr(o), B, H, T, D, dt,
                            float(a), int(r), int(chunk), _ptr(final_state), _ptr(workspace),
                            workspace.numel() * workspace.element_size(), _stream(stream))
    _check("gka_forward", rc)
    return o


def gka_forward_gated(q, k, v, beta, gate, a: float, r: int, chunk: int, *, o=None,
                      final_state=None, workspace=None, stream=None):
    """Write-gated forward (see include/gka.h): as gka_forward, with gate [B, H, T]
    fp32 in [0, 1] scaling each token's write into H and M (None: no gate)."""
    _dev(q, k, v, beta, gate, o, final_state, workspace)
    B, H, T, D = q.shape
    if k.shape != q.shape or v.shape != q.shape or beta.shape != (B, H, T):
        raise ValueError("shape mismatch")
    if gate is not None and (gate.shape != (B, H, T) or gate.dtype != torch.float32):
        raise ValueError("gate must be float32 [B, H, T]")
    dt = _dtype(q)
    if k.dtype != q.dtype or v.dtype != q.dtype or beta.dtype != torch.float32:
        raise TypeError("q, k, v must share a dtype; beta must be float32")
    if o is None:
        o = torch.empty_like(v)
    if final_state is not None and (final_state.dtype != torch.float32 or
                                    final_state.shape != (B, H, 2, D, D)):
        raise ValueError("final_state must be float32 [B, H, 2, D, D]")
    if workspace is None:
        workspace = alloc_workspace(B, H, T, D, chunk, q.dtype, q.device)
    rc = _lib().gka_forward_gated(_ptr(q), _ptr(k), _ptr(v), _ptr(beta), _ptr(gate), _ptr(o),
                                  B, H, T, D, dt, float(a), int(r), int(chunk), _ptr(final_state),
                                  _ptr(workspace), workspace.numel() * workspace.element_size(),
                                  _stream(stream))
    _check("gka_forward_gated", rc)
    return o


def host_workspace_bytes(B, H, T, D, chunk, dtype=torch.bfloat16, slice_pairs=0) -> int:
    return int(_lib().gka_forward_host_workspace_bytes(B, H, T, D, chunk, _DT[dtype], slice_pairs))


def alloc_host_workspace(B, H, T, D, chunk, dtype=torch.bfloat16, slice_pairs=0,
                         device=None) -> torch.Tensor:
    n = host_workspace_bytes(B, H, T, D, chunk, dtype, slice_pairs)
    return torch.empty(max(n, 256), dtype=torch.uint8, device=device or "cuda")


def gka_forward_host(q, k, v, beta, a: float, r: int, chunk: int, *, o=None, final_state=None,
                     slice_pairs=0, workspace=None, stream=None):
    """gka_forward from HOST tensors with the copies overlapped with the compute
    (see include/gka.h).  q, k, v: [B, H, T, D] fp32 or bf16 CPU tensors (pinned
    for overlap), beta: [B, H, T] fp32.  Returns o on the host; it is complete
    once `stream` (default: the current CUDA stream) has completed."""
    for t in (q, k, v, beta, o, final_state):
        if t is not None and (t.is_cuda or not t.is_contiguous()):
            raise ValueError("tensors must be contiguous host tensors")
    B, H, T, D = q.shape
    if k.shape != q.shape or v.shape != q.shape or beta.shape != (B, H, T):
        raise ValueError("shape mismatch")
    dt = _dtype(q)
    if k.dtype != q.dtype or v.dtype != q.dtype or beta.dtype != torch.float32:
        raise TypeError("q, k, v must share a dtype; beta must be float32")
    if o is None:
        o = torch.empty(q.shape, dtype=q.dtype, pin_memory=q.is_pinned())
    if final_state is not None and (final_state.dtype != torch.float32 or
                                    final_state.shape != (B, H, 2, D, D)):
        raise ValueError("final_state must be float32 [B, H, 2, D, D]")
    if workspace is None:
        workspace = alloc_host_workspace(B, H, T, D, chunk, q.dtype, slice_pairs)
    rc = _lib().gka_forward_host(_ptr(q), _ptr(k), _ptr(v), _ptr(beta), _ptr(o), B, H, T, D, dt,
                                 float(a), int(r), int(chunk), _ptr(final_state), int(slice_pairs),
                                 _ptr(workspace), workspace.numel() * workspace.element_size(),
                                 _stream(stream))
    _check("gka_forward_host", rc)
    return o


def gka_forward_static_scratch(q, k, v, beta, a: float, r: int, chunk: int, *, o=None,
                               final_state=None, stream=None):
    """gka_forward whose scratch is the library's own static device array
    (for callers that cannot allocate device memory; see include/gka.h).
    Calls that overlap on the GPU race on that array."""
    _dev(q, k, v, beta, o, final_state)
    B, H, T, D = q.shape
    if k.shape != q.shape or v.shape != q.shape or beta.shape != (B, H, T):
        raise ValueError("shape mismatch")
    dt = _dtype(q)
    if k.dtype != q.dtype or v.dtype != q.dtype or beta.dtype != torch.float32:
        raise TypeError("q, k, v must share a dtype; beta must be float32")
    if o is None:
        o = torch.empty_like(v)
    rc = _lib().gka_forward_static_scratch(_ptr(q), _ptr(k), _ptr(v), _ptr(beta), _ptr(o), B, H,
                                           T, D, dt, float(a), int(r), int(chunk),
                                           _ptr(final_state), _stream(stream))
    _check("gka_forward_static_scratch", rc)
    return o


def gka_decode_step(state, q, k, v, beta, a: float, r: int, *, o=None, stream=None):
    """One recurrent step in place on state [B, H, 2, D, D] fp32; q, k, v: [B, H, D];
    beta: [B, H] fp32.  Returns o [B, H, D]."""
    _dev(state, q, k, v, beta, o)
    B, H, D = q.shape
    if state.dtype != torch.float32 or state.shape != (B, H, 2, D, D):
        raise ValueError("state must be float32 [B, H, 2, D, D]")
    if k.shape != q.shape or v.shape != q.shape or beta.shape != (B, H):
        raise ValueError("shape mismatch")
    dt = _dtype(q)
    if o is None:
        o = torch.empty_like(v)
    rc = _lib().gka_decode_step(_ptr(state), _ptr(q), _ptr(k), _ptr(v), _ptr(beta), _ptr(o),
                                B, H, D, dt, float(a), int(r), _stream(stream))
    _check("gka_decode_step", rc)
    return o


def gka_decode_step_gated(state, q, k, v, beta, gate, a: float, r: int, *, o=None,
                          stream=None):
    """Write-gated decode step in place on state [B, H, 2, D, D] fp32; gate [B, H]
    fp32 in [0, 1] (None: no gate).  Returns o [B, H, D]."""
    _dev(state, q, k, v, beta, gate, o)
    B, H, D = q.shape
    if state.dtype != torch.float32 or state.shape != (B, H, 2, D, D):
        raise ValueError("state must be float32 [B, H, 2, D, D]")
    if k.shape != q.shape or v.shape != q.shape or beta.shape != (B, H):
        raise ValueError("shape mismatch")
    if gate is not None and (gate.shape != (B, H) or gate.dtype != torch.float32):
        raise ValueError("gate must be float32 [B, H]")
    dt = _dtype(q)
    if o is None:
        o = torch.empty_like(v)
    rc = _lib().gka_decode_step_gated(_ptr(state), _ptr(q), _ptr(k), _ptr(v), _ptr(beta),
                                      _ptr(gate), _ptr(o), B, H, D, dt, float(a), int(r),
                                      _stream(stream))
    _check("gka_decode_step_gated", rc)
    return o


def backward_workspace_bytes(B, H, T, D, chunk, dtype=torch.bfloat16) -> int:
    return int(_lib().gka_backward_workspace_bytes(B, H, T, D, chunk, _DT[dtype]))


def gka_backward(q, k, v, beta, dout, a: float, r: int, chunk: int = 32, *, gate=None,
                 workspace=None, stream=None):
    """Implicit-differentiation backward (see include/gka.h).  q, k, v, dout:
    [B, H, T, D] fp32 or bf16 CUDA tensors; beta (and the optional gate):
    [B, H, T] fp32.  Returns a dict with dq, dk, dv (dtype of q), dbeta and, with a
    gate, dgate (fp32)."""
    _dev(q, k, v, beta, gate, dout, workspace)
    B, H, T, D = q.shape
    if any(t.shape != q.shape for t in (k, v, dout)) or beta.shape != (B, H, T):
        raise ValueError("shape mismatch")
    if gate is not None and (gate.shape != (B, H, T) or gate.dtype != torch.float32):
        raise ValueError("gate must be float32 [B, H, T]")
    dt = _dtype(q)
    if any(t.dtype != q.dtype for t in (k, v, dout)) or beta.dtype != torch.float32:
        raise TypeError("q, k, v, dout must share a dtype; beta must be float32")
    out = {n: torch.empty_like(q) for n in ("dq", "dk", "dv")}
    out["dbeta"] = torch.empty_like(beta)
    if gate is not None:
        out["dgate"] = torch.empty_like(gate)
    if workspace is None:
        n = backward_workspace_bytes(B, H, T, D, chunk, q.dtype)
        workspace = torch.empty(max(n, 256), dtype=torch.uint8, device=q.device)
    rc = _lib().gka_backward(_ptr(q), _ptr(k), _ptr(v), _ptr(beta), _ptr(gate), _ptr(dout),
                             _ptr(out["dq"]), _ptr(out["dk"]), _ptr(out["dv"]), _ptr(out["dbeta"]),
                             _ptr(out.get("dgate")), B, H, T, D, dt, float(a), int(r), int(chunk),
                             _ptr(workspace), workspace.numel() * workspace.element_size(),
                             _stream(stream))
    _check("gka_backward", rc)
    return out


# ---------------------------------------------------------------------------
# The gated linear recurrence and the block's row operations.  These calls run on
# the device that holds their tensors, whichever is current, on `stream` or that
# device's current stream, to which outputs and workspaces that a call allocates
# belong too, as torch's allocator has it.
# ---------------------------------------------------------------------------
def _device_of(first, *rest):
    """The one CUDA device of the tensors given (None: not given)."""
    index = first.get_device()
    if index < 0:
        raise ValueError("tensors must be CUDA tensors")
    for t in rest:
        if t is not None and t.get_device() != index:
            raise ValueError("tensors must be on one CUDA device")
    return first.device


def _dense(*ts):
    for t in ts:
        if t is not None and not t.is_contiguous():
            raise ValueError("tensors must be contiguous CUDA tensors")


def _need(name, t, shape, dtype):
    if t is not None and (t.shape != shape or t.dtype != dtype):
        raise ValueError(f"{name} must be {str(dtype)[6:]} {list(shape)}")


def _apart(*outs):
    """No two of a call's outputs (and the inputs given with them) share memory; of a strided
    tensor, from its first element to its last."""
    spans = sorted((t.data_ptr(), t.data_ptr() + _extent(t)) for t in outs if t is not None and t.numel())
    for (_, e), (b, _) in zip(spans, spans[1:]):
        if b < e:
            raise ValueError("outputs must not share memory with each other or with inputs")


def _extent(t):
    """Bytes from a tensor's first element to behind its last."""
    if t.is_contiguous():
        return t.numel() * t.element_size()
    return (1 + sum((n - 1) * s for n, s in zip(t.shape, t.stride()))) * t.element_size()


def _under(stream, fn, *args, **kw):
    """The call with ``stream`` current: what it allocates is that stream's too."""
    if stream.device != args[0].device:
        raise ValueError("stream must belong to the tensors' device")
    with torch.cuda.stream(stream):
        return fn(*args, **kw)


def _invoke(fn, dev, *args):
    """Calls a C entry point whose last argument is the stream, on device ``dev``."""
    index = dev.index
    raw = torch._C._cuda_getCurrentRawStream(index)
    call = _entry(fn)
    if torch._C._cuda_getDevice() == index:
        rc = call(*args, raw)
    else:
        with torch.cuda.device(dev):
            rc = call(*args, raw)
    if rc != 0:
        raise GkaError(fn, rc)


@functools.lru_cache(maxsize=None)
def _entry(fn):
    return getattr(_lib(), fn)


@functools.lru_cache(maxsize=1024)
def _query(fn, *sizes):
    """A workspace query of the library (a function of the sizes alone)."""
    return int(getattr(_lib(), fn)(*sizes))


def _p(t):
    return None if t is None else t.data_ptr()


def _scratch(n, workspace, dev):
    if workspace is None:
        return torch.empty(n, dtype=torch.uint8, device=dev) if n else None
    if not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    return workspace


def _nbytes(t):
    return 0 if t is None else t.numel() * t.element_size()


def linear_workspace_bytes(B, H, T, D, dtype=torch.bfloat16, *, backward=False) -> int:
    """Workspace bytes of gka_linear_forward (or gka_linear_backward); may be 0."""
    fn = "gka_linear_backward_workspace_bytes" if backward else "gka_linear_forward_workspace_bytes"
    return _query(fn, B, H, T, D, _DT[dtype])


def _linear_inputs(q, k, v, beta, gate, shape):
    if k.shape != q.shape or v.shape != q.shape or beta.shape != shape:
        raise ValueError("shape mismatch")
    dt = _dtype(q)
    if k.dtype != q.dtype or v.dtype != q.dtype or beta.dtype != torch.float32:
        raise TypeError("q, k, v must share a dtype; beta must be float32")
    _need("gate", gate, shape, torch.float32)
    return dt


def gka_linear_forward(q, k, v, beta, *, gate=None, scale=1.0, initial_state=None,
                       final_state=None, o=None, workspace=None, stream=None):
    """Gated linear recurrence M_t = beta_t M_{t-1} + g_t v_t k_t^T, o_t = scale M_t q_t
    (see include/gka.h).  q, k, v: [B, H, T, D] fp32 or bf16 CUDA tensors, any T; beta
    (and the optional gate): [B, H, T] fp32; initial_state, final_state (written; may be
    initial_state): fp32 [B, H, D, D].  Returns o (shape and dtype of v)."""
    if stream is not None:
        return _under(stream, gka_linear_forward, q, k, v, beta, gate=gate, scale=scale,
                      initial_state=initial_state, final_state=final_state, o=o,
                      workspace=workspace)
    dev = _device_of(q, k, v, beta, gate, initial_state, final_state, o, workspace)
    _dense(q, k, v, beta, gate, initial_state, final_state, o)
    B, H, T, D = q.shape
    dt = _linear_inputs(q, k, v, beta, gate, (B, H, T))
    _need("initial_state", initial_state, (B, H, D, D), torch.float32)
    _need("final_state", final_state, (B, H, D, D), torch.float32)
    if o is None:
        o = torch.empty_like(v)
    else:
        _need("o", o, q.shape, q.dtype)
        for t in (q, k, v, beta, gate, initial_state, final_state, workspace):
            _apart(o, t)
    if final_state is not None and initial_state is not None and \
            0 < abs(final_state.data_ptr() - initial_state.data_ptr()) < _nbytes(final_state):
        raise ValueError("final_state must be initial_state itself or share none of its memory")
    n = _query("gka_linear_forward_workspace_bytes", B, H, T, D, dt)
    workspace = _scratch(n, workspace, dev)
    _invoke("gka_linear_forward", dev, _p(q), _p(k), _p(v), _p(beta), _p(gate), _p(o), B, H,
            T, D, dt, scale, _p(initial_state), _p(final_state), _p(workspace), _nbytes(workspace))
    return o


def gka_linear_decode_step(state, q, k, v, beta, *, gate=None, scale=1.0, o=None, stream=None):
    """One token of the gated linear recurrence, in place on state [B, H, D, D] fp32;
    q, k, v: [B, H, D]; beta (and the optional gate): [B, H] fp32.  Returns o [B, H, D]."""
    if stream is not None:
        return _under(stream, gka_linear_decode_step, state, q, k, v, beta, gate=gate,
                      scale=scale, o=o)
    dev = _device_of(state, q, k, v, beta, gate, o)
    _dense(state, q, k, v, beta, gate, o)
    B, H, D = q.shape
    dt = _linear_inputs(q, k, v, beta, gate, (B, H))
    if state.dtype != torch.float32 or state.shape != (B, H, D, D):
        raise ValueError("state must be float32 [B, H, D, D]")
    if o is None:
        o = torch.empty_like(v)
    else:
        _need("o", o, q.shape, q.dtype)
        for t in (state, q, k, v, beta, gate):
            _apart(o, t)
    _invoke("gka_linear_decode_step", dev, _p(state), _p(q), _p(k), _p(v), _p(beta),
            _p(gate), _p(o), B, H, D, dt, scale)
    return o


def gka_linear_backward(q, k, v, beta, dout, *, gate=None, scale=1.0, initial_state=None,
                        dfinal_state=None, workspace=None, stream=None):
    """Gradients of gka_linear_forward (see include/gka.h).  dout: [B, H, T, D] in the
    inputs' dtype; dfinal_state: optional gradient of the final state, fp32 [B, H, D, D].
    Returns a dict with dq, dk, dv (dtype of q), dbeta, with a gate dgate (fp32), and with
    an initial_state dstate (its gradient, fp32)."""
    if stream is not None:
        return _under(stream, gka_linear_backward, q, k, v, beta, dout, gate=gate,
                      scale=scale, initial_state=initial_state, dfinal_state=dfinal_state,
                      workspace=workspace)
    dev = _device_of(q, k, v, beta, gate, dout, initial_state, dfinal_state, workspace)
    _dense(q, k, v, beta, gate, dout, initial_state, dfinal_state)
    B, H, T, D = q.shape
    dt = _linear_inputs(q, k, v, beta, gate, (B, H, T))
    _need("dout", dout, q.shape, q.dtype)
    _need("initial_state", initial_state, (B, H, D, D), torch.float32)
    _need("dfinal_state", dfinal_state, (B, H, D, D), torch.float32)
    out = {n: torch.empty_like(q) for n in ("dq", "dk", "dv")}
    out["dbeta"] = torch.empty_like(beta)
    if gate is not None:
        out["dgate"] = torch.empty_like(gate)
    if initial_state is not None:
        out["dstate"] = torch.empty_like(initial_state)
    n = _query("gka_linear_backward_workspace_bytes", B, H, T, D, dt)
    workspace = _scratch(n, workspace, dev)
    _invoke("gka_linear_backward", dev, _p(q), _p(k), _p(v), _p(beta), _p(gate), _p(dout),
            _p(initial_state), _p(dfinal_state), _p(out["dq"]), _p(out["dk"]), _p(out["dv"]),
            _p(out["dbeta"]), _p(out.get("dgate")), _p(out.get("dstate")), B, H, T, D, dt, scale,
            _p(workspace), _nbytes(workspace))
    return out


_pack_strided = struct.Struct("Pqqq").pack   # gka_strided: pointer, strides of b, t, heads


def _strided(name, t, dtype, shape):
    """gka_strided of a [B, T, heads(, D)] tensor with contiguous rows (None: NULL)."""
    if t is None:
        return None
    if t.shape != shape or t.dtype != dtype:
        raise ValueError(f"{name} must be {str(dtype)[6:]} {list(shape)}")
    s = t.stride()
    if len(s) == 4 and s[3] != 1 and t.numel():
        raise ValueError(f"{name} must have contiguous rows")
    # the stride of an axis of one is never used, whatever torch reports for it
    return _pack_strided(t.data_ptr(), s[0] if shape[0] > 1 else 0, s[1] if shape[1] > 1 else 0,
                         s[2] if shape[2] > 1 else 0)


def _block_in_args(q, k, beta_logit, gate_logit, beta_bias, gate_bias, lengths):
    B, T, H, D = q.shape
    Hk = k.shape[2]
    dt = _dtype(q)
    _need("beta_bias", beta_bias, (H,), torch.float32)
    _need("gate_bias", gate_bias, (H,), torch.float32)
    _need("lengths", lengths, (B,), torch.int32)
    if gate_bias is not None and gate_logit is None:
        raise ValueError("gate_bias needs gate_logit")
    _dense(beta_bias, gate_bias, lengths)
    return B, T, H, Hk, D, dt, (
        _strided("q", q, q.dtype, (B, T, H, D)), _strided("k", k, q.dtype, (B, T, Hk, D)),
        _strided("beta_logit", beta_logit, q.dtype, (B, T, H)),
        _strided("gate_logit", gate_logit, q.dtype, (B, T, H)))


def gka_block_in(q, k, v, beta_logit, *, gate_logit=None, beta_bias=None, gate_bias=None,
                 lengths=None, eps=1e-6, stream=None):
    """Before the layer (see include/gka.h): unit rows of q and k, sigmoid gates, head-major
    layout.  q: [B, T, H, D], k, v: [B, T, Hk, D] (Hk divides H) fp32 or bf16 CUDA tensors
    at any strides with contiguous rows; beta_logit, gate_logit: [B, T, H] in the same
    dtype; beta_bias, gate_bias: [H] fp32; lengths: [B] int32, tokens past it are padding.
    Returns (q, k, v [B, H, T, D], beta [B, H, T] fp32, gate or None): the inputs of
    gka_forward_gated and gka_linear_forward."""
    if stream is not None:
        return _under(stream, gka_block_in, q, k, v, beta_logit, gate_logit=gate_logit,
                      beta_bias=beta_bias, gate_bias=gate_bias, lengths=lengths, eps=eps)
    dev = _device_of(q, k, v, beta_logit, gate_logit, beta_bias, gate_bias, lengths)
    B, T, H, Hk, D, dt, (sq, sk, sb, sg) = _block_in_args(q, k, beta_logit, gate_logit, beta_bias,
                                                          gate_bias, lengths)
    sv = _strided("v", v, q.dtype, (B, T, Hk, D))
    qo = torch.empty((B, H, T, D), dtype=q.dtype, device=dev)
    ko, vo = torch.empty_like(qo), torch.empty_like(qo)
    beta = torch.empty((B, H, T), device=dev, dtype=torch.float32)
    gate = torch.empty_like(beta) if gate_logit is not None or lengths is not None else None
    _invoke("gka_block_in_forward", dev, sq, sk, sv, sb, sg, _p(beta_bias), _p(gate_bias),
            _p(lengths), _p(qo), _p(ko), _p(vo), _p(beta), _p(gate), B, T, H, Hk, D, dt, eps)
    return qo, ko, vo, beta, gate


def gka_block_in_backward(q, k, beta_logit, dq, dk, dv, dbeta, *, gate_logit=None, dgate=None,
                          beta_bias=None, gate_bias=None, lengths=None, eps=1e-6, workspace=None,
                          stream=None):
    """Gradients of gka_block_in from those of its outputs: dq, dk, dv [B, H, T, D] in the
    inputs' dtype, dbeta (and dgate exactly with gate_logit) [B, H, T] fp32.  Returns a dict
    with dq [B, T, H, D], dk, dv [B, T, Hk, D], dbeta_logit (dgate_logit) [B, T, H], and for
    each bias given dbeta_bias (dgate_bias) [H] fp32."""
    if stream is not None:
        return _under(stream, gka_block_in_backward, q, k, beta_logit, dq, dk, dv, dbeta,
                      gate_logit=gate_logit, dgate=dgate, beta_bias=beta_bias,
                      gate_bias=gate_bias, lengths=lengths, eps=eps, workspace=workspace)
    dev = _device_of(q, k, beta_logit, gate_logit, dq, dk, dv, dbeta, dgate, beta_bias, gate_bias,
                       lengths, workspace)
    B, T, H, Hk, D, dt, (sq, sk, sb, sg) = _block_in_args(q, k, beta_logit, gate_logit, beta_bias,
                                                          gate_bias, lengths)
    _dense(dq, dk, dv, dbeta, dgate)
    for n, t in (("dq", dq), ("dk", dk), ("dv", dv)):
        _need(n, t, (B, H, T, D), q.dtype)
    _need("dbeta", dbeta, (B, H, T), torch.float32)
    _need("dgate", dgate, (B, H, T), torch.float32)
    if (gate_logit is None) != (dgate is None):
        raise ValueError("dgate is needed exactly with gate_logit")
    out = {"dq": torch.empty(B, T, H, D, dtype=q.dtype, device=dev),
           "dk": torch.empty(B, T, Hk, D, dtype=q.dtype, device=dev),
           "dv": torch.empty(B, T, Hk, D, dtype=q.dtype, device=dev),
           "dbeta_logit": torch.empty(B, T, H, dtype=q.dtype, device=dev)}
    if gate_logit is not None:
        out["dgate_logit"] = torch.empty(B, T, H, dtype=q.dtype, device=dev)
    for n, t in (("dbeta_bias", beta_bias), ("dgate_bias", gate_bias)):
        if t is not None:
            out[n] = torch.empty_like(t)
    n = _query("gka_block_in_backward_workspace_bytes", B, T, H, Hk, D, dt)
    workspace = _scratch(n, workspace, dev)
    _invoke("gka_block_in_backward", dev, sq, sk, sb, sg, _p(beta_bias), _p(gate_bias),
            _p(lengths), _p(dq), _p(dk), _p(dv), _p(dbeta), _p(dgate), _p(out["dq"]), _p(out["dk"]),
            _p(out["dv"]), _p(out["dbeta_logit"]), _p(out.get("dgate_logit")),
            _p(out.get("dbeta_bias")), _p(out.get("dgate_bias")), B, T, H, Hk, D, dt, eps,
            _p(workspace), _nbytes(workspace))
    return out


def _block_out_args(o, w, z, v, skip):
    B, H, T, D = o.shape
    dt = _dtype(o)
    _dense(o, w, v, skip)
    _need("w", w, (D,), torch.float32)
    _need("v", v, o.shape, o.dtype)
    _need("skip", skip, (H,), torch.float32)
    if (v is None) != (skip is None):
        raise ValueError("v and skip come together")
    return B, H, T, D, dt, _strided("z", z, o.dtype, (B, T, H, D))


def gka_block_out(o, w, *, z=None, v=None, skip=None, eps=1e-6, y=None, stream=None):
    """After the layer (see include/gka.h): y = rmsnorm(o + skip_h v) w silu(z), token-major.
    o (and the layer's v): [B, H, T, D] fp32 or bf16; w: [D] fp32; skip: [H] fp32, with v;
    z: [B, T, H, D] at any strides with contiguous rows.  Returns y [B, T, H, D]."""
    if stream is not None:
        return _under(stream, gka_block_out, o, w, z=z, v=v, skip=skip, eps=eps, y=y)
    dev = _device_of(o, w, z, v, skip, y)
    B, H, T, D, dt, sz = _block_out_args(o, w, z, v, skip)
    if y is None:
        y = torch.empty(B, T, H, D, dtype=o.dtype, device=dev)
    else:
        _dense(y)
        _need("y", y, (B, T, H, D), o.dtype)
        for t in (o, w, z, v, skip):
            _apart(y, t)
    _invoke("gka_block_out_forward", dev, _p(o), _p(v), sz, _p(w), _p(skip), _p(y), B, T, H,
            D, dt, eps)
    return y


def gka_block_out_backward(o, w, dy, *, z=None, v=None, skip=None, eps=1e-6, workspace=None,
                           stream=None):
    """Gradients of gka_block_out from dy [B, T, H, D].  Returns a dict with do [B, H, T, D],
    dw [D] fp32; with z: dz [B, T, H, D]; with v and skip: dv [B, H, T, D], dskip [H] fp32."""
    if stream is not None:
        return _under(stream, gka_block_out_backward, o, w, dy, z=z, v=v, skip=skip,
                      eps=eps, workspace=workspace)
    dev = _device_of(o, w, dy, z, v, skip, workspace)
    B, H, T, D, dt, sz = _block_out_args(o, w, z, v, skip)
    _dense(dy)
    _need("dy", dy, (B, T, H, D), o.dtype)
    out = {"do": torch.empty_like(o), "dw": torch.empty_like(w)}
    if z is not None:
        out["dz"] = torch.empty(B, T, H, D, dtype=o.dtype, device=dev)
    if v is not None:
        out["dv"], out["dskip"] = torch.empty_like(v), torch.empty_like(skip)
    n = _query("gka_block_out_backward_workspace_bytes", B, T, H, D, dt)
    workspace = _scratch(n, workspace, dev)
    _invoke("gka_block_out_backward", dev, _p(o), _p(v), sz, _p(w), _p(skip), _p(dy),
            _p(out["do"]), _p(out.get("dv")), _p(out.get("dz")), _p(out["dw"]), _p(out.get("dskip")),
            B, T, H, D, dt, eps, _p(workspace), _nbytes(workspace))
    return out


SOLVERS = ("chebyshev", "gd", "agd", "cg")


def gka_solver_study(q, k, beta, a: float, r: int, solver: str, chunk: int = 64, *, gate=None,
                     workspace=None, stream=None):
    """Residual history ||q_t - A_t x_i|| / ||q_t||, i = 0..r, of ``solver`` (one of
    SOLVERS) on every token's system (see include/gka.h).  Returns [B, H, T, r + 1] fp32."""
    _dev(q, k, beta, gate, workspace)
    B, H, T, D = q.shape
    if k.shape != q.shape or beta.shape != (B, H, T):
        raise ValueError("shape mismatch")
    if gate is not None and (gate.shape != (B, H, T) or gate.dtype != torch.float32):
        raise ValueError("gate must be float32 [B, H, T]")
    dt = _dtype(q)
    if k.dtype != q.dtype or beta.dtype != torch.float32:
        raise TypeError("q, k must share a dtype; beta must be float32")
    resid = torch.empty(B, H, T, r + 1, dtype=torch.float32, device=q.device)
    if workspace is None:
        n = int(_lib().gka_solver_study_workspace_bytes(B, H, T, D, chunk, dt))
        workspace = torch.empty(max(n, 256), dtype=torch.uint8, device=q.device)
    rc = _lib().gka_solver_study(_ptr(q), _ptr(k), _ptr(beta), _ptr(gate), B, H, T, D, dt,
                                 float(a), int(r), int(chunk), SOLVERS.index(solver), _ptr(resid),
                                 _ptr(workspace), workspace.numel() * workspace.element_size(),
                                 _stream(stream))
    _check("gka_solver_study", rc)
    return resid


def selftest_timeout(stream=None) -> None:
    """Launch the bounded-wait self-test (see include/gka.h)."""
    _check("gka_selftest_timeout", _lib().gka_selftest_timeout(_stream(stream)))


def device_status(stream=None) -> int:
    """Synchronises the stream and returns the library's device status code."""
    return int(_lib().gka_device_status(_stream(stream)))


def profiler_enable(on: bool = True) -> None:
    """Bracket every library kernel launch with CUDA events on its stream."""
    _check("gka_profiler_enable", _lib().gka_profiler_enable(1 if on else 0))


def profiler_read() -> dict:
    """Per-kernel {name: (total_ms, launches)} since the last read (waits on the events)."""
    out = KernelTimes()
    _check("gka_profiler_read", _lib().gka_profiler_read(ctypes.byref(out)))
    return {name: (out.ms[i], out.launches[i]) for i, name in enumerate(KERNEL_NAMES)
            if out.launches[i]}
