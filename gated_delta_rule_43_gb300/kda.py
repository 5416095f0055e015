"""Thin Python binding of libkda.so (the C ABI in include/kda.h).

Argument marshalling only: every step of the computation runs in the CUDA
kernels behind the C ABI.  PyTorch supplies device memory and the stream.
There is no CPU fallback: if the library is missing or no GPU is present the
calls raise.  Calls run on the current device: tensors or a stream of
another one are refused.
"""
from __future__ import annotations

import ctypes
import functools
import math
import os
import threading

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libkda.so")

KDA_OK, KDA_ERR_INVALID_ARG, KDA_ERR_UNSUPPORTED, KDA_ERR_DECAY_RANGE = 0, 1, 2, 3
KDA_ERR_TIMEOUT, KDA_ERR_CUDA, KDA_ERR_SEQLENS = 4, 5, 6
KDA_F32, KDA_BF16 = 0, 1
_DT = {torch.float32: KDA_F32, torch.bfloat16: KDA_BF16}
_F32 = torch.float32
_NORM = {"none": 0, "l2": 1, "rms": 2}
_LAYOUT = {"half": 0, "interleaved": 1}

# name -> (restype, argtypes) of every symbol include/kda.h declares
P, I32, I64, SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
F32 = ctypes.c_float
SIGNATURES = {
    "kda_abi_version": (I32, []),
    "kda_status_string": (ctypes.c_char_p, [I32]),
    "kda_chunk_fwd_workspace_size": (SZ, [I64, I32, I32, I32, I32, I32]),
    "kda_chunk_fwd": (I32, [P, P, P, P, P, P, P, I32, I64, I32, I32, I32, I32, P, P, P, P, SZ,
                            P]),
    "kda_chunk_fwd_profiled": (I32, [P, P, P, P, P, P, P, I32, I64, I32, I32, I32, I32, P, P,
                                     P, P, SZ, P, ctypes.POINTER(ctypes.c_void_p), I32,
                                     ctypes.POINTER(ctypes.c_int32)]),
    "kda_chunk_fwd_segmented_workspace_size": (SZ, [I64, I32, I32, I32, I32, I32, I32]),
    "kda_chunk_fwd_segmented": (I32, [P, P, P, P, P, P, P, I32, I64, I32, I32, I32, I32, P, P,
                                      P, I32, P, SZ, P]),
    "kda_chunk_fwd_noalloc": (I32, [P, P, P, P, P, P, P, I32, I64, I32, I32, I32, I32, P, P, P,
                                    P, P]),
    "kda_decode_workspace_size": (SZ, []),
    "kda_decode_step": (I32, [P, P, P, P, P, P, P, P, I32, I32, I32, I32, I32, P, SZ, P]),
    "kda_decode_step_indexed": (I32, [P, P, P, P, P, P, P, P, I32, P, I32, I32, I32, I32, I32, P,
                                      SZ, P]),
    "kda_gate_cumsum": (I32, [P, P, P, I32, I64, I32, I32, I32, I32, I32, P, P, SZ, P]),
    "kda_query_status": (I32, [P, P, ctypes.POINTER(ctypes.c_int64)]),
    "kda_test_chain_fault": (I32, [I64, I32]),
    "kda_la_chunk_fwd_workspace_size": (SZ, [I64, I32, I32, I32, I32, I32, I32]),
    "kda_la_chunk_fwd": (I32, [P, P, P, P, P, I32, I64, I32, I32, I32, I32, I32, I64, I64, I64,
                               I32, P, P, P, P, SZ, P]),
    "kda_test_la_fault": (I32, [I32]),
    "kda_la_decode_step": (I32, [P, P, P, P, P, P, I32, I32, I32, I32, I32, I32, I64, I64, I64,
                                 I32, P]),
    "kda_la_decode_step_indexed": (I32, [P, P, P, P, P, P, I32, P, I32, I32, I32, I32, I32, I32,
                                         I64, I64, I64, I32, P, SZ, P]),
    "kda_qk_norm_rope": (I32, [P, P, P, P, I64, I32, I32, I32, I32, I64, I64, I64, I64, P, P, I32,
                               F32, F32, F32, P, P, I32, I32, F32, P]),
    "kda_state_pool_workspace_size": (SZ, [I32]),
    "kda_state_pool_copy": (I32, [P, I32, I64, P, P, I32, P, SZ, P]),
    "kda_state_pool_compact": (I32, [P, I32, I64, P, P, P, P, SZ, P]),
}

_lock = threading.Lock()
_lib = None


class KdaError(RuntimeError):
    def __init__(self, code: int, where: str, info: int | None = None):
        self.code = code
        self.info = info
        msg = f"{where}: {status_string(code)}"
        if info is not None:
            msg += f" (info={info})"
        super().__init__(msg)


def load(path: str = LIB_PATH):
    """Load libkda.so (once).  Raises if it has not been built."""
    global _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(path):
                raise RuntimeError(
                    f"{path} is missing: build it with `python -c 'import __graft_entry__ as g; "
                    "g.build()'` (there is no CPU fallback)")
            lib = ctypes.CDLL(path)
            for name, (res, args) in SIGNATURES.items():
                fn = getattr(lib, name)
                fn.restype = res
                fn.argtypes = args
            _lib = lib
    return _lib


def status_string(code: int) -> str:
    return load().kda_status_string(int(code)).decode()


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


_current_device = getattr(torch._C, "_cuda_getDevice", None)


def _check_current(device):
    """The library launches on the current device: a call with another device's tensors would
    run there with foreign addresses, unordered with the work that made them."""
    if device != _current_device():
        raise ValueError(f"the tensors live on cuda:{device}, but cuda:{_current_device()} is "
                         f"current: make the call under torch.cuda.device({device})")


def _check_cuda(*ts):
    device = None
    for t in ts:
        if t is not None:
            if not t.is_cuda:
                raise ValueError("every tensor must live on a CUDA device (no CPU fallback)")
            if not t.is_contiguous():
                raise ValueError("tensors must be contiguous")
            if device is None:
                device = t.get_device()
                _check_current(device)
            elif t.get_device() != device:
                raise ValueError("every tensor must live on one CUDA device")


def _expect(name, t, shape, dtype=None):
    """t (when given) has exactly `shape` (and `dtype`): the C ABI takes raw pointers and
    sizes, so a tensor smaller than the sizes say would be read or written past its end."""
    if t is None:
        return
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")


def _check_step_inputs(q, k, v, z, beta, A_log, lead):
    """q, k, z [*lead, H, dk], v [*lead, H, dv], beta [*lead, H], one dtype (fp32 or bf16);
    A_log [H] fp32.  Returns (H, dk, dv)."""
    if q.dim() != len(lead) + 2 or v.dim() != len(lead) + 2:
        raise ValueError(f"q and v must be [{', '.join(map(str, lead))}, H, D]")
    H, dk = q.shape[-2:]
    dv = v.shape[-1]
    if q.dtype not in _DT:
        raise TypeError(f"q has dtype {q.dtype}; fp32 and bf16 are supported")
    _expect("k", k, (*lead, H, dk), q.dtype)
    _expect("z", z, (*lead, H, dk), q.dtype)
    _expect("v", v, (*lead, H, dv), q.dtype)
    _expect("beta", beta, (*lead, H), q.dtype)
    _expect("A_log", A_log, (H,), torch.float32)
    return H, dk, dv


def _check_prefill(q, k, v, z, beta, A_log, cu_seqlens, initial_state, o, final_state):
    if q.dim() != 3:
        raise ValueError("q must be [T, H, dk]")
    T = q.shape[0]
    H, dk, dv = _check_step_inputs(q, k, v, z, beta, A_log, (T,))
    if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 1 or cu_seqlens.dtype != torch.int32:
        raise TypeError("cu_seqlens must be a 1-D int32 tensor [N + 1]")
    N = cu_seqlens.numel() - 1
    _expect("initial_state", initial_state, (N, H, dk, dv), torch.float32)
    _expect("final_state", final_state, (N, H, dk, dv), torch.float32)
    _expect("o", o, (T, H, dv), q.dtype)
    return T, N, H, dk, dv


def chunk_fwd_workspace_size(total_tokens: int, num_seqs: int, H: int, dk: int, dv: int,
                             dtype: torch.dtype) -> int:
    return int(load().kda_chunk_fwd_workspace_size(total_tokens, num_seqs, H, dk, dv,
                                                   _DT[dtype]))


def alloc_workspace(nbytes: int, device) -> torch.Tensor:
    # torch's caching allocator returns 512-byte aligned blocks
    return torch.empty(max(int(nbytes), 256), dtype=torch.uint8, device=device)


def chunk_fwd(q, k, v, z, beta, A_log, cu_seqlens, initial_state=None, *,
              output_final_state: bool = True, o=None, final_state=None, workspace=None,
              stream=None, check: bool = False):
    """KDA chunked prefill over packed sequences (kda_chunk_fwd).

    q, k, z [T, H, dk], v [T, H, dv], beta [T, H] (fp32 or bf16, one dtype);
    A_log [H] fp32; cu_seqlens [N+1] int32; initial_state [N, H, dk, dv] fp32
    or None.  Returns (o [T, H, dv], final_state [N, H, dk, dv] fp32 or None).
    ``final_state`` may be passed as ``initial_state`` for an in-place update.
    With ``check=True`` the stream is synchronised and a device-side error
    raises KdaError.
    """
    lib = load()
    T, N, H, dk, dv = _check_prefill(q, k, v, z, beta, A_log, cu_seqlens, initial_state, o,
                                     final_state)
    _check_cuda(q, k, v, z, beta, A_log, cu_seqlens, initial_state, o, final_state, workspace)
    dt = _DT[q.dtype]
    if o is None:
        o = torch.empty(T, H, dv, dtype=q.dtype, device=q.device)
    if final_state is None and output_final_state:
        final_state = torch.empty(N, H, dk, dv, dtype=torch.float32, device=q.device)
    need = int(lib.kda_chunk_fwd_workspace_size(T, N, H, dk, dv, dt))
    if workspace is None:
        workspace = alloc_workspace(need, q.device)
    rc = lib.kda_chunk_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(z), _ptr(beta), _ptr(A_log),
                           _ptr(cu_seqlens), N, T, H, dk, dv, dt, _ptr(initial_state),
                           _ptr(final_state), _ptr(o), _ptr(workspace), workspace.numel(),
                           _stream(stream))
    if rc != KDA_OK:
        raise KdaError(rc, "kda_chunk_fwd")
    if check:
        query_status(workspace, stream, raise_on_error=True)
    return o, final_state


def chunk_fwd_segmented(q, k, v, z, beta, A_log, cu_seqlens, initial_state=None, *,
                        segments: int, output_final_state: bool = True, o=None,
                        final_state=None, workspace=None, stream=None, check: bool = False):
    """Segment-parallel prefill (kda_chunk_fwd_segmented): chunk_fwd's arguments and
    results, each sequence's chunks of a window cut into up to ``segments`` segments."""
    lib = load()
    T, N, H, dk, dv = _check_prefill(q, k, v, z, beta, A_log, cu_seqlens, initial_state, o,
                                     final_state)
    _check_cuda(q, k, v, z, beta, A_log, cu_seqlens, initial_state, o, final_state, workspace)
    dt = _DT[q.dtype]
    if o is None:
        o = torch.empty(T, H, dv, dtype=q.dtype, device=q.device)
    if final_state is None and output_final_state:
        final_state = torch.empty(N, H, dk, dv, dtype=torch.float32, device=q.device)
    need = int(lib.kda_chunk_fwd_segmented_workspace_size(T, N, H, dk, dv, dt, int(segments)))
    if workspace is None:
        workspace = alloc_workspace(need, q.device)
    rc = lib.kda_chunk_fwd_segmented(_ptr(q), _ptr(k), _ptr(v), _ptr(z), _ptr(beta),
                                     _ptr(A_log), _ptr(cu_seqlens), N, T, H, dk, dv, dt,
                                     _ptr(initial_state), _ptr(final_state), _ptr(o),
                                     int(segments), _ptr(workspace), workspace.numel(),
                                     _stream(stream))
    if rc != KDA_OK:
        raise KdaError(rc, "kda_chunk_fwd_segmented")
    if check:
        query_status(workspace, stream, raise_on_error=True)
    return o, final_state


def chunk_fwd_profiled(q, k, v, z, beta, A_log, cu_seqlens, initial_state, o, final_state,
                       workspace, events, stream=None) -> int:
    """kda_chunk_fwd with CUDA events recorded around each kernel it launches.

    `events` is a list of torch.cuda.Event(enable_timing=True); returns how many
    were recorded.  Kernel j of the call runs between events[2j] and events[2j+1],
    both recorded on the stream that kernel was launched on.
    """
    lib = load()
    T, N, H, dk, dv = _check_prefill(q, k, v, z, beta, A_log, cu_seqlens, initial_state, o,
                                     final_state)
    _check_cuda(q, k, v, z, beta, A_log, cu_seqlens, initial_state, o, final_state, workspace)
    for e in events:
        if not e.cuda_event:  # torch creates the CUDA event on its first record
            e.record(stream if stream is not None else torch.cuda.current_stream())
    handles = (ctypes.c_void_p * len(events))(*[ctypes.c_void_p(e.cuda_event) for e in events])
    used = ctypes.c_int32(0)
    rc = lib.kda_chunk_fwd_profiled(_ptr(q), _ptr(k), _ptr(v), _ptr(z), _ptr(beta), _ptr(A_log),
                                    _ptr(cu_seqlens), N, T, H, dk, dv, _DT[q.dtype],
                                    _ptr(initial_state), _ptr(final_state), _ptr(o),
                                    _ptr(workspace), workspace.numel(), _stream(stream),
                                    handles, len(events), ctypes.byref(used))
    if rc != KDA_OK:
        raise KdaError(rc, "kda_chunk_fwd_profiled")
    return used.value


def chunk_fwd_noalloc(q, k, v, z, beta, A_log, cu_seqlens, initial_state, o, final_state,
                      status_out=None, stream=None):
    """kda_chunk_fwd_noalloc: the chunked forward with the library's own fixed scratch.

    For callers that cannot allocate device memory; o, final_state and the
    optional 16-byte status_out buffer are supplied by the caller.  Work on the
    shared scratch must not overlap between calls (serialise them).
    """
    lib = load()
    T, N, H, dk, dv = _check_prefill(q, k, v, z, beta, A_log, cu_seqlens, initial_state, o,
                                     final_state)
    _check_cuda(q, k, v, z, beta, A_log, cu_seqlens, initial_state, o, final_state, status_out)
    if status_out is not None and status_out.numel() * status_out.element_size() < 16:
        raise ValueError("status_out must hold at least 16 bytes")
    rc = lib.kda_chunk_fwd_noalloc(_ptr(q), _ptr(k), _ptr(v), _ptr(z), _ptr(beta), _ptr(A_log),
                                   _ptr(cu_seqlens), N, T, H, dk, dv, _DT[q.dtype],
                                   _ptr(initial_state), _ptr(final_state), _ptr(o),
                                   _ptr(status_out), _stream(stream))
    if rc != KDA_OK:
        raise KdaError(rc, "kda_chunk_fwd_noalloc")
    return o, final_state


def decode_step(q, k, v, z, beta, A_log, state, *, o=None, workspace=None, stream=None):
    """One decode step for N sequences (kda_decode_step); `state` is updated in place.

    q, k, z [N, H, dk], v [N, H, dv], beta [N, H]; state [N, H, dk, dv] fp32.
    Returns o [N, H, dv].
    """
    lib = load()
    if q.dim() != 3:
        raise ValueError("q must be [N, H, dk]")
    N = q.shape[0]
    H, dk, dv = _check_step_inputs(q, k, v, z, beta, A_log, (N,))
    _expect("state", state, (N, H, dk, dv), torch.float32)
    _expect("o", o, (N, H, dv), q.dtype)
    _check_cuda(q, k, v, z, beta, A_log, state, o, workspace)
    if o is None:
        o = torch.empty(N, H, dv, dtype=q.dtype, device=q.device)
    if workspace is None:
        workspace = alloc_workspace(int(lib.kda_decode_workspace_size()), q.device)
    rc = lib.kda_decode_step(_ptr(q), _ptr(k), _ptr(v), _ptr(z), _ptr(beta), _ptr(A_log),
                             _ptr(state), _ptr(o), N, H, dk, dv, _DT[q.dtype], _ptr(workspace),
                             workspace.numel(), _stream(stream))
    if rc != KDA_OK:
        raise KdaError(rc, "kda_decode_step")
    return o


def decode_step_indexed(q, k, v, z, beta, A_log, state_pool, state_idx, *, o=None,
                        workspace=None, stream=None, check: bool = False):
    """One decode step where sequence n owns slot state_idx[n] of state_pool (in place).

    q, k, z [N, H, dk], v [N, H, dv], beta [N, H]; state_pool [P, H, dk, dv] fp32;
    state_idx [N] int32 (distinct values in [0, P)).  Returns o [N, H, dv].
    """
    lib = load()
    if q.dim() != 3 or state_pool.dim() != 4:
        raise ValueError("q must be [N, H, dk] and state_pool [P, H, dk, dv]")
    N = q.shape[0]
    H, dk, dv = _check_step_inputs(q, k, v, z, beta, A_log, (N,))
    _expect("state_pool", state_pool, (state_pool.shape[0], H, dk, dv), torch.float32)
    _expect("state_idx", state_idx, (N,), torch.int32)
    _expect("o", o, (N, H, dv), q.dtype)
    _check_cuda(q, k, v, z, beta, A_log, state_pool, state_idx, o, workspace)
    if o is None:
        o = torch.empty(N, H, dv, dtype=q.dtype, device=q.device)
    if workspace is None:
        workspace = alloc_workspace(int(lib.kda_decode_workspace_size()), q.device)
    rc = lib.kda_decode_step_indexed(_ptr(q), _ptr(k), _ptr(v), _ptr(z), _ptr(beta),
                                     _ptr(A_log), _ptr(state_pool), _ptr(state_idx),
                                     state_pool.shape[0], _ptr(o), N, H, dk, dv, _DT[q.dtype],
                                     _ptr(workspace), workspace.numel(), _stream(stream))
    if rc != KDA_OK:
        raise KdaError(rc, "kda_decode_step_indexed")
    if check:
        query_status(workspace, stream, raise_on_error=True)
    return o


def gate_cumsum(z, A_log, cu_seqlens, chunk: int = 64, *, softplus: bool = False,
                workspace=None, stream=None, check: bool = False):
    """The standalone gate kernel (kda_gate_cumsum): fp32 in-chunk cumsum of g [T, H, dk].

    softplus=True evaluates the unbounded -Softplus baseline instead of the
    lower-bounded gate (same 16-token range check)."""
    lib = load()
    if z.dim() != 3 or z.dtype not in _DT:
        raise ValueError("z must be [T, H, dk], fp32 or bf16")
    T, H, dk = z.shape
    _expect("A_log", A_log, (H,), torch.float32)
    if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 1 or cu_seqlens.dtype != torch.int32:
        raise TypeError("cu_seqlens must be a 1-D int32 tensor [N + 1]")
    _check_cuda(z, A_log, cu_seqlens, workspace)
    N = cu_seqlens.numel() - 1
    G = torch.empty(T, H, dk, dtype=torch.float32, device=z.device)
    dt = _DT[z.dtype]
    if workspace is None:
        workspace = alloc_workspace(int(lib.kda_chunk_fwd_workspace_size(T, N, H, dk, dk, dt)),
                                    z.device)
    rc = lib.kda_gate_cumsum(_ptr(z), _ptr(A_log), _ptr(cu_seqlens), N, T, H, dk, dt, chunk,
                             1 if softplus else 0, _ptr(G), _ptr(workspace), workspace.numel(),
                             _stream(stream))
    if rc != KDA_OK:
        raise KdaError(rc, "kda_gate_cumsum")
    if check:
        query_status(workspace, stream, raise_on_error=True)
    return G, workspace


# The calls below are short on the GPU (a decode step of one sequence takes 4 us), so their
# checks are written to cost little: one comparison where everything fits, the message only
# where something does not.
def _addr(t):
    return None if t is None else t.data_ptr()


_current_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _raw_stream(stream, device):
    if stream is not None:
        of = getattr(stream, "device", None)
        if of is not None and of.index != device:
            raise ValueError(f"the stream is of {of}, the tensors live on cuda:{device}")
        return stream.cuda_stream
    return _current_raw_stream(device)


def _off_gpu():
    raise ValueError("every tensor must live on one CUDA device (no CPU fallback)")


def _same_gpu(q, *ts):
    """The index of q's GPU, which is the current one; every tensor given lives there."""
    device = q.get_device()
    if device < 0:
        _off_gpu()
    if device != _current_device():
        _check_current(device)
    for t in ts:
        if t is not None and t.get_device() != device:
            _off_gpu()
    return device


def _dense(name, t, shape, dtype):
    """t has exactly this shape and dtype and is contiguous; returns its address."""
    if t.shape != shape or t.dtype != dtype:
        _expect(name, t, shape, dtype)
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _rows(name, t, T, heads, D, dtype):
    """Checks a [T, heads, D] tensor whose tokens may lie further apart than heads * D (a
    slice of a fused projection); returns the distance in elements.  A single token or none
    has no distance: the packed one stands for it."""
    if t.shape != (T, heads, D) or t.dtype != dtype:
        _expect(name, t, (T, heads, D), dtype)
    s = t.stride()
    if (s[2] != 1 and D > 1) or (s[1] != D and heads > 1):
        raise ValueError(f"{name}: heads and channels must be packed (strides {s})")
    return s[0] if T > 1 else heads * D


def _new(like, shape, dtype, stream):
    """Buffers that a call allocates belong to the stream that it runs on, so that the caching
    allocator hands their memory on in that stream's order."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=like.device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=like.device)


def _workspace(like, nbytes, workspace, stream):
    """(workspace, its address, its bytes): the caller's, or a new one."""
    if workspace is None:
        workspace = _new(like, max(nbytes, 256), torch.uint8, stream)
        return workspace, workspace.data_ptr(), max(nbytes, 256)
    if not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    return workspace, workspace.data_ptr(), workspace.numel() * workspace.element_size()


def _check_la(q, k, v, g):
    """q, k [T, Hk, dk], v [T, H, dv] (token strides free), g [T, H] or [H] fp32.
    Returns (T, H, Hk, dk, dv, dtype, token strides, g per token, g's address)."""
    if q.dim() != 3 or v.dim() != 3:
        raise ValueError("q must be [T, Hk, dk] and v [T, H, dv]")
    dtype = q.dtype
    if dtype not in _DT:
        raise TypeError(f"q has dtype {dtype}; fp32 and bf16 are supported")
    T, Hk, dk = q.shape
    _, H, dv = v.shape
    if Hk < 1 or H % Hk:
        raise ValueError(f"{H} value heads cannot share {Hk} query/key heads")
    strides = (_rows("q", q, T, Hk, dk, dtype), _rows("k", k, T, Hk, dk, dtype),
               _rows("v", v, T, H, dv, dtype))
    if g.dim() == 2:
        return T, H, Hk, dk, dv, dtype, strides, 1, _dense("g", g, (T, H), _F32)
    return T, H, Hk, dk, dv, dtype, strides, 0, _dense("g", g, (H,), _F32)


@functools.lru_cache(maxsize=1024)
def _la_workspace_size(device, *sizes):   # (the size goes by the device's SMs, too)
    return load().kda_la_chunk_fwd_workspace_size(*sizes)


def la_chunk_fwd(q, k, v, g, cu_seqlens, initial_state=None, *, output_final_state: bool = True,
                 o=None, final_state=None, workspace=None, stream=None, check: bool = False):
    """Chunked prefill of linear attention with one decay per head (kda_la_chunk_fwd).

    S_t = exp(g_t) S_{t-1} + k_t v_t^T, o_t = S_t^T q_t over packed sequences: q, k
    [T, Hk, dk] and v [T, H, dv] (fp32 or bf16, one dtype; tokens may be slices of wider
    rows), Hk divides H; g the log decays, <= 0, fp32, [T, H] or [H]; cu_seqlens [N+1] int32;
    initial_state [N, H, dk, dv] fp32 or None.  Returns (o [T, H, dv], final_state fp32 or
    None).  ``final_state`` may be ``initial_state``.  ``check=True`` synchronises the stream
    and raises device-found errors.
    """
    lib = _lib or load()
    T, H, Hk, dk, dv, dtype, (qs, ks, vs), gpt, ga = _check_la(q, k, v, g)
    if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 1 or cu_seqlens.dtype != torch.int32:
        raise TypeError("cu_seqlens must be a 1-D int32 tensor [N + 1]")
    N = cu_seqlens.numel() - 1
    ca = _dense("cu_seqlens", cu_seqlens, (N + 1,), torch.int32)
    ia = None
    if initial_state is not None:
        ia = _dense("initial_state", initial_state, (N, H, dk, dv), torch.float32)
    if final_state is not None:
        _dense("final_state", final_state, (N, H, dk, dv), torch.float32)
    if o is not None:
        _dense("o", o, (T, H, dv), dtype)
    device = _same_gpu(q, k, v, g, cu_seqlens, initial_state, o, final_state, workspace)
    if o is None:
        o = _new(q, (T, H, dv), dtype, stream)
    if final_state is None and output_final_state:
        final_state = _new(q, (N, H, dk, dv), torch.float32, stream)
    dt = _DT[dtype]
    need = 0
    if workspace is None:
        need = _la_workspace_size(device, T, N, H, Hk, dk, dv, dt)
    workspace, wa, wb = _workspace(q, need, workspace, stream)
    rc = lib.kda_la_chunk_fwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), ga, ca, N, T, H, Hk, dk, dv,
                              dt, qs, ks, vs, gpt, ia, _addr(final_state), o.data_ptr(), wa, wb,
                              _raw_stream(stream, device))
    if rc != KDA_OK:
        raise KdaError(rc, "kda_la_chunk_fwd")
    if check:
        query_status(workspace, stream, raise_on_error=True)
    return o, final_state


def la_decode_step(q, k, v, g, state, *, o=None, stream=None):
    """One token of the decayed linear attention for N sequences (kda_la_decode_step).

    q, k [N, Hk, dk], v [N, H, dv], g [N, H] or [H] fp32; state [N, H, dk, dv] fp32, updated
    in place.  Returns o [N, H, dv].
    """
    lib = _lib or load()
    N, H, Hk, dk, dv, dtype, (qs, ks, vs), gpt, ga = _check_la(q, k, v, g)
    sa = _dense("state", state, (N, H, dk, dv), torch.float32)
    if o is not None:
        _dense("o", o, (N, H, dv), dtype)
    device = _same_gpu(q, k, v, g, state, o)
    if o is None:
        o = _new(q, (N, H, dv), dtype, stream)
    rc = lib.kda_la_decode_step(q.data_ptr(), k.data_ptr(), v.data_ptr(), ga, sa, o.data_ptr(), N, H,
                                Hk, dk, dv, _DT[dtype], qs, ks, vs, gpt,
                                _raw_stream(stream, device))
    if rc != KDA_OK:
        raise KdaError(rc, "kda_la_decode_step")
    return o


def la_decode_step_indexed(q, k, v, g, state_pool, state_idx, *, o=None, workspace=None,
                           stream=None, check: bool = False):
    """la_decode_step where sequence n owns slot state_idx[n] (distinct, int32) of state_pool
    [P, H, dk, dv].  With a workspace (or check=True) an index outside the pool is recorded
    in its status word; that sequence is skipped either way and its row of o not written."""
    lib = _lib or load()
    N, H, Hk, dk, dv, dtype, (qs, ks, vs), gpt, ga = _check_la(q, k, v, g)
    if state_pool.dim() != 4:
        raise ValueError("state_pool must be [P, H, dk, dv]")
    P_ = state_pool.shape[0]
    sa = _dense("state_pool", state_pool, (P_, H, dk, dv), torch.float32)
    xa = _dense("state_idx", state_idx, (N,), torch.int32)
    if o is not None:
        _dense("o", o, (N, H, dv), dtype)
    device = _same_gpu(q, k, v, g, state_pool, state_idx, o, workspace)
    if o is None:
        o = _new(q, (N, H, dv), dtype, stream)
    wa, wb = None, 0
    if workspace is not None or check:
        workspace, wa, wb = _workspace(q, lib.kda_decode_workspace_size(), workspace, stream)
    rc = lib.kda_la_decode_step_indexed(q.data_ptr(), k.data_ptr(), v.data_ptr(), ga, sa, xa, P_,
                                        o.data_ptr(), N, H, Hk, dk, dv, _DT[dtype], qs, ks, vs, gpt,
                                        wa, wb, _raw_stream(stream, device))
    if rc != KDA_OK:
        raise KdaError(rc, "kda_la_decode_step_indexed")
    if check:
        query_status(workspace, stream, raise_on_error=True)
    return o


def rope_inv_freq(rot_dim: int, base: float = 10000.0, *, scaling: str = "none",
                  factor: float = 1.0, original_length: int = 8192, fast_turns: float = 32.0,
                  slow_turns: float = 1.0, device=None):
    """(inv_freq [rot_dim / 2] fp32, rope_scale) for qk_norm_rope.

    The rates are base^(-2 i / rot_dim).  For contexts ``factor`` times as long as the
    ``original_length`` a model was trained with, scaling "linear" divides every rate by the
    factor (positions are interpolated), "base" raises the base so that only the slowest
    rate is divided by it, and "parts" divides the rates that turn less than ``slow_turns``
    times over the original length, keeps those that turn more than ``fast_turns`` times,
    and blends in between, linearly in the number of turns; it returns rope_scale =
    1 + 0.1 ln(factor), which sharpens the scores of the longer context (1 for the others).
    A model that was trained with other rates (a blend linear in the channel's index, for
    one) brings its own: qk_norm_rope takes any table.
    """
    if rot_dim < 0 or rot_dim % 2:
        raise ValueError("rot_dim must be even")
    if scaling not in ("none", "linear", "base", "parts"):
        raise ValueError(f"unknown scaling {scaling!r}")
    if not factor >= 1.0:
        raise ValueError("factor must be at least 1")
    i = torch.arange(rot_dim // 2, dtype=torch.float64)
    if scaling == "base" and rot_dim > 2:
        base = base * factor ** (rot_dim / (rot_dim - 2))
    rate = base ** (-2.0 * i / max(rot_dim, 1))
    scale = 1.0
    if scaling == "linear":
        rate = rate / factor
    elif scaling == "parts":
        turns = original_length * rate / (2.0 * math.pi)
        keep = ((turns - slow_turns) / (fast_turns - slow_turns)).clamp(0.0, 1.0)
        rate = rate * (keep + (1.0 - keep) / factor)
        scale = 1.0 + 0.1 * math.log(factor)
    return rate.to(torch.float32).to(device or "cpu"), scale


def qk_norm_rope(q, k, positions, inv_freq, *, norm: str = "l2", layout: str = "half",
                 eps: float = 1e-6, q_weight=None, k_weight=None, q_scale: float = 1.0,
                 k_scale: float = 1.0, rope_scale: float = 1.0, q_out=None, k_out=None,
                 stream=None):
    """Per-head norm of queries and keys and their position rotation (kda_qk_norm_rope).

    q [T, Hq, D] and k [T, Hk, D] or None (fp32 or bf16; tokens may be slices of wider rows);
    positions [T] int32 and inv_freq [rot_dim / 2] fp32 (see rope_inv_freq), or None and None
    for no rotation; norm "none", "l2" or "rms"; layout "half" or "interleaved"; weights [D]
    fp32 or None.  q_out and k_out may be q and k (in place); by default new packed tensors
    are returned.
    """
    lib = _lib or load()
    dtype = q.dtype
    if q.dim() != 3 or dtype not in _DT:
        raise TypeError("q must be [T, Hq, D], fp32 or bf16")
    if norm not in _NORM or layout not in _LAYOUT:
        raise ValueError(f"unknown norm {norm!r} or layout {layout!r}")
    T, Hq, D = q.shape
    qs, ks, kos, Hk = _rows("q", q, T, Hq, D, dtype), 0, 0, 0
    if k is not None:
        Hk = k.shape[1] if k.dim() == 3 else 0
        ks = _rows("k", k, T, Hk, D, dtype)
    elif k_out is not None or k_weight is not None:
        raise ValueError("k_out and k_weight need k")
    if (positions is None) != (inv_freq is None):
        raise ValueError("positions and inv_freq come together")
    rot, pa, fa, qwa, kwa = 0, None, None, None, None
    if inv_freq is not None:
        pa = _dense("positions", positions, (T,), torch.int32)
        fa = _dense("inv_freq", inv_freq, (inv_freq.numel(),), torch.float32)
        rot = 2 * inv_freq.numel()
    if q_weight is not None:
        qwa = _dense("q_weight", q_weight, (D,), torch.float32)
    if k_weight is not None:
        kwa = _dense("k_weight", k_weight, (D,), torch.float32)
    device = _same_gpu(q, k, positions, inv_freq, q_weight, k_weight, q_out, k_out)
    if q_out is None:
        q_out = _new(q, (T, Hq, D), dtype, stream)
    qos = _rows("q_out", q_out, T, Hq, D, dtype)
    if k is not None:
        if k_out is None:
            k_out = _new(q, (T, Hk, D), dtype, stream)
        kos = _rows("k_out", k_out, T, Hk, D, dtype)
    rc = lib.kda_qk_norm_rope(q.data_ptr(), _addr(k), q_out.data_ptr(), _addr(k_out), T, Hq, Hk, D,
                              _DT[dtype], qs, ks, qos, kos, qwa, kwa, _NORM[norm], eps, q_scale,
                              k_scale, pa, fa, rot, _LAYOUT[layout], rope_scale,
                              _raw_stream(stream, device))
    if rc != KDA_OK:
        raise KdaError(rc, "kda_qk_norm_rope")
    return q_out, k_out


def _check_pool(pool):
    if pool.dim() < 2 or pool.dtype != torch.float32:
        raise TypeError("a state pool is [P, ...] fp32")
    if not pool.is_contiguous():
        raise ValueError("the pool must be contiguous")
    slots = pool.shape[0]
    return slots, pool.numel() // slots if slots else 4


def state_pool_copy(pool, src_idx, dst_idx, *, workspace=None, stream=None, check: bool = False):
    """Slot dst_idx[i] of the pool [P, ...] fp32 becomes slot src_idx[i], or zeros where
    src_idx[i] is -1 (kda_state_pool_copy): copies, forks and clears.  No destination may be
    named twice or be another copy's source (a slot copied to itself may be); copies that
    break this or leave the pool are left out, and recorded in the workspace's status word
    when there is one (check=True raises).  More than 65536 copies need one of
    kda_state_pool_workspace_size(P) bytes where one is given."""
    lib = _lib or load()
    slots, elems = _check_pool(pool)
    if src_idx.dim() != 1:
        raise ValueError("src_idx must be [n]")
    n = src_idx.numel()
    sa = _dense("src_idx", src_idx, (n,), torch.int32)
    da = _dense("dst_idx", dst_idx, (n,), torch.int32)
    device = _same_gpu(pool, src_idx, dst_idx, workspace)
    wa, wb = None, 0
    many = n > 2048   # room for a mark a slot: checked against each other in linear time
    if workspace is not None or check or many:
        need = lib.kda_state_pool_workspace_size(slots) if many else lib.kda_decode_workspace_size()
        workspace, wa, wb = _workspace(pool, need, workspace, stream)
    rc = lib.kda_state_pool_copy(pool.data_ptr(), slots, elems, sa, da, n, wa, wb,
                                 _raw_stream(stream, device))
    if rc != KDA_OK:
        raise KdaError(rc, "kda_state_pool_copy")
    if check:
        query_status(workspace, stream, raise_on_error=True)


def state_pool_compact(pool, live, *, new_index=None, n_live=None, workspace=None, stream=None):
    """Packs the live slots of a pool to its front with the fewest moves
    (kda_state_pool_compact).  live [P] bool or uint8.  Returns (new_index [P] int32: where
    each live slot is now, -1 for dead ones; n_live [1] int32), both on the device."""
    lib = _lib or load()
    slots, elems = _check_pool(pool)
    if live.dtype not in (torch.bool, torch.uint8):
        raise TypeError(f"live has dtype {live.dtype}, expected bool or uint8")
    la = _dense("live", live, (slots,), live.dtype)
    if new_index is not None:
        _dense("new_index", new_index, (slots,), torch.int32)
    if n_live is not None:
        _dense("n_live", n_live, (1,), torch.int32)
    device = _same_gpu(pool, live, new_index, n_live, workspace)
    if new_index is None:
        new_index = _new(pool, (slots,), torch.int32, stream)
    if n_live is None:
        n_live = _new(pool, (1,), torch.int32, stream)
    need = lib.kda_state_pool_workspace_size(slots) if workspace is None else 0
    workspace, wa, wb = _workspace(pool, need, workspace, stream)
    rc = lib.kda_state_pool_compact(pool.data_ptr(), slots, elems, la, new_index.data_ptr(),
                                    n_live.data_ptr(), wa, wb, _raw_stream(stream, device))
    if rc != KDA_OK:
        raise KdaError(rc, "kda_state_pool_compact")
    return new_index, n_live


def query_status(workspace, stream=None, *, raise_on_error: bool = False):
    """(code, info) recorded in `workspace` by the last call (synchronises the stream)."""
    if workspace.is_cuda:
        _check_current(workspace.get_device())
    info = ctypes.c_int64(0)
    rc = load().kda_query_status(_ptr(workspace), _stream(stream), ctypes.byref(info))
    if raise_on_error and rc != KDA_OK:
        raise KdaError(rc, "device status", info.value)
    return rc, info.value
