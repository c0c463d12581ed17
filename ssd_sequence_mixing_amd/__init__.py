"""Python binding of libssd, the gfx950 SSD core (argument marshalling only).

Every function here forwards to the C ABI declared in include/ssd.h through
ctypes: it checks that tensors are on the GPU and contiguous, allocates outputs
and workspace with torch when the caller gives none, and passes raw device
pointers plus the current HIP stream. All arithmetic runs in the library's
kernels. There is no fallback: if libssd.so is missing, load() raises.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional, Tuple

__all__ = [
    "SSD_F32", "SSD_BF16", "SSDError", "load", "lib_path", "ssd_status_string",
    "ssd_chunk_scan_fwd_workspace_bytes", "ssd_chunk_scan_fwd", "ssd_chunk_scan_prepare",
    "ssd_chunk_scan_walk", "ssd_step", "ssd_chunk_scan_varlen_workspace_bytes",
    "ssd_chunk_scan_fwd_varlen", "ssd_chunk_scan_fwd_gated", "ssd_step_gated",
    "ssd_chunk_scan_bwd_workspace_bytes", "ssd_chunk_scan_bwd", "ssd_chunk_scan_fwd_fused",
    "ssd_chunk_scan_fwd_noalloc", "ssd_step_fused", "NOALLOC_SCRATCH_BYTES", "EXPORTS",
    "ssd_step_beam", "ssd_beam_select_workspace_bytes", "ssd_beam_select", "ssd_rms_norm", "ssd_rms_norm_mx",
    "ssd_mx_quantize", "ssd_rms_norm_bwd_workspace_bytes", "ssd_rms_norm_bwd", "ssd_linear_workspace_bytes",
    "ssd_linear", "ssd_linear_mx_workspace_bytes", "ssd_linear_mx", "ssd_linear_bwd_workspace_bytes",
    "ssd_linear_bwd", "ACTS",
]

SSD_F32 = 0
SSD_BF16 = 1
_PKG = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_PKG, "libssd.so")
_lib = None
torch = None   # imported by load(): libssd binds to torch's HIP runtime
_CODES = {}    # storage types

# Entry points include/ssd.h declares.
EXPORTS = ("ssd_status_string", "ssd_chunk_scan_fwd_workspace_bytes", "ssd_chunk_scan_fwd",
           "ssd_chunk_scan_prepare", "ssd_chunk_scan_walk", "ssd_step",
           "ssd_chunk_scan_varlen_workspace_bytes", "ssd_chunk_scan_fwd_varlen",
           "ssd_chunk_scan_fwd_gated", "ssd_step_gated", "ssd_chunk_scan_bwd_workspace_bytes",
           "ssd_chunk_scan_bwd", "ssd_chunk_scan_fwd_fused", "ssd_chunk_scan_fwd_noalloc", "ssd_step_fused",
           "ssd_step_beam", "ssd_beam_select_workspace_bytes", "ssd_beam_select", "ssd_rms_norm",
           "ssd_rms_norm_mx", "ssd_mx_quantize", "ssd_rms_norm_bwd_workspace_bytes", "ssd_rms_norm_bwd",
           "ssd_linear_workspace_bytes", "ssd_linear", "ssd_linear_mx_workspace_bytes", "ssd_linear_mx",
           "ssd_linear_bwd_workspace_bytes", "ssd_linear_bwd")

# SSD_NOALLOC_SCRATCH_BYTES: the static workspace of ssd_chunk_scan_fwd_noalloc.
NOALLOC_SCRATCH_BYTES = 64 << 20

# ssd_act: the activations of ssd_linear's epilogue.
ACTS = {"none": 0, "silu": 1, "gelu": 2}

_V = ctypes.c_void_p
_I = ctypes.c_int64


class SSDError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        super().__init__(f"{where}: {ssd_status_string(code)} (status {code})")


def lib_path() -> str:
    return _LIB_PATH


def _hip_runtimes_mapped():
    """Paths of every libamdhip64 mapped into this process."""
    paths = set()
    try:
        with open("/proc/self/maps") as f:
            for line in f:
                if "libamdhip64" in line:
                    paths.add(os.path.realpath(line.split()[-1]))
    except OSError:
        pass
    return paths


def load():
    """Loads libssd.so (built by ssd_sequence_mixing_amd.build); raises if absent.

    torch is imported first on purpose: torch ships its own HIP runtime, whose
    soname (libamdhip64.so.7) is the one libssd.so asks for, so loading torch
    first makes libssd bind to that same runtime. Loading libssd first would
    bring in a second HIP runtime (torch asks for its copy under another
    name), and device memory and streams owned by one runtime are not valid
    in the other."""
    global _lib, torch
    if _lib is not None:
        return _lib
    if not os.path.exists(_LIB_PATH):
        raise FileNotFoundError(
            f"{_LIB_PATH} is missing: build it with `python -m ssd_sequence_mixing_amd.build` "
            "(or __graft_entry__.build()). There is no fallback path.")
    import torch as t  # see the docstring: one HIP runtime per process
    torch = t
    _CODES.update({t.bfloat16: SSD_BF16, t.float32: SSD_F32})
    lib = ctypes.CDLL(_LIB_PATH)
    runtimes = _hip_runtimes_mapped()
    if len(runtimes) > 1:
        raise RuntimeError(f"two HIP runtimes are loaded in this process: {sorted(runtimes)}; "
                           "import torch before loading libssd.so")
    lib.ssd_status_string.restype = ctypes.c_char_p
    lib.ssd_status_string.argtypes = [ctypes.c_int]
    lib.ssd_chunk_scan_fwd_workspace_bytes.restype = ctypes.c_size_t
    lib.ssd_chunk_scan_fwd_workspace_bytes.argtypes = [_I] * 7 + [ctypes.c_int]
    lib.ssd_chunk_scan_fwd.restype = ctypes.c_int
    lib.ssd_chunk_scan_fwd.argtypes = [_V] * 6 + [_I, _V, _V] + [_I] * 6 + [ctypes.c_int, _V,
                                                                          ctypes.c_size_t, _V]
    lib.ssd_chunk_scan_prepare.restype = ctypes.c_int
    lib.ssd_chunk_scan_prepare.argtypes = [_V] * 4 + [_I] * 7 + [ctypes.c_int, _V, ctypes.c_size_t, _V]
    lib.ssd_chunk_scan_walk.restype = ctypes.c_int
    lib.ssd_chunk_scan_walk.argtypes = [_V] * 5 + [_I, _V, _V] + [_I] * 6 + [ctypes.c_int, _V,
                                                                           ctypes.c_size_t, _V]
    lib.ssd_step.restype = ctypes.c_int
    lib.ssd_step.argtypes = [_V] * 8 + [_I] * 5 + [ctypes.c_int, _V]
    lib.ssd_chunk_scan_varlen_workspace_bytes.restype = ctypes.c_size_t
    lib.ssd_chunk_scan_varlen_workspace_bytes.argtypes = [_I] * 7 + [ctypes.c_int]
    lib.ssd_chunk_scan_fwd_gated.restype = ctypes.c_int
    lib.ssd_chunk_scan_fwd_gated.argtypes = ([_V, _V, _V, ctypes.c_int] + [_V] * 5 + [_I, _V, _V] + [_I] * 6 +
                                             [ctypes.c_int, _V, ctypes.c_size_t, _V])
    lib.ssd_step_gated.restype = ctypes.c_int
    lib.ssd_step_gated.argtypes = ([_V, _V, _V, _V, ctypes.c_int] + [_V] * 6 + [_I] * 5 +
                                   [ctypes.c_int, _V])
    lib.ssd_chunk_scan_fwd_varlen.restype = ctypes.c_int
    lib.ssd_chunk_scan_fwd_varlen.argtypes = ([_V] * 6 + [_I, _V] + [_I] * 3 + [_V, _V, _V] + [_I] * 4 +
                                              [ctypes.c_int, _V, ctypes.c_size_t, _V])
    lib.ssd_chunk_scan_fwd_fused.restype = ctypes.c_int
    lib.ssd_chunk_scan_fwd_fused.argtypes = ([_V] * 5 + [ctypes.c_int] + [_V] * 5 + [_I, _V, _V] + [_I] * 6 +
                                             [ctypes.c_int, _V, ctypes.c_size_t, _V])
    lib.ssd_step_fused.restype = ctypes.c_int
    lib.ssd_step_fused.argtypes = ([_V] * 7 + [ctypes.c_int] + [_V] * 6 + [_I] * 5 + [ctypes.c_int, _V])
    lib.ssd_chunk_scan_fwd_noalloc.restype = ctypes.c_int
    lib.ssd_chunk_scan_fwd_noalloc.argtypes = [_V] * 6 + [_I, _V, _V] + [_I] * 6 + [ctypes.c_int, _V]
    lib.ssd_chunk_scan_bwd_workspace_bytes.restype = ctypes.c_size_t
    lib.ssd_chunk_scan_bwd_workspace_bytes.argtypes = [_I] * 7 + [ctypes.c_int]
    lib.ssd_chunk_scan_bwd.restype = ctypes.c_int
    lib.ssd_chunk_scan_bwd.argtypes = ([_V] * 6 + [_I] + [_V] * 10 + [_I] * 6 +
                                       [ctypes.c_int, _V, ctypes.c_size_t, _V])
    _F, _E, _S = ctypes.c_float, ctypes.c_int, ctypes.c_size_t
    for name, res, args in (
            ("ssd_step_beam", _E, [_V, _V, _V, _I] + [_V] * 6 + [_V, _E] + [_V] * 6 + [_I] * 5 + [_E, _V]),
            ("ssd_beam_select_workspace_bytes", _S, [_I] * 3),
            ("ssd_beam_select", _E, [_V] * 3 + [_I] + [_V] * 4 + [_I] * 3 + [_E, _V, _S, _V]),
            ("ssd_rms_norm", _E, [_V] * 3 + [_F] + [_V] * 3 + [_I] * 3 + [_E, _E, _V]),
            ("ssd_rms_norm_mx", _E, [_V] * 3 + [_F] + [_V] * 3 + [_I] * 3 + [_E, _E, _V]),
            ("ssd_mx_quantize", _E, [_V] * 3 + [_I] * 2 + [_E, _V]),
            ("ssd_rms_norm_bwd_workspace_bytes", _S, [_I] * 3 + [_E] * 2),
            ("ssd_rms_norm_bwd", _E, [_V] * 8 + [_I] * 3 + [_E, _E, _V, _S, _V]),
            ("ssd_linear_workspace_bytes", _S, [_I] * 3 + [_E]),
            ("ssd_linear", _E, [_V] * 3 + [_E] + [_V] * 3 + [_I] * 3 + [_E, _V, _S, _V]),
            ("ssd_linear_mx_workspace_bytes", _S, [_I] * 3),
            ("ssd_linear_mx", _E, [_V] * 5 + [_E] + [_V] * 2 + [_I] * 3 + [_V, _S, _V]),
            ("ssd_linear_bwd_workspace_bytes", _S, [_I] * 3 + [_E, _E]),
            ("ssd_linear_bwd", _E, [_V] * 3 + [_E] + [_V] * 4 + [_I] * 3 + [_E, _V, _S, _V]),
    ):
        fn = getattr(lib, name)
        fn.restype, fn.argtypes = res, args
    _lib = lib
    return lib


def ssd_status_string(code: int) -> str:
    return load().ssd_status_string(int(code)).decode()


def _dtype_code(t) -> int:
    code = _CODES.get(t.dtype)
    if code is None:
        load()
        if t.dtype not in _CODES:
            raise TypeError(f"unsupported storage dtype {t.dtype}; use torch.bfloat16 or torch.float32")
        code = _CODES[t.dtype]
    return code


def _chk(name: str, t, shape, dtype) -> None:
    """Raises ValueError unless tensor t (when given) has this shape and dtype:
    the C ABI takes raw pointers and trusts the sizes it is told."""
    if t is None or (t.shape == shape and t.dtype == dtype):
        return
    if tuple(t.shape) != tuple(int(d) for d in shape):
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(int(d) for d in shape)}")
    if t.dtype != dtype:
        raise ValueError(f"{name}: dtype {t.dtype}, expected {dtype}")


def _check_scan(X, dt, A, B, C, D, *, Y=None, final_state=None, initial_state=None, z=None, dY=None,
                packed_seqs: Optional[int] = None):
    """Shapes and dtypes of a forward's (or backward's) tensors against X and B:
    X (b, T, H, P) and B (b, T, G, N), or for a packed batch X (total, H, P) and
    B (total, G, N) with packed_seqs sequences. X, dt, B, C, Y, z, dY share one
    storage dtype; A, D and the states are fp32."""
    if packed_seqs is None:
        if X.dim() != 4 or B.dim() != 4:
            raise ValueError("X must be (batch, T, H, P) and B (batch, T, G, N)")
        bsz, T, H, P = X.shape
        G, N = B.shape[2], B.shape[3]
        lead, nst = (bsz, T), bsz
    else:
        if X.dim() != 3 or B.dim() != 3:
            raise ValueError("packed X must be (total, H, P) and B (total, G, N)")
        total, H, P = X.shape
        G, N = B.shape[1], B.shape[2]
        lead, nst = (total,), packed_seqs
    st = X.dtype
    _dtype_code(X)
    _chk("dt", dt, (*lead, H), st)
    _chk("B", B, (*lead, G, N), st)
    _chk("C", C, (*lead, G, N), st)
    _chk("A", A, (H,), torch.float32)
    _chk("D", D, (H,), torch.float32)
    _chk("Y", Y, X.shape, st)
    _chk("z", z, X.shape, st)
    _chk("dY", dY, X.shape, st)
    _chk("final_state", final_state, (nst, H, P, N), torch.float32)
    _chk("initial_state", initial_state, (nst, H, P, N), torch.float32)


def _check_step(state, x, dt, A, B, C, D, y=None, z=None):
    """Shapes and dtypes of a decode step's tensors against state (b, H, P, N)
    and B (b, G, N)."""
    if state.dim() != 4 or B.dim() != 3:
        raise ValueError("state must be (batch, H, P, N) and B (batch, G, N)")
    bsz, H, P, N = state.shape
    G = B.shape[1]
    st = x.dtype
    _dtype_code(x)
    _chk("state", state, (bsz, H, P, N), torch.float32)
    _chk("x", x, (bsz, H, P), st)
    _chk("dt", dt, (bsz, H), st)
    _chk("B", B, (bsz, G, N), st)
    _chk("C", C, (bsz, G, N), st)
    _chk("A", A, (H,), torch.float32)
    _chk("D", D, (H,), torch.float32)
    _chk("y", y, (bsz, H, P), st)
    _chk("z", z, (bsz, H, P), st)


def _ptr(t) -> Optional[int]:
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("tensors must be on the GPU")
    if not t.is_contiguous():
        raise ValueError("tensors must be contiguous")
    return t.data_ptr()


def _stream(stream) -> Optional[int]:
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def ssd_chunk_scan_fwd_workspace_bytes(batch, seqlen, nheads, headdim, dstate, ngroups, chunk,
                                       dtype: int) -> int:
    n = load().ssd_chunk_scan_fwd_workspace_bytes(batch, seqlen, nheads, headdim, dstate, ngroups,
                                                  chunk, dtype)
    if n == ctypes.c_size_t(-1).value:
        raise SSDError(3, "ssd_chunk_scan_fwd_workspace_bytes")
    return int(n)


def ssd_chunk_scan_fwd(X, dt, A, B, C, D, chunk: int, Y=None, final_state=None, *,
                       want_final: bool = True, workspace=None, stream=None):
    """Chunked SSD forward. Shapes: X (b, T, H, P), dt (b, T, H), A/D (H,) fp32,
    B/C (b, T, G, N); X/dt/B/C share one storage dtype (bf16 or fp32).

    Returns (Y, final_state); final_state is None when want_final is False and
    none was passed in."""
    lib = load()
    _check_scan(X, dt, A, B, C, D, Y=Y, final_state=final_state)
    bsz, T, H, P = X.shape
    G, N = B.shape[2], B.shape[3]
    code = _dtype_code(X)
    if Y is None:
        Y = torch.empty_like(X)
    if final_state is None and want_final:
        final_state = torch.empty((bsz, H, P, N), dtype=torch.float32, device=X.device)
    need = ssd_chunk_scan_fwd_workspace_bytes(bsz, T, H, P, N, G, chunk, code)
    if workspace is None and need > 0:
        workspace = torch.empty(need, dtype=torch.uint8, device=X.device)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    st = lib.ssd_chunk_scan_fwd(_ptr(X), _ptr(dt), _ptr(A), _ptr(B), _ptr(C), _ptr(D), chunk,
                                _ptr(Y), _ptr(final_state), bsz, T, H, P, N, G, code,
                                _ptr(workspace), ws_bytes, _stream(stream))
    if st != 0:
        raise SSDError(st, "ssd_chunk_scan_fwd")
    return Y, final_state


def ssd_chunk_scan_fwd_noalloc(X, dt, A, B, C, D, chunk: int, Y, final_state=None, *, stream=None):
    """ssd_chunk_scan_fwd with the library's static workspace: the C call
    allocates nothing, so the caller passes Y (and final_state, or None to
    skip it) already allocated. Calls that may overlap on one GPU race on the
    shared workspace. Returns (Y, final_state)."""
    lib = load()
    if Y is None:
        raise ValueError("ssd_chunk_scan_fwd_noalloc allocates nothing: pass Y")
    _check_scan(X, dt, A, B, C, D, Y=Y, final_state=final_state)
    bsz, T, H, P = X.shape
    G, N = B.shape[2], B.shape[3]
    st = lib.ssd_chunk_scan_fwd_noalloc(_ptr(X), _ptr(dt), _ptr(A), _ptr(B), _ptr(C), _ptr(D), chunk,
                                        _ptr(Y), _ptr(final_state), bsz, T, H, P, N, G, _dtype_code(X),
                                        _stream(stream))
    if st != 0:
        raise SSDError(st, "ssd_chunk_scan_fwd_noalloc")
    return Y, final_state


def ssd_step_fused(state, conv_state, x, dt, A, B, C, D, *, conv_w, conv_b=None, dt_bias=None,
                   dt_softplus: int = 0, z=None, y=None, stream=None):
    """ssd_step_gated with the layer's causal conv1d(4) + SiLU on x: conv_state
    (b, H*P, 3) in x's dtype holds the 3 earlier raw inputs (oldest first) and
    is shifted in place, as is the fp32 state. conv_w (H*P, 4), conv_b (H*P)
    fp32. Returns y."""
    lib = load()
    _check_step(state, x, dt, A, B, C, D, y=y, z=z)
    bsz, H, P, N = state.shape
    G = B.shape[1]
    _chk("conv_state", conv_state, (bsz, H * P, 3), x.dtype)
    _chk("conv_w", conv_w, (H * P, 4), torch.float32)
    _chk("conv_b", conv_b, (H * P,), torch.float32)
    _chk("dt_bias", dt_bias, (H,), torch.float32)
    code = _dtype_code(x)
    if y is None:
        y = torch.empty_like(x)
    st = lib.ssd_step_fused(_ptr(state), _ptr(conv_state), _ptr(x), _ptr(conv_w), _ptr(conv_b), _ptr(dt),
                            _ptr(dt_bias), int(dt_softplus), _ptr(A), _ptr(B), _ptr(C), _ptr(D), _ptr(z),
                            _ptr(y), bsz, H, P, N, G, code, _stream(stream))
    if st != 0:
        raise SSDError(st, "ssd_step_fused")
    return y


def _workspace(workspace, need, device):
    if workspace is None and need > 0:
        workspace = torch.empty(need, dtype=torch.uint8, device=device)
    nbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    return workspace, nbytes


def ssd_chunk_scan_prepare(dt, A, B, C, chunk: int, headdim: int, *, workspace=None, stream=None):
    """Phase 1 of the forward: fills and returns the workspace."""
    lib = load()
    if dt.dim() != 3 or B.dim() != 4:
        raise ValueError("dt must be (batch, T, H) and B (batch, T, G, N)")
    bsz, T, H = dt.shape
    G, N = B.shape[2], B.shape[3]
    code = _dtype_code(dt)
    _chk("B", B, (bsz, T, G, N), dt.dtype)
    _chk("C", C, (bsz, T, G, N), dt.dtype)
    _chk("A", A, (H,), torch.float32)
    need = ssd_chunk_scan_fwd_workspace_bytes(bsz, T, H, headdim, N, G, chunk, code)
    workspace, nbytes = _workspace(workspace, need, dt.device)
    st = lib.ssd_chunk_scan_prepare(_ptr(dt), _ptr(A), _ptr(B), _ptr(C), chunk, bsz, T, H, headdim,
                                    N, G, code, _ptr(workspace), nbytes, _stream(stream))
    if st != 0:
        raise SSDError(st, "ssd_chunk_scan_prepare")
    return workspace


def ssd_chunk_scan_walk(X, B, C, D, workspace, chunk: int, initial_state=None, Y=None,
                        final_state=None, *, want_final: bool = True, stream=None):
    """Phase 2 of the forward: the chunk walk over a prepared workspace."""
    lib = load()
    if X.dim() != 4 or B.dim() != 4:
        raise ValueError("X must be (batch, T, H, P) and B (batch, T, G, N)")
    bsz, T, H, P = X.shape
    G, N = B.shape[2], B.shape[3]
    code = _dtype_code(X)
    _chk("B", B, (bsz, T, G, N), X.dtype)
    _chk("C", C, (bsz, T, G, N), X.dtype)
    _chk("D", D, (H,), torch.float32)
    _chk("Y", Y, X.shape, X.dtype)
    _chk("final_state", final_state, (bsz, H, P, N), torch.float32)
    _chk("initial_state", initial_state, (bsz, H, P, N), torch.float32)
    if Y is None:
        Y = torch.empty_like(X)
    if final_state is None and want_final:
        final_state = torch.empty((bsz, H, P, N), dtype=torch.float32, device=X.device)
    nbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    st = lib.ssd_chunk_scan_walk(_ptr(X), _ptr(B), _ptr(C), _ptr(D), _ptr(initial_state), chunk,
                                 _ptr(Y), _ptr(final_state), bsz, T, H, P, N, G, code,
                                 _ptr(workspace), nbytes, _stream(stream))
    if st != 0:
        raise SSDError(st, "ssd_chunk_scan_walk")
    return Y, final_state


def ssd_step(state, x, dt, A, B, C, D, y=None, *, stream=None):
    """One decode step; `state` (b, H, P, N) fp32 is updated in place. Returns y."""
    lib = load()
    _check_step(state, x, dt, A, B, C, D, y=y)
    bsz, H, P, N = state.shape
    G = B.shape[1]
    code = _dtype_code(x)
    if y is None:
        y = torch.empty_like(x)
    st = lib.ssd_step(_ptr(state), _ptr(x), _ptr(dt), _ptr(A), _ptr(B), _ptr(C), _ptr(D), _ptr(y),
                      bsz, H, P, N, G, code, _stream(stream))
    if st != 0:
        raise SSDError(st, "ssd_step")
    return y


def ssd_chunk_scan_varlen_workspace_bytes(num_seqs, max_seqlen, nheads, headdim, dstate, ngroups,
                                          chunk, dtype: int) -> int:
    n = load().ssd_chunk_scan_varlen_workspace_bytes(num_seqs, max_seqlen, nheads, headdim, dstate,
                                                     ngroups, chunk, dtype)
    if n == ctypes.c_size_t(-1).value:
        raise SSDError(3, "ssd_chunk_scan_varlen_workspace_bytes")
    return int(n)


def ssd_chunk_scan_fwd_varlen(X, dt, A, B, C, D, chunk: int, cu_seqlens, max_seqlen: int,
                              initial_state=None, Y=None, final_state=None, *,
                              want_final: bool = True, workspace=None, stream=None):
    """Forward over a packed variable-length batch. X (total, H, P), dt (total, H),
    B/C (total, G, N); cu_seqlens int32 on the GPU, (num_seqs + 1) cumulative
    lengths; max_seqlen the longest sequence (a host int, so that no device value
    has to be read here). Returns (Y, final_state) with final_state
    (num_seqs, H, P, N) fp32."""
    lib = load()
    if cu_seqlens.dtype != torch.int32 or cu_seqlens.dim() != 1 or cu_seqlens.numel() < 1:
        raise ValueError("cu_seqlens must be a 1-d int32 tensor of num_seqs + 1 offsets")
    nseq = cu_seqlens.numel() - 1
    _check_scan(X, dt, A, B, C, D, Y=Y, final_state=final_state, initial_state=initial_state,
                packed_seqs=nseq)
    total, H, P = X.shape
    G, N = B.shape[1], B.shape[2]
    code = _dtype_code(X)
    if Y is None:
        Y = torch.empty_like(X)
    if final_state is None and want_final:
        final_state = torch.empty((nseq, H, P, N), dtype=torch.float32, device=X.device)
    need = ssd_chunk_scan_varlen_workspace_bytes(nseq, max_seqlen, H, P, N, G, chunk, code)
    workspace, nbytes = _workspace(workspace, need, X.device)
    st = lib.ssd_chunk_scan_fwd_varlen(_ptr(X), _ptr(dt), _ptr(A), _ptr(B), _ptr(C), _ptr(D), chunk,
                                       _ptr(cu_seqlens), nseq, max_seqlen, total, _ptr(initial_state),
                                       _ptr(Y), _ptr(final_state), H, P, N, G, code, _ptr(workspace),
                                       nbytes, _stream(stream))
    if st != 0:
        raise SSDError(st, "ssd_chunk_scan_fwd_varlen")
    return Y, final_state


def ssd_chunk_scan_fwd_gated(X, dt, A, B, C, D, chunk: int, *, dt_bias=None, dt_softplus: int = 0, z=None,
                             Y=None, final_state=None, want_final: bool = True, workspace=None, stream=None):
    """ssd_chunk_scan_fwd with the fused prologue (dt_bias, dt_softplus: 0 none,
    1 softplus(dt + bias), 2 softplus(dt) + bias) and output gate Y * silu(z)."""
    lib = load()
    _check_scan(X, dt, A, B, C, D, Y=Y, final_state=final_state, z=z)
    _chk("dt_bias", dt_bias, (X.shape[2],), torch.float32)
    bsz, T, H, P = X.shape
    G, N = B.shape[2], B.shape[3]
    code = _dtype_code(X)
    if Y is None:
        Y = torch.empty_like(X)
    if final_state is None and want_final:
        final_state = torch.empty((bsz, H, P, N), dtype=torch.float32, device=X.device)
    need = ssd_chunk_scan_fwd_workspace_bytes(bsz, T, H, P, N, G, chunk, code)
    workspace, nbytes = _workspace(workspace, need, X.device)
    st = lib.ssd_chunk_scan_fwd_gated(_ptr(X), _ptr(dt), _ptr(dt_bias), int(dt_softplus), _ptr(A), _ptr(B),
                                      _ptr(C), _ptr(D), _ptr(z), chunk, _ptr(Y), _ptr(final_state), bsz, T,
                                      H, P, N, G, code, _ptr(workspace), nbytes, _stream(stream))
    if st != 0:
        raise SSDError(st, "ssd_chunk_scan_fwd_gated")
    return Y, final_state


def ssd_chunk_scan_fwd_fused(X, dt, A, B, C, D, chunk: int, *, conv_w=None, conv_b=None, dt_bias=None,
                             dt_softplus: int = 0, z=None, Y=None, final_state=None, want_final: bool = True,
                             workspace=None, stream=None):
    """ssd_chunk_scan_fwd_gated with the input activation fused in: X is taken before the
    causal 4-tap depthwise convolution (conv_w (H*P, 4), conv_b (H*P) fp32) and SiLU."""
    lib = load()
    _check_scan(X, dt, A, B, C, D, Y=Y, final_state=final_state, z=z)
    _chk("dt_bias", dt_bias, (X.shape[2],), torch.float32)
    _chk("conv_w", conv_w, (X.shape[2] * X.shape[3], 4), torch.float32)
    _chk("conv_b", conv_b, (X.shape[2] * X.shape[3],), torch.float32)
    bsz, T, H, P = X.shape
    G, N = B.shape[2], B.shape[3]
    code = _dtype_code(X)
    if Y is None:
        Y = torch.empty_like(X)
    if final_state is None and want_final:
        final_state = torch.empty((bsz, H, P, N), dtype=torch.float32, device=X.device)
    need = ssd_chunk_scan_fwd_workspace_bytes(bsz, T, H, P, N, G, chunk, code)
    workspace, nbytes = _workspace(workspace, need, X.device)
    st = lib.ssd_chunk_scan_fwd_fused(_ptr(X), _ptr(conv_w), _ptr(conv_b), _ptr(dt), _ptr(dt_bias),
                                      int(dt_softplus), _ptr(A), _ptr(B), _ptr(C), _ptr(D), _ptr(z), chunk,
                                      _ptr(Y), _ptr(final_state), bsz, T, H, P, N, G, code, _ptr(workspace),
                                      nbytes, _stream(stream))
    if st != 0:
        raise SSDError(st, "ssd_chunk_scan_fwd_fused")
    return Y, final_state


def ssd_step_gated(state, x, dt, A, B, C, D, *, dt_bias=None, dt_softplus: int = 0, z=None, y=None,
                   stream=None):
    """ssd_step with the fused prologue and output gate (see ssd_chunk_scan_fwd_gated)."""
    lib = load()
    _check_step(state, x, dt, A, B, C, D, y=y, z=z)
    _chk("dt_bias", dt_bias, (state.shape[1],), torch.float32)
    bsz, H, P, N = state.shape
    G = B.shape[1]
    code = _dtype_code(x)
    if y is None:
        y = torch.empty_like(x)
    st = lib.ssd_step_gated(_ptr(state), _ptr(x), _ptr(dt), _ptr(dt_bias), int(dt_softplus), _ptr(A),
                            _ptr(B), _ptr(C), _ptr(D), _ptr(z), _ptr(y), bsz, H, P, N, G, code,
                            _stream(stream))
    if st != 0:
        raise SSDError(st, "ssd_step_gated")
    return y


def ssd_chunk_scan_bwd_workspace_bytes(batch, seqlen, nheads, headdim, dstate, ngroups, chunk,
                                       dtype=SSD_BF16) -> int:
    n = load().ssd_chunk_scan_bwd_workspace_bytes(batch, seqlen, nheads, headdim, dstate, ngroups, chunk,
                                                  int(dtype))
    if n == ctypes.c_size_t(-1).value:
        raise SSDError(3, "ssd_chunk_scan_bwd_workspace_bytes")
    return int(n)


def ssd_chunk_scan_bwd(X, dt, A, B, C, D, chunk: int, dY, *, initial_state=None, d_final_state=None,
                       want_initial_grad: bool = False, workspace=None, stream=None):
    """Gradients of <dY, Y> + <dF, final_state> for ssd_chunk_scan_fwd(X, dt, A, B, C, D, chunk)
    from initial_state (zero when None). Returns (dX, ddt, dA, dB, dC, dD, d_initial_state);
    the last is None unless want_initial_grad."""
    lib = load()
    _check_scan(X, dt, A, B, C, D, dY=dY, final_state=d_final_state, initial_state=initial_state)
    bsz, T, H, P = X.shape
    G, N = B.shape[2], B.shape[3]
    code = _dtype_code(X)
    dX, ddt = torch.empty_like(X), torch.empty_like(dt)
    dB, dC = torch.empty_like(B), torch.empty_like(C)
    dA = torch.empty((H,), dtype=torch.float32, device=X.device)
    dD = torch.empty((H,), dtype=torch.float32, device=X.device)
    dinit = (torch.empty((bsz, H, P, N), dtype=torch.float32, device=X.device)
             if want_initial_grad else None)
    nbytes = ssd_chunk_scan_bwd_workspace_bytes(bsz, T, H, P, N, G, chunk, code)
    if workspace is None:
        workspace = torch.empty((max(nbytes, 1),), dtype=torch.uint8, device=X.device)
    st = lib.ssd_chunk_scan_bwd(_ptr(X), _ptr(dt), _ptr(A), _ptr(B), _ptr(C), _ptr(D), int(chunk),
                                _ptr(initial_state), _ptr(dY), _ptr(d_final_state), _ptr(dX), _ptr(ddt),
                                _ptr(dA), _ptr(dB), _ptr(dC), _ptr(dD), _ptr(dinit), bsz, T, H, P, N, G,
                                code, _ptr(workspace), workspace.numel() * workspace.element_size(),
                                _stream(stream))
    if st != 0:
        raise SSDError(st, "ssd_chunk_scan_bwd")
    return dX, ddt, dA, dB, dC, dD, dinit


def _device(t) -> int:
    """The GPU that t is on, which has to be the current one: the stream a call goes to is that device's."""
    dev = t.get_device()
    if dev < 0:
        raise ValueError("tensors must be on the GPU")
    now = torch._C._cuda_getDevice()  # current_device() without its check that CUDA is there: a tensor is on it
    if dev != now:
        raise ValueError(f"tensor on cuda:{dev}, but the current device is cuda:{now}")
    return dev


def _stream_on(dev: int, stream) -> Optional[int]:
    """_stream, the current device being known. A stream of another device cannot run on this one's memory."""
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(dev)
    other = getattr(stream, "device_index", dev)
    if other != dev:
        raise ValueError(f"stream of cuda:{other}, but the tensors are on cuda:{dev}")
    return _stream(stream)


def _in(dev: int, name: str, t, shape, dtype) -> Optional[int]:
    """The address of an argument (None for None) that is checked: shape, type, device, contiguous."""
    if t is None:
        return None
    if t.shape == shape and t.dtype is dtype and t.get_device() == dev and t.is_contiguous():
        return t.data_ptr()
    _chk(name, t, shape, dtype)
    if t.get_device() != dev:
        raise ValueError(f"{name} is on {t.device}, not on cuda:{dev}")
    raise ValueError(f"{name}: tensors must be contiguous")


def _first(name: str, t) -> int:
    """_in of the argument that the device and the shapes are taken from."""
    if not t.is_contiguous():
        raise ValueError(f"{name}: tensors must be contiguous")
    return t.data_ptr()


def _scratch(workspace, need: int, like, dev: int, stream):
    """(tensor, address, bytes) of a call's workspace: the caller's, or a new one."""
    if workspace is None:
        if not need:
            return None, None, 0
        workspace = _new((need,), torch.uint8, like, stream)
    elif workspace.get_device() != dev or not workspace.is_contiguous():
        raise ValueError("workspace: must be contiguous and on the device of the tensors")
    return workspace, workspace.data_ptr(), workspace.numel() * workspace.element_size()


def _new(shape, dtype, like, stream):
    """An output or workspace for a call on `stream`. It is allocated as that
    stream's memory, so that it is not handed out again before the call is done."""
    if stream is None:
        return like.new_empty(shape, dtype=dtype)
    with torch.cuda.stream(stream if hasattr(stream, "cuda_stream") else torch.cuda.ExternalStream(int(stream))):
        return like.new_empty(shape, dtype=dtype)


def _like(t, stream, dtype=None):
    """_new of the shape (and type) of t, which is contiguous."""
    if stream is not None:
        return _new(t.shape, dtype or t.dtype, t, stream)
    return torch.empty_like(t) if dtype is None else torch.empty_like(t, dtype=dtype)


def _sized(name: str, n: int) -> int:
    if n == ctypes.c_size_t(-1).value:
        raise SSDError(3, name)
    return int(n)


def _rows_dim(name: str, t):
    """(product of the leading dimensions, last dimension) of a tensor whose rows lie in its last one."""
    if t.dim() < 1 or t.shape[-1] == 0:
        raise ValueError(f"{name} must have a last dimension of at least 1")
    return t.numel() // t.shape[-1], t.shape[-1]


def ssd_step_beam(state_in, state_out, parent, x, dt, A, B, C, D, *, conv_in=None, conv_out=None, conv_w=None,
                  conv_b=None, dt_bias=None, dt_softplus: int = 0, z=None, y=None, stream=None):
    """The decode step of a beam search: row b of state_out (batch, H, P, N) fp32 is the step from row parent[b]
    (int32, on the GPU) of state_in (src_rows, H, P, N); a parent outside it starts from a zero state. With conv_w
    (H*P, 4) the layer's convolution runs on x, and conv_in (src_rows, H*P, 3) is reordered and shifted into
    conv_out (batch, H*P, 3). Other arguments as ssd_step_fused. Returns y."""
    lib = load()
    if state_in.dim() != 4 or state_out.dim() != 4 or B.dim() != 3:
        raise ValueError("state_in must be (src_rows, H, P, N), state_out (batch, H, P, N) and B (batch, G, N)")
    bsz, H, P, N = state_out.shape
    G, src = B.shape[1], state_in.shape[0]
    st, f32 = x.dtype, torch.float32
    code = _dtype_code(x)
    dev = _device(state_out)
    p_y = _in(dev, "y", y, (bsz, H, P), st)
    if y is None:
        y = _like(x, stream)
        p_y = y.data_ptr()
    rc = lib.ssd_step_beam(
        _in(dev, "state_in", state_in, (src, H, P, N), f32), _in(dev, "state_out", state_out, (bsz, H, P, N), f32),
        _in(dev, "parent", parent, (bsz,), torch.int32), src, _in(dev, "conv_in", conv_in, (src, H * P, 3), st),
        _in(dev, "conv_out", conv_out, (bsz, H * P, 3), st), _in(dev, "x", x, (bsz, H, P), st),
        _in(dev, "conv_w", conv_w, (H * P, 4), f32), _in(dev, "conv_b", conv_b, (H * P,), f32),
        _in(dev, "dt", dt, (bsz, H), st), _in(dev, "dt_bias", dt_bias, (H,), f32), int(dt_softplus),
        _in(dev, "A", A, (H,), f32), _in(dev, "B", B, (bsz, G, N), st), _in(dev, "C", C, (bsz, G, N), st),
        _in(dev, "D", D, (H,), f32), _in(dev, "z", z, (bsz, H, P), st), p_y, bsz, H, P, N, G, code, _stream_on(dev, stream))
    if rc != 0:
        raise SSDError(rc, "ssd_step_beam")
    return y


def ssd_beam_select_workspace_bytes(batch, beams, vocab) -> int:
    return _sized("ssd_beam_select_workspace_bytes", load().ssd_beam_select_workspace_bytes(batch, beams, vocab))


def ssd_beam_select(logits, scores, *, finished=None, eos: int = -1, workspace=None, stream=None):
    """Beam search's choice: logits (batch, beams, vocab) bf16 or fp32, scores (batch, beams) fp32
    log-probabilities (-inf for a beam not in use), finished (batch, beams) bool or uint8, or None.
    Returns (next_scores fp32, parent int32, token int32, next_finished bool), each (batch, beams); parent is a
    row of the batch * beams states, as ssd_step_beam takes it."""
    lib = load()
    if logits.dim() != 3:
        raise ValueError("logits must be (batch, beams, vocab)")
    bsz, K, V = shape = logits.shape
    rows = (bsz, K)
    code = _dtype_code(logits)
    if finished is not None and finished.dtype not in (torch.bool, torch.uint8):
        raise ValueError(f"finished: dtype {finished.dtype}, expected bool or uint8")
    dev = _device(logits)
    p_l, p_s = _first("logits", logits), _in(dev, "scores", scores, rows, torch.float32)
    p_f = None if finished is None else _in(dev, "finished", finished, rows, finished.dtype)
    need = 0 if workspace is not None else ssd_beam_select_workspace_bytes(bsz, K, V)
    workspace, p_w, nbytes = _scratch(workspace, need, logits, dev, stream)
    out = _like(scores, stream)
    parent = _like(scores, stream, torch.int32)
    token = _like(parent, stream)
    done = _like(scores, stream, torch.bool)
    st = lib.ssd_beam_select(p_l, p_s, p_f, int(eos), out.data_ptr(), parent.data_ptr(), token.data_ptr(),
                             done.data_ptr(), bsz, K, V, code, p_w, nbytes, _stream_on(dev, stream))
    if st != 0:
        raise SSDError(st, "ssd_beam_select")
    return out, parent, token, done


def _norm_args(x, weight, residual, residual_out, stream):
    """The checked arguments that both norms share: (rows, dim, codes of x and residual, device, addresses of x,
    weight, residual and residual_out, residual_out)."""
    rows, dim = _rows_dim("x", x)
    shape = x.shape
    code = rcode = _dtype_code(x)
    dev = _device(x)
    p_x, p_w = _first("x", x), _in(dev, "weight", weight, (dim,), torch.float32)
    p_r = p_ro = None
    if residual is None:
        if residual_out is not None:
            raise ValueError("residual_out without a residual")
    else:
        rcode = _dtype_code(residual)
        p_r = _in(dev, "residual", residual, shape, residual.dtype)
        if residual_out is None:
            residual_out = _like(residual, stream)
            p_ro = residual_out.data_ptr()
        else:
            p_ro = _in(dev, "residual_out", residual_out, shape, residual.dtype)
    return rows, dim, code, rcode, dev, p_x, p_w, p_r, p_ro, residual_out


def ssd_rms_norm(x, weight, eps: float, *, residual=None, groups: int = 1, residual_out=None, y=None,
                 want_rstd: bool = False, stream=None):
    """y = h * weight / sqrt(mean(h^2) + eps), h = x + residual, over the last dimension of x (or each of `groups`
    equal pieces of it). residual: x's type or fp32. Returns (y, residual_out, rstd): residual_out is h in
    residual's type (None without one; may be passed as residual itself), rstd (rows..., groups) fp32 for the
    backward pass, or None."""
    lib = load()
    rows, dim, code, rcode, dev, p_x, p_w, p_r, p_ro, residual_out = _norm_args(x, weight, residual, residual_out, stream)
    p_y = _in(dev, "y", y, x.shape, x.dtype)
    if y is None:
        y = _like(x, stream)
        p_y = y.data_ptr()
    rstd = _new((*x.shape[:-1], groups), torch.float32, x, stream) if want_rstd else None
    st = lib.ssd_rms_norm(p_x, p_r, p_w, eps, p_ro, p_y, None if rstd is None else rstd.data_ptr(), rows, dim, groups,
                          code, rcode, _stream_on(dev, stream))
    if st != 0:
        raise SSDError(st, "ssd_rms_norm")
    return y, residual_out, rstd


def _new_mx(x, dim: int, stream):
    return (_new(x.shape, torch.float8_e4m3fn, x, stream),
            _new((*x.shape[:-1], dim // 32), torch.float8_e8m0fnu, x, stream))


def ssd_rms_norm_mx(x, weight, eps: float, *, residual=None, groups: int = 1, residual_out=None, stream=None):
    """ssd_rms_norm with an 8-bit output. Returns (q, scale, residual_out): q float8_e4m3fn like x, scale
    float8_e8m0fnu (..., dim / 32), a power of two for each 32 values of a row."""
    lib = load()
    rows, dim, code, rcode, dev, p_x, p_w, p_r, p_ro, residual_out = _norm_args(x, weight, residual, residual_out, stream)
    q, scale = _new_mx(x, dim, stream)
    st = lib.ssd_rms_norm_mx(p_x, p_r, p_w, eps, p_ro, q.data_ptr(), scale.data_ptr(), rows, dim, groups, code, rcode,
                             _stream_on(dev, stream))
    if st != 0:
        raise SSDError(st, "ssd_rms_norm_mx")
    return q, scale, residual_out


def ssd_mx_quantize(x, *, stream=None):
    """x (..., dim), dim a multiple of 32, in 8 bits: (q float8_e4m3fn, scale float8_e8m0fnu), as ssd_rms_norm_mx."""
    lib = load()
    rows, dim = _rows_dim("x", x)
    code = _dtype_code(x)
    dev = _device(x)
    p_x = _first("x", x)
    q, scale = _new_mx(x, dim, stream)
    st = lib.ssd_mx_quantize(p_x, q.data_ptr(), scale.data_ptr(), rows, dim, code, _stream_on(dev, stream))
    if st != 0:
        raise SSDError(st, "ssd_mx_quantize")
    return q, scale


def ssd_rms_norm_bwd_workspace_bytes(rows, dim, groups, dtype: int, residual_dtype: int) -> int:
    return _sized("ssd_rms_norm_bwd_workspace_bytes",
                  load().ssd_rms_norm_bwd_workspace_bytes(rows, dim, groups, dtype, residual_dtype))


def ssd_rms_norm_bwd(dy, h, weight, rstd, *, d_residual_out=None, groups: int = 1, workspace=None, stream=None):
    """Gradients of ssd_rms_norm: dy like y, h its residual_out (its x, where it had no residual), rstd from it,
    d_residual_out like h or None. Returns (dx, d_residual, dweight): dx in dy's type; d_residual is the same
    gradient in h's type where that differs, else None (dx serves for both); dweight fp32."""
    lib = load()
    rows, dim = _rows_dim("dy", dy)
    shape = dy.shape
    code, rcode = _dtype_code(dy), _dtype_code(h)
    dev = _device(dy)
    need = 0 if workspace is not None else ssd_rms_norm_bwd_workspace_bytes(rows, dim, groups, code, rcode)
    workspace, p_ws, nbytes = _scratch(workspace, need, dy, dev, stream)
    dx = _new(shape, dy.dtype, dy, stream)
    dh = _new(shape, h.dtype, dy, stream) if rcode != code else None
    dw = _new((dim,), torch.float32, dy, stream)
    st = lib.ssd_rms_norm_bwd(
        _first("dy", dy), _in(dev, "h", h, shape, h.dtype),
        _in(dev, "weight", weight, (dim,), torch.float32), _in(dev, "rstd", rstd, (*shape[:-1], groups), torch.float32),
        _in(dev, "d_residual_out", d_residual_out, shape, h.dtype), dx.data_ptr(), None if dh is None else dh.data_ptr(),
        dw.data_ptr(), rows, dim, groups, code, rcode, p_ws, nbytes, _stream_on(dev, stream))
    if st != 0:
        raise SSDError(st, "ssd_rms_norm_bwd")
    return dx, dh, dw


def _act_code(act: str) -> int:
    if act not in ACTS:
        raise ValueError(f"act {act!r}: one of {sorted(ACTS)}")
    return ACTS[act]


def _linear_dims(x, w, what: str):
    """(rows, in, out, shape of y) of a product of x (..., in) and w (out, in)."""
    rows, k = _rows_dim("x", x)
    if w.dim() != 2 or w.shape[1] != k:
        raise ValueError(f"{what}: shape {tuple(w.shape)}, expected (out, {k})")
    n = w.shape[0]
    return rows, k, n, (*x.shape[:-1], n)


def ssd_linear_workspace_bytes(rows, in_, out, dtype: int) -> int:
    return _sized("ssd_linear_workspace_bytes", load().ssd_linear_workspace_bytes(rows, in_, out, dtype))


def ssd_linear(x, w, *, bias=None, act: str = "none", residual=None, y=None, want_preact: bool = False, workspace=None,
               stream=None):
    """y = act(x w^T + bias) + residual: x (..., in) and w (out, in) bf16 or fp32, bias (out) fp32, act "none", "silu"
    or "gelu", residual (..., out) in x's type. Returns (y, preact): preact is x w^T + bias for ssd_linear_bwd, or
    None."""
    lib = load()
    rows, k, n, shape = _linear_dims(x, w, "w")
    st, code, acode = x.dtype, _dtype_code(x), _act_code(act)
    dev = _device(x)
    p_y = _in(dev, "y", y, shape, st)
    if y is None:
        y = _new(shape, st, x, stream)
        p_y = y.data_ptr()
    pre = _new(shape, st, x, stream) if want_preact else None
    need = 0 if workspace is not None else ssd_linear_workspace_bytes(rows, k, n, code)
    workspace, p_ws, nbytes = _scratch(workspace, need, x, dev, stream)
    rc = lib.ssd_linear(_first("x", x), _in(dev, "w", w, (n, k), st),
                        _in(dev, "bias", bias, (n,), torch.float32), acode, _in(dev, "residual", residual, shape, st), p_y,
                        None if pre is None else pre.data_ptr(), rows, k, n, code, p_ws, nbytes, _stream_on(dev, stream))
    if rc != 0:
        raise SSDError(rc, "ssd_linear")
    return y, pre


def ssd_linear_mx_workspace_bytes(rows, in_, out) -> int:
    return _sized("ssd_linear_mx_workspace_bytes", load().ssd_linear_mx_workspace_bytes(rows, in_, out))


def ssd_linear_mx(xq, xscale, wq, wscale, *, bias=None, act: str = "none", residual=None, y=None, workspace=None,
                  stream=None):
    """ssd_linear from 8-bit operands as ssd_rms_norm_mx and ssd_mx_quantize return them: xq (..., in) and wq
    (out, in) float8_e4m3fn, xscale (..., in / 32) and wscale (out, in / 32) float8_e8m0fnu; residual and y bf16.
    Returns y."""
    lib = load()
    rows, k, n, shape = _linear_dims(xq, wq, "wq")
    acode = _act_code(act)
    q8, s8, f32, b16 = torch.float8_e4m3fn, torch.float8_e8m0fnu, torch.float32, torch.bfloat16
    sshape = (*xq.shape[:-1], k // 32)
    dev = _device(xq)
    p_y = _in(dev, "y", y, shape, b16)
    if y is None:
        y = _new(shape, b16, xq, stream)
        p_y = y.data_ptr()
    need = 0 if workspace is not None else ssd_linear_mx_workspace_bytes(rows, k, n)
    workspace, p_ws, nbytes = _scratch(workspace, need, xq, dev, stream)
    rc = lib.ssd_linear_mx(_in(dev, "xq", xq, xq.shape, q8), _in(dev, "xscale", xscale, sshape, s8),
                           _in(dev, "wq", wq, (n, k), q8), _in(dev, "wscale", wscale, (n, k // 32), s8),
                           _in(dev, "bias", bias, (n,), f32), acode, _in(dev, "residual", residual, shape, b16), p_y,
                           rows, k, n, p_ws, nbytes, _stream_on(dev, stream))
    if rc != 0:
        raise SSDError(rc, "ssd_linear_mx")
    return y


def ssd_linear_bwd_workspace_bytes(rows, in_, out, act: str, dtype: int) -> int:
    return _sized("ssd_linear_bwd_workspace_bytes",
                  load().ssd_linear_bwd_workspace_bytes(rows, in_, out, _act_code(act), dtype))


def ssd_linear_bwd(dy, x, w, *, act: str = "none", preact=None, want_x: bool = True, want_w: bool = True,
                   want_bias: bool = False, workspace=None, stream=None):
    """Gradients of ssd_linear: dy (..., out), x (..., in), w (out, in), preact as the forward returned it (act other
    than "none"). Returns (dx, dw, dbias fp32), None for one that is not wanted; the residual's gradient is dy."""
    lib = load()
    rows, k, n, shape = _linear_dims(x, w, "w")
    st, code, acode = x.dtype, _dtype_code(x), _act_code(act)
    if acode and preact is None:
        raise ValueError("act needs preact")
    dev = _device(x)
    dx = _new(x.shape, st, x, stream) if want_x else None
    dw = _new((n, k), st, x, stream) if want_w else None
    db = _new((n,), torch.float32, x, stream) if want_bias else None
    need = 0 if workspace is not None else ssd_linear_bwd_workspace_bytes(rows, k, n, act, code)
    workspace, p_ws, nbytes = _scratch(workspace, need, x, dev, stream)
    rc = lib.ssd_linear_bwd(_in(dev, "dy", dy, shape, st), _first("x", x), _in(dev, "w", w, (n, k), st),
                            acode, _in(dev, "preact", preact, shape, st), _ptr(dx), _ptr(dw), _ptr(db), rows, k, n,
                            code, p_ws, nbytes, _stream_on(dev, stream))
    if rc != 0:
        raise SSDError(rc, "ssd_linear_bwd")
    return dx, dw, db


def raw_call(name: str, *args) -> int:
    """Calls a C entry point with raw integer/pointer arguments; returns its status."""
    return int(getattr(load(), name)(*args))
