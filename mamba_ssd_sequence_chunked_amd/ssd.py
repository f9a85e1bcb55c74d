"""Python binding of the C ABI in include/ssd.h (ctypes).

Argument marshalling only: shapes, dtypes, devices and contiguity are
checked, outputs and the workspace are allocated with torch on the
tensors' device, and the C entry point is called on torch's current HIP
stream.  Every step of the computation runs in the library's HIP kernels;
there is no fallback: without the built library every call raises.
"""
from __future__ import annotations

import contextlib
import ctypes
import os
from typing import Optional, Tuple

import torch

from ._build import LIB_PATH

SSD_F32, SSD_BF16 = 0, 1
_STATUS_OK = 0

_lib = None


class SSDError(RuntimeError):
    """A non-zero status returned by the library."""

    def __init__(self, fn: str, status: int):
        self.status = status
        super().__init__(f"{fn}: {status_string(status)}")


def load_library():
    """Load libssd_mi355x.so (built by __graft_entry__.build()); raise if it is missing."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(
            f"the SSD HIP library is not built ({LIB_PATH} missing); run __graft_entry__.build() "
            "or python -m mamba_ssd_sequence_chunked_amd._build")
    lib = ctypes.CDLL(LIB_PATH)
    vp, fp, i64, i32, sz = ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t
    lib.ssd_status_string.restype = ctypes.c_char_p
    lib.ssd_status_string.argtypes = [i32]
    lib.ssd_abi_version.restype = i32
    lib.ssd_abi_version.argtypes = []
    lib.ssd_num_chunks.restype = i64
    lib.ssd_num_chunks.argtypes = [i64, i64]
    lib.ssd_forward_workspace_bytes.restype = sz
    lib.ssd_forward_workspace_bytes.argtypes = [i64] * 6 + [i32]
    lib.ssd_forward.restype = i32
    lib.ssd_forward.argtypes = [vp] * 9 + [i64] * 7 + [i32, vp, sz, vp]
    lib.ssd_forward_noalloc.restype = i32
    lib.ssd_forward_noalloc.argtypes = [vp] * 9 + [i64] * 7 + [i32, vp]
    lib.ssd_forward_noalloc_scratch_bytes.restype = sz
    lib.ssd_forward_noalloc_scratch_bytes.argtypes = []
    lib.ssd_forward_fused.restype = i32
    lib.ssd_forward_fused.argtypes = [vp] * 9 + [i64] * 6 + [i32, vp]
    lib.ssd_dA_cumsum.restype = i32
    lib.ssd_dA_cumsum.argtypes = [fp] * 4 + [i64] * 4 + [vp]
    lib.ssd_chunk_state.restype = i32
    lib.ssd_chunk_state.argtypes = [vp] * 5 + [i64] * 7 + [i32, vp]
    lib.ssd_state_passing.restype = i32
    lib.ssd_state_passing.argtypes = [vp] * 5 + [i64] * 6 + [i32, vp]
    lib.ssd_chunk_scan.restype = i32
    lib.ssd_chunk_scan.argtypes = [vp] * 8 + [i64] * 7 + [i32, vp]
    lib.ssd_step.restype = i32
    lib.ssd_step.argtypes = [vp] * 8 + [i64] * 5 + [i32, vp]
    lib.ssd_forward_varlen_workspace_bytes.restype = sz
    lib.ssd_forward_varlen_workspace_bytes.argtypes = [i64] * 5 + [i32]
    lib.ssd_forward_varlen.restype = i32
    lib.ssd_forward_varlen.argtypes = [vp] * 7 + [i64] + [vp] * 2 + [i64] * 6 + [i32, vp, sz, vp]
    lib.ssd_backward_workspace_bytes.restype = sz
    lib.ssd_backward_workspace_bytes.argtypes = [i64] * 7 + [i32]
    lib.ssd_backward.restype = i32
    lib.ssd_backward.argtypes = [vp] * 16 + [i64] * 7 + [i32, vp, sz, vp]
    lib.ssd_selective_scan.restype = i32
    lib.ssd_selective_scan.argtypes = [vp] * 9 + [i64] * 4 + [i32, vp]
    lib.ssd_delta_forward_workspace_bytes.restype = sz
    lib.ssd_delta_forward_workspace_bytes.argtypes = [i64] * 6 + [i32]
    lib.ssd_delta_forward.restype = i32
    lib.ssd_delta_forward.argtypes = [vp] * 8 + [i64] * 6 + [i32, vp, sz, vp]
    lib.ssd_delta_forward_varlen_workspace_bytes.restype = sz
    lib.ssd_delta_forward_varlen_workspace_bytes.argtypes = [i64] * 6 + [i32]
    lib.ssd_delta_forward_varlen.restype = i32
    lib.ssd_delta_forward_varlen.argtypes = [vp] * 6 + [i64] + [vp] * 3 + [i64] * 5 + [i32, vp, sz, vp]
    lib.ssd_delta_backward_workspace_bytes.restype = sz
    lib.ssd_delta_backward_workspace_bytes.argtypes = [i64] * 6 + [i32]
    lib.ssd_delta_backward.restype = i32
    lib.ssd_delta_backward.argtypes = [vp] * 14 + [i64] * 6 + [i32, vp, sz, vp]
    lib.ssd_delta_step.restype = i32
    lib.ssd_delta_step.argtypes = [vp] * 7 + [i64] * 5 + [i32, vp]
    lib.ssd_linear_forward_workspace_bytes.restype = sz
    lib.ssd_linear_forward_workspace_bytes.argtypes = [i64] * 6 + [i32]
    lib.ssd_linear_forward.restype = i32
    lib.ssd_linear_forward.argtypes = [vp] * 7 + [i64] * 6 + [i32, vp, sz, vp]
    lib.ssd_linear_forward_varlen_workspace_bytes.restype = sz
    lib.ssd_linear_forward_varlen_workspace_bytes.argtypes = [i64] * 6 + [i32]
    lib.ssd_linear_forward_varlen.restype = i32
    lib.ssd_linear_forward_varlen.argtypes = [vp] * 5 + [i64] + [vp] * 3 + [i64] * 5 + [i32, vp, sz, vp]
    lib.ssd_linear_backward_workspace_bytes.restype = sz
    lib.ssd_linear_backward_workspace_bytes.argtypes = [i64] * 6 + [i32]
    lib.ssd_linear_backward.restype = i32
    lib.ssd_linear_backward.argtypes = [vp] * 12 + [i64] * 6 + [i32, vp, sz, vp]
    lib.ssd_linear_step.restype = i32
    lib.ssd_linear_step.argtypes = [vp] * 2 + [i64] + [vp] * 5 + [i64] * 5 + [i32, vp]
    lib.ssd_state_move.restype = i32
    lib.ssd_state_move.argtypes = [vp] * 3 + [i64] * 4 + [vp]
    _lib = lib
    return lib


def status_string(status: int) -> str:
    return load_library().ssd_status_string(int(status)).decode()


def _check(fn: str, rc: int):
    if rc != _STATUS_OK:
        raise SSDError(fn, rc)


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return SSD_F32
    if t.dtype == torch.bfloat16:
        return SSD_BF16
    raise ValueError(f"x/B/C must be float32 or bfloat16, got {t.dtype}")


def _need(t: Optional[torch.Tensor], name: str, shape, dtype, device) -> None:
    if t is None:
        raise ValueError(f"{name} is required")
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name} must be a torch.Tensor")
    if t.shape != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.dtype != dtype:
        raise ValueError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if device.type != "cuda":
        raise ValueError(f"{name} must be a GPU tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(device) -> ctypes.c_void_p:
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def num_chunks(seqlen: int, chunk_size: int) -> int:
    return int(load_library().ssd_num_chunks(seqlen, chunk_size))


def workspace_bytes(batch, seqlen, nheads, headdim, dstate, chunk_size, dtype_code) -> int:
    return int(load_library().ssd_forward_workspace_bytes(batch, seqlen, nheads, headdim, dstate,
                                                          chunk_size, dtype_code))


def _forward_dims(x, B):
    if x.dim() != 4 or B.dim() != 4:
        raise ValueError("x must be (batch, seqlen, nheads, headdim) and B, C (batch, seqlen, ngroups, dstate)")
    b, L, H, P = x.shape
    G, N = B.shape[2], B.shape[3]
    return b, L, H, P, N, G


def forward(x: torch.Tensor, dt: torch.Tensor, A: torch.Tensor, B: torch.Tensor, C: torch.Tensor,
            D: torch.Tensor, chunk_size: int, init_states: Optional[torch.Tensor] = None,
            workspace: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Chunked (dual) mode: returns (y, final_states); see ssd_forward in include/ssd.h."""
    lib = load_library()
    b, L, H, P, N, G = _forward_dims(x, B)
    dev = x.device
    code = _dtype_code(x)
    _need(x, "x", (b, L, H, P), x.dtype, dev)
    _need(dt, "dt", (b, L, H), torch.float32, dev)
    _need(A, "A", (H,), torch.float32, dev)
    _need(B, "B", (b, L, G, N), x.dtype, dev)
    _need(C, "C", (b, L, G, N), x.dtype, dev)
    _need(D, "D", (H,), torch.float32, dev)
    if init_states is not None:
        _need(init_states, "init_states", (b, H, P, N), torch.float32, dev)
    y = torch.empty_like(x)
    final = torch.empty((b, H, P, N), dtype=torch.float32, device=dev)
    ws_bytes = lib.ssd_forward_workspace_bytes(b, L, H, P, N, chunk_size, code)
    if ws_bytes == 0:
        _check("ssd_forward", -2)
    if workspace is None or workspace.numel() < ws_bytes:
        workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=dev)
    rc = lib.ssd_forward(_ptr(x), _ptr(dt), _ptr(A), _ptr(B), _ptr(C), _ptr(D), _ptr(init_states), _ptr(y),
                         _ptr(final), b, L, H, P, N, G, chunk_size, code, _ptr(workspace),
                         workspace.numel(), _stream(dev))
    _check("ssd_forward", rc)
    return y, final


def forward_noalloc(x: torch.Tensor, dt: torch.Tensor, A: torch.Tensor, B: torch.Tensor, C: torch.Tensor,
                    D: torch.Tensor, chunk_size: int, init_states: Optional[torch.Tensor] = None,
                    y: Optional[torch.Tensor] = None,
                    final_states: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """ssd_forward on the library's static scratch (no workspace; see ssd_forward_noalloc in
    include/ssd.h).  y and final_states may be passed in, so that the call allocates nothing."""
    lib = load_library()
    b, L, H, P, N, G = _forward_dims(x, B)
    dev = x.device
    code = _dtype_code(x)
    _need(x, "x", (b, L, H, P), x.dtype, dev)
    _need(dt, "dt", (b, L, H), torch.float32, dev)
    _need(A, "A", (H,), torch.float32, dev)
    _need(B, "B", (b, L, G, N), x.dtype, dev)
    _need(C, "C", (b, L, G, N), x.dtype, dev)
    _need(D, "D", (H,), torch.float32, dev)
    if init_states is not None:
        _need(init_states, "init_states", (b, H, P, N), torch.float32, dev)
    if y is None:
        y = torch.empty_like(x)
    _need(y, "y", (b, L, H, P), x.dtype, dev)
    if final_states is None:
        final_states = torch.empty((b, H, P, N), dtype=torch.float32, device=dev)
    _need(final_states, "final_states", (b, H, P, N), torch.float32, dev)
    rc = lib.ssd_forward_noalloc(_ptr(x), _ptr(dt), _ptr(A), _ptr(B), _ptr(C), _ptr(D), _ptr(init_states), _ptr(y),
                                 _ptr(final_states), b, L, H, P, N, G, chunk_size, code, _stream(dev))
    _check("ssd_forward_noalloc", rc)
    return y, final_states


def forward_fused(x: torch.Tensor, dt: torch.Tensor, A: torch.Tensor, B: torch.Tensor, C: torch.Tensor,
                  D: torch.Tensor, init_states: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """One pass over the sequence per (batch, head), the state on chip: returns (y, final_states);
    see ssd_forward_fused in include/ssd.h."""
    lib = load_library()
    b, L, H, P, N, G = _forward_dims(x, B)
    dev = x.device
    code = _dtype_code(x)
    _need(x, "x", (b, L, H, P), x.dtype, dev)
    _need(dt, "dt", (b, L, H), torch.float32, dev)
    _need(A, "A", (H,), torch.float32, dev)
    _need(B, "B", (b, L, G, N), x.dtype, dev)
    _need(C, "C", (b, L, G, N), x.dtype, dev)
    _need(D, "D", (H,), torch.float32, dev)
    if init_states is not None:
        _need(init_states, "init_states", (b, H, P, N), torch.float32, dev)
    y = torch.empty_like(x)
    final = torch.empty((b, H, P, N), dtype=torch.float32, device=dev)
    rc = lib.ssd_forward_fused(_ptr(x), _ptr(dt), _ptr(A), _ptr(B), _ptr(C), _ptr(D), _ptr(init_states), _ptr(y),
                               _ptr(final), b, L, H, P, N, G, code, _stream(dev))
    _check("ssd_forward_fused", rc)
    return y, final


def step(state: torch.Tensor, x: torch.Tensor, dt: torch.Tensor, A: torch.Tensor, B: torch.Tensor,
         C: torch.Tensor, D: torch.Tensor, y: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Recurrent mode: advances ``state`` in place by one token and returns y; see ssd_step."""
    lib = load_library()
    if state.dim() != 4 or B.dim() != 3:
        raise ValueError("state must be (batch, nheads, headdim, dstate) and B, C (batch, ngroups, dstate)")
    b, H, P, N = state.shape
    G = B.shape[1]
    dev = state.device
    code = _dtype_code(x)
    _need(state, "state", (b, H, P, N), torch.float32, dev)
    _need(x, "x", (b, H, P), x.dtype, dev)
    _need(dt, "dt", (b, H), torch.float32, dev)
    _need(A, "A", (H,), torch.float32, dev)
    _need(B, "B", (b, G, N), x.dtype, dev)
    _need(C, "C", (b, G, N), x.dtype, dev)
    _need(D, "D", (H,), torch.float32, dev)
    if y is None:
        y = torch.empty_like(x)
    else:
        _need(y, "y", (b, H, P), x.dtype, dev)
    rc = lib.ssd_step(_ptr(state), _ptr(x), _ptr(dt), _ptr(A), _ptr(B), _ptr(C), _ptr(D), _ptr(y), b, H, P, N,
                      G, code, _stream(dev))
    _check("ssd_step", rc)
    return y


def backward(x: torch.Tensor, dt: torch.Tensor, A: torch.Tensor, B: torch.Tensor, C: torch.Tensor,
             D: torch.Tensor, dy: torch.Tensor, chunk_size: int, init_states: Optional[torch.Tensor] = None,
             dfinal: Optional[torch.Tensor] = None) -> dict:
    """Gradients of ``forward`` for dL/dy = dy and dL/d(final_states) = dfinal (None = 0); see
    ssd_backward.  Returns a dict with dx, ddt, dA, dB, dC, dD, dinit (dx, dB, dC in x's dtype)."""
    lib = load_library()
    b, L, H, P, N, G = _forward_dims(x, B)
    dev = x.device
    code = _dtype_code(x)
    _need(x, "x", (b, L, H, P), x.dtype, dev)
    _need(dt, "dt", (b, L, H), torch.float32, dev)
    _need(A, "A", (H,), torch.float32, dev)
    _need(B, "B", (b, L, G, N), x.dtype, dev)
    _need(C, "C", (b, L, G, N), x.dtype, dev)
    _need(D, "D", (H,), torch.float32, dev)
    _need(dy, "dy", (b, L, H, P), x.dtype, dev)
    if init_states is not None:
        _need(init_states, "init_states", (b, H, P, N), torch.float32, dev)
    if dfinal is not None:
        _need(dfinal, "dfinal", (b, H, P, N), torch.float32, dev)
    ws_bytes = lib.ssd_backward_workspace_bytes(b, L, H, P, N, G, chunk_size, code)
    if ws_bytes == 0:
        raise SSDError("ssd_backward_workspace_bytes", -2)
    ws = torch.empty(ws_bytes, dtype=torch.uint8, device=dev)
    out = dict(dx=torch.empty_like(x), ddt=torch.empty_like(dt), dA=torch.empty_like(A), dB=torch.empty_like(B),
               dC=torch.empty_like(C), dD=torch.empty_like(D),
               dinit=torch.empty((b, H, P, N), dtype=torch.float32, device=dev))
    rc = lib.ssd_backward(_ptr(x), _ptr(dt), _ptr(A), _ptr(B), _ptr(C), _ptr(D), _ptr(init_states), _ptr(dy),
                          _ptr(dfinal), _ptr(out["dx"]), _ptr(out["ddt"]), _ptr(out["dA"]), _ptr(out["dB"]),
                          _ptr(out["dC"]), _ptr(out["dD"]), _ptr(out["dinit"]), b, L, H, P, N, G, chunk_size, code,
                          _ptr(ws), ws.numel(), _stream(dev))
    _check("ssd_backward", rc)
    return out


def forward_varlen(x: torch.Tensor, dt: torch.Tensor, A: torch.Tensor, B: torch.Tensor, C: torch.Tensor,
                   D: torch.Tensor, cu_seqlens: torch.Tensor, chunk_size: int) -> Tuple[torch.Tensor, torch.Tensor]:
    """Packed variable-length batch; see ssd_forward_varlen.

    x (T, nheads, headdim); dt (T, nheads) fp32; A, D (nheads,) fp32; B, C (T, ngroups, dstate) in
    x's dtype; cu_seqlens int32 (nseq + 1,) on the same device.  Every sequence starts from a zero
    state.  Returns (y (T, nheads, headdim) in x's dtype, final_states (nseq, nheads, headdim, dstate))."""
    lib = load_library()
    if x.dim() != 3 or B.dim() != 3:
        raise ValueError("x must be (T, nheads, headdim) and B, C (T, ngroups, dstate)")
    T, H, P = x.shape
    G, N = B.shape[1], B.shape[2]
    dev = x.device
    code = _dtype_code(x)
    _need(x, "x", (T, H, P), x.dtype, dev)
    _need(dt, "dt", (T, H), torch.float32, dev)
    _need(A, "A", (H,), torch.float32, dev)
    _need(B, "B", (T, G, N), x.dtype, dev)
    _need(C, "C", (T, G, N), x.dtype, dev)
    _need(D, "D", (H,), torch.float32, dev)
    if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 1:
        raise ValueError("cu_seqlens must be a 1-D tensor of nseq + 1 offsets")
    _need(cu_seqlens, "cu_seqlens", (cu_seqlens.numel(),), torch.int32, dev)
    nseq = cu_seqlens.numel() - 1
    ws_bytes = lib.ssd_forward_varlen_workspace_bytes(T, H, P, N, chunk_size, code)
    if ws_bytes == 0:
        raise SSDError("ssd_forward_varlen_workspace_bytes", -2)
    workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=dev)
    y = torch.empty_like(x)
    final = torch.empty((nseq, H, P, N), dtype=torch.float32, device=dev)
    rc = lib.ssd_forward_varlen(_ptr(x), _ptr(dt), _ptr(A), _ptr(B), _ptr(C), _ptr(D), _ptr(cu_seqlens), nseq,
                                _ptr(y), _ptr(final), T, H, P, N, G, chunk_size, code, _ptr(workspace),
                                workspace.numel(), _stream(dev))
    _check("ssd_forward_varlen", rc)
    return y, final


def selective_scan(x: torch.Tensor, delta: torch.Tensor, A: torch.Tensor, B: torch.Tensor, C: torch.Tensor,
                   D: torch.Tensor, init_states: Optional[torch.Tensor] = None
                   ) -> Tuple[torch.Tensor, torch.Tensor]:
    """The Mamba-1 selective scan (per-channel diagonal decays); see ssd_selective_scan.

    x (batch, seqlen, dim); delta (batch, seqlen, dim) fp32; A (dim, dstate) fp32;
    B, C (batch, seqlen, dstate) in x's dtype; D (dim,) fp32; init_states (batch, dim, dstate)
    fp32 or None.  Returns (y in x's dtype, final_states fp32)."""
    lib = load_library()
    if x.dim() != 3 or A.dim() != 2:
        raise ValueError("x must be (batch, seqlen, dim) and A (dim, dstate)")
    b, L, Dm = x.shape
    N = A.shape[1]
    dev = x.device
    code = _dtype_code(x)
    _need(x, "x", (b, L, Dm), x.dtype, dev)
    _need(delta, "delta", (b, L, Dm), torch.float32, dev)
    _need(A, "A", (Dm, N), torch.float32, dev)
    _need(B, "B", (b, L, N), x.dtype, dev)
    _need(C, "C", (b, L, N), x.dtype, dev)
    _need(D, "D", (Dm,), torch.float32, dev)
    if init_states is not None:
        _need(init_states, "init_states", (b, Dm, N), torch.float32, dev)
    y = torch.empty_like(x)
    final = torch.empty((b, Dm, N), dtype=torch.float32, device=dev)
    rc = lib.ssd_selective_scan(_ptr(x), _ptr(delta), _ptr(A), _ptr(B), _ptr(C), _ptr(D), _ptr(init_states),
                                _ptr(y), _ptr(final), b, L, Dm, N, code, _stream(dev))
    _check("ssd_selective_scan", rc)
    return y, final


# --- the gated delta rule ----------------------------------------------------------------------

def _on_device(device):
    """The device the tensors are on made current for the launch, if it is not."""
    return contextlib.nullcontext() if torch.cuda.current_device() == device.index else torch.cuda.device(device)


def _delta_need(v, g, beta, k, q, lead, H, P, N, G, dev):
    _need(v, "v", (*lead, H, P), v.dtype, dev)
    _need(g, "g", (*lead, H), torch.float32, dev)
    _need(beta, "beta", (*lead, H), torch.float32, dev)
    _need(k, "k", (*lead, G, N), v.dtype, dev)
    _need(q, "q", (*lead, G, N), v.dtype, dev)


def delta_forward(v: torch.Tensor, g: torch.Tensor, beta: torch.Tensor, k: torch.Tensor, q: torch.Tensor,
                  init_states: Optional[torch.Tensor] = None,
                  workspace: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """The gated delta rule over whole sequences: returns (y, final_states); see ssd_delta_forward.

    v (batch, seqlen, nheads, headdim) in bf16 or fp32; g (log decays) and beta (batch, seqlen, nheads)
    fp32; k, q (batch, seqlen, ngroups, dstate) in v's dtype; init_states (batch, nheads, headdim, dstate)
    fp32 or None.  A workspace (uint8, ssd_delta_forward_workspace_bytes() long) may be passed in."""
    lib = load_library()
    if v.dim() != 4 or k.dim() != 4:
        raise ValueError("v must be (batch, seqlen, nheads, headdim) and k, q (batch, seqlen, ngroups, dstate)")
    b, L, H, P = v.shape
    G, N = k.shape[2], k.shape[3]
    dev = v.device
    code = _dtype_code(v)
    _delta_need(v, g, beta, k, q, (b, L), H, P, N, G, dev)
    if init_states is not None:
        _need(init_states, "init_states", (b, H, P, N), torch.float32, dev)
    ws_bytes = lib.ssd_delta_forward_workspace_bytes(b, L, H, P, N, G, code)
    if ws_bytes == 0:
        raise SSDError("ssd_delta_forward_workspace_bytes", -2)
    if workspace is None:
        workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=dev)
    else:
        _need(workspace, "workspace", (workspace.numel(),), torch.uint8, dev)
    y = torch.empty_like(v)
    final = torch.empty((b, H, P, N), dtype=torch.float32, device=dev)
    with _on_device(dev):
        rc = lib.ssd_delta_forward(_ptr(v), _ptr(g), _ptr(beta), _ptr(k), _ptr(q), _ptr(init_states), _ptr(y),
                                   _ptr(final), b, L, H, P, N, G, code, _ptr(workspace), workspace.numel(),
                                   _stream(dev))
    _check("ssd_delta_forward", rc)
    return y, final


def delta_forward_varlen(v: torch.Tensor, g: torch.Tensor, beta: torch.Tensor, k: torch.Tensor, q: torch.Tensor,
                         cu_seqlens: torch.Tensor, init_states: Optional[torch.Tensor] = None
                         ) -> Tuple[torch.Tensor, torch.Tensor]:
    """Packed variable-length batch of the gated delta rule; see ssd_delta_forward_varlen.

    v (T, nheads, headdim); g, beta (T, nheads) fp32; k, q (T, ngroups, dstate) in v's dtype; cu_seqlens
    int32 (nseq + 1,) on the same device; init_states (nseq, nheads, headdim, dstate) fp32 or None.
    Returns (y in v's dtype, final_states (nseq, nheads, headdim, dstate))."""
    lib = load_library()
    if v.dim() != 3 or k.dim() != 3:
        raise ValueError("v must be (T, nheads, headdim) and k, q (T, ngroups, dstate)")
    T, H, P = v.shape
    G, N = k.shape[1], k.shape[2]
    dev = v.device
    code = _dtype_code(v)
    _delta_need(v, g, beta, k, q, (T,), H, P, N, G, dev)
    if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 1:
        raise ValueError("cu_seqlens must be a 1-D tensor of nseq + 1 offsets")
    _need(cu_seqlens, "cu_seqlens", (cu_seqlens.numel(),), torch.int32, dev)
    nseq = cu_seqlens.numel() - 1
    if init_states is not None:
        _need(init_states, "init_states", (nseq, H, P, N), torch.float32, dev)
    ws_bytes = lib.ssd_delta_forward_varlen_workspace_bytes(T, nseq, H, P, N, G, code)
    if ws_bytes == 0:
        raise SSDError("ssd_delta_forward_varlen_workspace_bytes", -2)
    workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=dev)
    y = torch.empty_like(v)
    final = torch.empty((nseq, H, P, N), dtype=torch.float32, device=dev)
    with _on_device(dev):
        rc = lib.ssd_delta_forward_varlen(_ptr(v), _ptr(g), _ptr(beta), _ptr(k), _ptr(q), _ptr(cu_seqlens), nseq,
                                          _ptr(init_states), _ptr(y), _ptr(final), T, H, P, N, G, code,
                                          _ptr(workspace), workspace.numel(), _stream(dev))
    _check("ssd_delta_forward_varlen", rc)
    return y, final


def delta_backward(v: torch.Tensor, g: torch.Tensor, beta: torch.Tensor, k: torch.Tensor, q: torch.Tensor,
                   dy: torch.Tensor, init_states: Optional[torch.Tensor] = None,
                   dfinal: Optional[torch.Tensor] = None) -> dict:
    """Gradients of ``delta_forward`` for dL/dy = dy and dL/d(final_states) = dfinal (None = 0); see
    ssd_delta_backward.  Returns a dict with dv, dg, dbeta, dk, dq, dinit (dv, dk, dq in v's dtype)."""
    lib = load_library()
    if v.dim() != 4 or k.dim() != 4:
        raise ValueError("v must be (batch, seqlen, nheads, headdim) and k, q (batch, seqlen, ngroups, dstate)")
    b, L, H, P = v.shape
    G, N = k.shape[2], k.shape[3]
    dev = v.device
    code = _dtype_code(v)
    _delta_need(v, g, beta, k, q, (b, L), H, P, N, G, dev)
    _need(dy, "dy", (b, L, H, P), v.dtype, dev)
    if init_states is not None:
        _need(init_states, "init_states", (b, H, P, N), torch.float32, dev)
    if dfinal is not None:
        _need(dfinal, "dfinal", (b, H, P, N), torch.float32, dev)
    ws_bytes = lib.ssd_delta_backward_workspace_bytes(b, L, H, P, N, G, code)
    if ws_bytes == 0:
        raise SSDError("ssd_delta_backward_workspace_bytes", -2)
    ws = torch.empty(ws_bytes, dtype=torch.uint8, device=dev)
    out = dict(dv=torch.empty_like(v), dg=torch.empty_like(g), dbeta=torch.empty_like(beta), dk=torch.empty_like(k),
               dq=torch.empty_like(q), dinit=torch.empty((b, H, P, N), dtype=torch.float32, device=dev))
    with _on_device(dev):
        rc = lib.ssd_delta_backward(_ptr(v), _ptr(g), _ptr(beta), _ptr(k), _ptr(q), _ptr(init_states), _ptr(dy),
                                    _ptr(dfinal), _ptr(out["dv"]), _ptr(out["dg"]), _ptr(out["dbeta"]),
                                    _ptr(out["dk"]), _ptr(out["dq"]), _ptr(out["dinit"]), b, L, H, P, N, G, code,
                                    _ptr(ws), ws.numel(), _stream(dev))
    _check("ssd_delta_backward", rc)
    return out


def delta_step(state: torch.Tensor, v: torch.Tensor, g: torch.Tensor, beta: torch.Tensor, k: torch.Tensor,
               q: torch.Tensor, y: Optional[torch.Tensor] = None) -> torch.Tensor:
    """One token of the gated delta rule: advances ``state`` in place and returns y; see ssd_delta_step.

    state (batch, nheads, headdim, dstate) fp32; v (batch, nheads, headdim) in bf16 or fp32; g, beta
    (batch, nheads) fp32; k, q (batch, ngroups, dstate) in v's dtype."""
    lib = load_library()
    if state.dim() != 4 or k.dim() != 3:
        raise ValueError("state must be (batch, nheads, headdim, dstate) and k, q (batch, ngroups, dstate)")
    b, H, P, N = state.shape
    G = k.shape[1]
    dev = state.device
    code = _dtype_code(v)
    _need(state, "state", (b, H, P, N), torch.float32, dev)
    _delta_need(v, g, beta, k, q, (b,), H, P, N, G, dev)
    if y is None:
        y = torch.empty_like(v)
    else:
        _need(y, "y", (b, H, P), v.dtype, dev)
    with _on_device(dev):
        rc = lib.ssd_delta_step(_ptr(state), _ptr(v), _ptr(g), _ptr(beta), _ptr(k), _ptr(q), _ptr(y), b, H, P, N, G,
                                code, _stream(dev))
    _check("ssd_delta_step", rc)
    return y


# --- linear attention with a decay for each head, and pools of states --------------------------

def _is(t, shape, dtype, index) -> bool:
    """Whether t is what _need asks for, on GPU number index; without its messages, for the calls whose time is the host's."""
    return t.dtype is dtype and t.shape == shape and t.get_device() == index and t.is_contiguous()


def _linear_need(v, g, k, q, lead, H, P, N, G, dev):
    _need(v, "v", (*lead, G, P), v.dtype, dev)
    _need(g, "g", (H,), torch.float32, dev)
    _need(k, "k", (*lead, G, N), v.dtype, dev)
    _need(q, "q", (*lead, H, N), v.dtype, dev)


def linear_forward(v: torch.Tensor, g: torch.Tensor, k: torch.Tensor, q: torch.Tensor,
                   init_states: Optional[torch.Tensor] = None,
                   workspace: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Linear attention with a decay for each head over whole sequences: returns (y, final_states); see ssd_linear_forward.

    v (batch, seqlen, ngroups, headdim) in bf16 or fp32; g (nheads,) fp32, the log decays; k (batch, seqlen, ngroups,
    dstate) and q (batch, seqlen, nheads, dstate) in v's dtype; init_states (batch, nheads, headdim, dstate) fp32 or
    None.  A workspace (uint8, ssd_linear_forward_workspace_bytes() long) may be passed in."""
    lib = load_library()
    if v.dim() != 4 or q.dim() != 4:
        raise ValueError("v must be (batch, seqlen, ngroups, headdim) and q (batch, seqlen, nheads, dstate)")
    b, L, G, P = v.shape
    H, N = q.shape[2], q.shape[3]
    dev = v.device
    code = _dtype_code(v)
    _linear_need(v, g, k, q, (b, L), H, P, N, G, dev)
    if init_states is not None:
        _need(init_states, "init_states", (b, H, P, N), torch.float32, dev)
    ws_bytes = lib.ssd_linear_forward_workspace_bytes(b, L, H, P, N, G, code)
    if ws_bytes == 0:
        raise SSDError("ssd_linear_forward_workspace_bytes", -2)
    if workspace is None:
        workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=dev)
    else:
        _need(workspace, "workspace", (workspace.numel(),), torch.uint8, dev)
    y = torch.empty((b, L, H, P), dtype=v.dtype, device=dev)
    final = torch.empty((b, H, P, N), dtype=torch.float32, device=dev)
    with _on_device(dev):
        rc = lib.ssd_linear_forward(_ptr(v), _ptr(g), _ptr(k), _ptr(q), _ptr(init_states), _ptr(y), _ptr(final), b, L,
                                    H, P, N, G, code, _ptr(workspace), workspace.numel(), _stream(dev))
    _check("ssd_linear_forward", rc)
    return y, final


def linear_forward_varlen(v: torch.Tensor, g: torch.Tensor, k: torch.Tensor, q: torch.Tensor, cu_seqlens: torch.Tensor,
                          init_states: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Packed variable-length batch of linear attention; see ssd_linear_forward_varlen.

    v (T, ngroups, headdim); g (nheads,) fp32; k (T, ngroups, dstate), q (T, nheads, dstate) in v's dtype; cu_seqlens
    int32 (nseq + 1,) on the same device; init_states (nseq, nheads, headdim, dstate) fp32 or None.
    Returns (y (T, nheads, headdim) in v's dtype, final_states (nseq, nheads, headdim, dstate)); y of tokens behind
    cu_seqlens[nseq] is not set."""
    lib = load_library()
    if v.dim() != 3 or q.dim() != 3:
        raise ValueError("v must be (T, ngroups, headdim) and q (T, nheads, dstate)")
    T, G, P = v.shape
    H, N = q.shape[1], q.shape[2]
    dev = v.device
    code = _dtype_code(v)
    _linear_need(v, g, k, q, (T,), H, P, N, G, dev)
    if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 1:
        raise ValueError("cu_seqlens must be a 1-D tensor of nseq + 1 offsets")
    _need(cu_seqlens, "cu_seqlens", (cu_seqlens.numel(),), torch.int32, dev)
    nseq = cu_seqlens.numel() - 1
    if init_states is not None:
        _need(init_states, "init_states", (nseq, H, P, N), torch.float32, dev)
    ws_bytes = lib.ssd_linear_forward_varlen_workspace_bytes(T, nseq, H, P, N, G, code)
    if ws_bytes == 0:
        raise SSDError("ssd_linear_forward_varlen_workspace_bytes", -2)
    workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=dev)
    y = torch.empty((T, H, P), dtype=v.dtype, device=dev)
    final = torch.empty((nseq, H, P, N), dtype=torch.float32, device=dev)
    with _on_device(dev):
        rc = lib.ssd_linear_forward_varlen(_ptr(v), _ptr(g), _ptr(k), _ptr(q), _ptr(cu_seqlens), nseq,
                                           _ptr(init_states), _ptr(y), _ptr(final), T, H, P, N, G, code,
                                           _ptr(workspace), workspace.numel(), _stream(dev))
    _check("ssd_linear_forward_varlen", rc)
    return y, final


def linear_backward(v: torch.Tensor, g: torch.Tensor, k: torch.Tensor, q: torch.Tensor, dy: torch.Tensor,
                    init_states: Optional[torch.Tensor] = None, dfinal: Optional[torch.Tensor] = None) -> dict:
    """Gradients of ``linear_forward`` for dL/dy = dy and dL/d(final_states) = dfinal (None = 0); see
    ssd_linear_backward.  Returns a dict with dv, dg, dk, dq, dinit (dv, dk, dq in v's dtype)."""
    lib = load_library()
    if v.dim() != 4 or q.dim() != 4:
        raise ValueError("v must be (batch, seqlen, ngroups, headdim) and q (batch, seqlen, nheads, dstate)")
    b, L, G, P = v.shape
    H, N = q.shape[2], q.shape[3]
    dev = v.device
    code = _dtype_code(v)
    _linear_need(v, g, k, q, (b, L), H, P, N, G, dev)
    _need(dy, "dy", (b, L, H, P), v.dtype, dev)
    if init_states is not None:
        _need(init_states, "init_states", (b, H, P, N), torch.float32, dev)
    if dfinal is not None:
        _need(dfinal, "dfinal", (b, H, P, N), torch.float32, dev)
    ws_bytes = lib.ssd_linear_backward_workspace_bytes(b, L, H, P, N, G, code)
    if ws_bytes == 0:
        raise SSDError("ssd_linear_backward_workspace_bytes", -2)
    ws = torch.empty(ws_bytes, dtype=torch.uint8, device=dev)
    out = dict(dv=torch.empty_like(v), dg=torch.empty_like(g), dk=torch.empty_like(k), dq=torch.empty_like(q),
               dinit=torch.empty((b, H, P, N), dtype=torch.float32, device=dev))
    with _on_device(dev):
        rc = lib.ssd_linear_backward(_ptr(v), _ptr(g), _ptr(k), _ptr(q), _ptr(init_states), _ptr(dy), _ptr(dfinal),
                                     _ptr(out["dv"]), _ptr(out["dg"]), _ptr(out["dk"]), _ptr(out["dq"]),
                                     _ptr(out["dinit"]), b, L, H, P, N, G, code, _ptr(ws), ws.numel(), _stream(dev))
    _check("ssd_linear_backward", rc)
    return out


def linear_step(state: torch.Tensor, v: torch.Tensor, g: torch.Tensor, k: torch.Tensor, q: torch.Tensor,
                slots: Optional[torch.Tensor] = None, y: Optional[torch.Tensor] = None) -> torch.Tensor:
    """One token of linear attention: advances ``state`` in place and returns y; see ssd_linear_step.

    state (nslots, nheads, headdim, dstate) fp32; v (batch, ngroups, headdim) in bf16 or fp32; g (nheads,) fp32; k
    (batch, ngroups, dstate) and q (batch, nheads, dstate) in v's dtype.  slots int32 (batch,): row i advances
    state[slots[i]], a row with a slot out of range (-1) none, and its y is zero; None: nslots = batch, row i has state[i]."""
    lib = load_library()
    if state.dim() != 4 or v.dim() != 3:
        raise ValueError("state must be (nslots, nheads, headdim, dstate) and v (batch, ngroups, headdim)")
    n, H, P, N = state.shape
    b, G = v.shape[0], v.shape[1]
    dev, T = state.device, v.dtype
    i = state.get_device()
    code = _dtype_code(v)
    f32 = torch.float32
    if not (i >= 0 and _is(state, (b if slots is None else n, H, P, N), f32, i) and _is(v, (b, G, P), T, i)
            and _is(g, (H,), f32, i) and _is(k, (b, G, N), T, i) and _is(q, (b, H, N), T, i)
            and (slots is None or _is(slots, (b,), torch.int32, i)) and (y is None or _is(y, (b, H, P), T, i))):
        _need(state, "state", (b if slots is None else n, H, P, N), f32, dev)
        _linear_need(v, g, k, q, (b,), H, P, N, G, dev)
        if slots is not None:
            _need(slots, "slots", (b,), torch.int32, dev)
        if y is not None:
            _need(y, "y", (b, H, P), T, dev)
    if y is None:
        y = torch.empty((b, H, P), dtype=T, device=dev)
    with _on_device(dev):
        rc = lib.ssd_linear_step(state.data_ptr(), None if slots is None else slots.data_ptr(), n, v.data_ptr(),
                                 g.data_ptr(), k.data_ptr(), q.data_ptr(), y.data_ptr(), b, H, P, N, G, code, _stream(dev))
    _check("ssd_linear_step", rc)
    return y


def state_move(states: torch.Tensor, src: torch.Tensor, source: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Copies, forks, reorders, compacts or frees the states of a pool by one map of slots; see ssd_state_move.

    states (nslots, nheads, headdim, dstate) or (nlayers, nslots, nheads, headdim, dstate) fp32, changed in place and
    returned; src int32 (nslots,): slot i becomes source[src[i]], zeros where src[i] is -1, and stays otherwise.  source:
    another pool of the same layers and state sizes, or None: the pool itself, as it was before the call (then at most 2048
    slots: a larger pool moves through a buffer, in two calls)."""
    lib = load_library()
    if states.dim() not in (4, 5):
        raise ValueError("states must be ([nlayers,] nslots, nheads, headdim, dstate)")
    lead, n, one = states.shape[:-4], states.shape[-4], states.shape[-3:]
    dev = states.device
    i = states.get_device()
    if not (i >= 0 and _is(states, states.shape, torch.float32, i) and _is(src, (n,), torch.int32, i)):
        _need(states, "states", states.shape, torch.float32, dev)
        _need(src, "src", (n,), torch.int32, dev)
    m = n
    if source is not None:
        if source.dim() != states.dim():
            raise ValueError("source must have as many dimensions as states")
        m = source.shape[-4]
        _need(source, "source", (*lead, m, *one), torch.float32, dev)
    layers = lead[0] if lead else 1
    with _on_device(dev):
        rc = lib.ssd_state_move(states.data_ptr(), None if source is None else source.data_ptr(), src.data_ptr(), layers,
                                n, m, one[0] * one[1] * one[2], _stream(dev))
    _check("ssd_state_move", rc)
    return states


# --- the four stages of the chunked mode, one entry point each ---------------------------------

def dA_cumsum(dt: torch.Tensor, A: torch.Tensor, chunk_size: int) -> Tuple[torch.Tensor, torch.Tensor]:
    """Stage 1: returns (dA_cs, dt_chunked), both (batch, nheads, nchunks, chunk_size) float32."""
    lib = load_library()
    if dt.dim() != 3:
        raise ValueError("dt must be (batch, seqlen, nheads)")
    b, L, H = dt.shape
    dev = dt.device
    _need(dt, "dt", (b, L, H), torch.float32, dev)
    _need(A, "A", (H,), torch.float32, dev)
    nc = num_chunks(L, chunk_size)
    if nc < 0:
        _check("ssd_dA_cumsum", -2)
    cs = torch.empty((b, H, nc, chunk_size), dtype=torch.float32, device=dev)
    dtc = torch.empty_like(cs)
    rc = lib.ssd_dA_cumsum(_ptr(dt), _ptr(A), _ptr(cs), _ptr(dtc), b, L, H, chunk_size, _stream(dev))
    _check("ssd_dA_cumsum", rc)
    return cs, dtc


def chunk_state(x: torch.Tensor, B: torch.Tensor, dt_chunked: torch.Tensor, dA_cs: torch.Tensor,
                chunk_size: int) -> torch.Tensor:
    """Stage 2: returns chunk_states (batch, nchunks, nheads, headdim, dstate) float32."""
    lib = load_library()
    b, L, H, P, N, G = _forward_dims(x, B)
    dev = x.device
    code = _dtype_code(x)
    nc = num_chunks(L, chunk_size)
    _need(x, "x", (b, L, H, P), x.dtype, dev)
    _need(B, "B", (b, L, G, N), x.dtype, dev)
    _need(dt_chunked, "dt_chunked", (b, H, nc, chunk_size), torch.float32, dev)
    _need(dA_cs, "dA_cs", (b, H, nc, chunk_size), torch.float32, dev)
    out = torch.empty((b, nc, H, P, N), dtype=torch.float32, device=dev)
    rc = lib.ssd_chunk_state(_ptr(x), _ptr(B), _ptr(dt_chunked), _ptr(dA_cs), _ptr(out), b, L, H, P, N, G,
                             chunk_size, code, _stream(dev))
    _check("ssd_chunk_state", rc)
    return out


def state_passing(chunk_states: torch.Tensor, dA_cs: torch.Tensor, init_states: Optional[torch.Tensor],
                  seqlen: int, chunk_size: int, dtype: torch.dtype) -> Tuple[torch.Tensor, torch.Tensor]:
    """Stage 3: returns (entry_states (batch, nchunks, nheads, headdim, dstate) in ``dtype``,
    final_states (batch, nheads, headdim, dstate) float32)."""
    lib = load_library()
    b, nc, H, P, N = chunk_states.shape
    dev = chunk_states.device
    code = SSD_BF16 if dtype == torch.bfloat16 else SSD_F32
    _need(chunk_states, "chunk_states", (b, nc, H, P, N), torch.float32, dev)
    _need(dA_cs, "dA_cs", (b, H, nc, chunk_size), torch.float32, dev)
    if num_chunks(seqlen, chunk_size) != nc:
        raise ValueError("chunk_states does not match seqlen / chunk_size")
    if init_states is not None:
        _need(init_states, "init_states", (b, H, P, N), torch.float32, dev)
    entry = torch.empty((b, nc, H, P, N), dtype=dtype, device=dev)
    final = torch.empty((b, H, P, N), dtype=torch.float32, device=dev)
    rc = lib.ssd_state_passing(_ptr(chunk_states), _ptr(dA_cs), _ptr(init_states), _ptr(entry), _ptr(final), b,
                               seqlen, H, P, N, chunk_size, code, _stream(dev))
    _check("ssd_state_passing", rc)
    return entry, final


def chunk_scan(x: torch.Tensor, B: torch.Tensor, C: torch.Tensor, dt_chunked: torch.Tensor,
               dA_cs: torch.Tensor, entry_states: torch.Tensor, D: torch.Tensor, chunk_size: int) -> torch.Tensor:
    """Stage 4: returns y (batch, seqlen, nheads, headdim) in x's dtype."""
    lib = load_library()
    b, L, H, P, N, G = _forward_dims(x, B)
    dev = x.device
    code = _dtype_code(x)
    nc = num_chunks(L, chunk_size)
    _need(x, "x", (b, L, H, P), x.dtype, dev)
    _need(B, "B", (b, L, G, N), x.dtype, dev)
    _need(C, "C", (b, L, G, N), x.dtype, dev)
    _need(dt_chunked, "dt_chunked", (b, H, nc, chunk_size), torch.float32, dev)
    _need(dA_cs, "dA_cs", (b, H, nc, chunk_size), torch.float32, dev)
    _need(entry_states, "entry_states", (b, nc, H, P, N), x.dtype, dev)
    _need(D, "D", (H,), torch.float32, dev)
    y = torch.empty_like(x)
    rc = lib.ssd_chunk_scan(_ptr(x), _ptr(B), _ptr(C), _ptr(dt_chunked), _ptr(dA_cs), _ptr(entry_states), _ptr(D),
                            _ptr(y), b, L, H, P, N, G, chunk_size, code, _stream(dev))
    _check("ssd_chunk_scan", rc)
    return y
