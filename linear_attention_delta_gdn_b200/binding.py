"""ctypes binding of libgdn2.so (the C ABI declared in include/gdn2.h).

Argument marshalling only: every step of the operator runs in the library's
CUDA kernels. torch supplies device memory (outputs and the workspace are
allocated as torch tensors) and the current CUDA stream. There is no CPU or
library fallback: if ``libgdn2.so`` is missing or a tensor is not on a CUDA
device, these functions raise.

Names mirror the C entry points: :func:`gdn2_fwd`, :func:`gdn2_bwd`,
:func:`gdn2_decode_step`, :func:`gdn2_workspace_size`.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

import torch

_DEBUG_BUILD = os.environ.get("GDN2_DEBUG", "") not in ("", "0")
#: the library this process loads: the debug build (index checks, see build.py) when GDN2_DEBUG is set
_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)),
                         "libgdn2_debug.so" if _DEBUG_BUILD else "libgdn2.so")
_lib = None

GDN2_F32, GDN2_BF16 = 0, 1
GDN2_OP_FWD, GDN2_OP_FWD_SAVE, GDN2_OP_BWD, GDN2_OP_MAP = 0, 1, 2, 3
GDN2_OK, GDN2_ERR_INVALID, GDN2_ERR_TIMEOUT = 0, 1, 5
GDN2_ERR_UNSUPPORTED = 2
STATUS = {0: "GDN2_OK", 1: "GDN2_ERR_INVALID", 2: "GDN2_ERR_UNSUPPORTED", 3: "GDN2_ERR_WORKSPACE",
          4: "GDN2_ERR_CUDA", 5: "GDN2_ERR_TIMEOUT"}

#: exported symbols, as declared in include/gdn2.h
EXPORTS = ("gdn2_workspace_size", "gdn2_fwd", "gdn2_bwd", "gdn2_decode_step", "gdn2_status_string",
           "gdn2_last_error", "gdn2_version", "gdn2_bwd_no_alloc", "gdn2_no_alloc_scratch_bytes",
           "gdn2_trace_enable", "gdn2_trace_read", "gdn2_device_status", "gdn2_beta_workspace_size",
           "gdn2_beta_fwd", "gdn2_beta_bwd", "gdn2_varlen_workspace_size", "gdn2_varlen_fwd", "gdn2_varlen_bwd",
           "gdn2_fwd_map", "gdn2_bwd_map", "gdn2_state_affine", "gdn2_layer_gates_fwd", "gdn2_layer_gates_bwd",
           "gdn2_linear_workspace_size", "gdn2_linear_varlen_workspace_size", "gdn2_linear_fwd", "gdn2_linear_bwd",
           "gdn2_linear_varlen_fwd", "gdn2_linear_varlen_bwd", "gdn2_linear_decode_step",
           "gdn2_qk_norm_rope_workspace_size", "gdn2_qk_norm_rope_fwd", "gdn2_qk_norm_rope_bwd")
GDN2_GATE_KDA, GDN2_GATE_GDN = 1, 2


class Gdn2Error(RuntimeError):
    def __init__(self, fn, status, detail):
        super().__init__("%s -> %s: %s" % (fn, STATUS.get(status, status), detail))
        self.status = status


def lib(path: Optional[str] = None) -> ctypes.CDLL:
    """Load libgdn2.so (built by ``python -m linear_attention_delta_gdn_b200.build``)."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    p = path or _LIB_PATH
    if not os.path.exists(p):
        raise FileNotFoundError("%s is missing: build it with `python -m linear_attention_delta_gdn_b200.build`" % p)
    L = ctypes.CDLL(p)
    P, I, Z = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
    L.gdn2_workspace_size.argtypes = [I] * 8
    L.gdn2_workspace_size.restype = Z
    L.gdn2_fwd.argtypes = [P] * 9 + [I] * 8 + [P, Z, P]
    L.gdn2_fwd.restype = I
    L.gdn2_bwd.argtypes = [P] * 16 + [I] * 8 + [P, Z, P]
    L.gdn2_bwd.restype = I
    L.gdn2_decode_step.argtypes = [P] * 8 + [I] * 5 + [P]
    L.gdn2_decode_step.restype = I
    L.gdn2_status_string.argtypes = [I]
    L.gdn2_status_string.restype = ctypes.c_char_p
    L.gdn2_last_error.argtypes = []
    L.gdn2_last_error.restype = ctypes.c_char_p
    L.gdn2_version.argtypes = []
    L.gdn2_version.restype = I
    L.gdn2_bwd_no_alloc.argtypes = [P] * 16 + [I] * 7 + [P]
    L.gdn2_bwd_no_alloc.restype = I
    L.gdn2_no_alloc_scratch_bytes.argtypes = []
    L.gdn2_no_alloc_scratch_bytes.restype = Z
    L.gdn2_beta_workspace_size.argtypes = [I] * 9
    L.gdn2_beta_workspace_size.restype = Z
    L.gdn2_beta_fwd.argtypes = [I] + [P] * 8 + [I] * 8 + [P, Z, P]
    L.gdn2_beta_fwd.restype = I
    L.gdn2_beta_bwd.argtypes = [I] + [P] * 14 + [I] * 8 + [P, Z, P]
    L.gdn2_beta_bwd.restype = I
    LL = ctypes.c_longlong
    L.gdn2_varlen_workspace_size.argtypes = [I] * 8
    L.gdn2_varlen_workspace_size.restype = Z
    L.gdn2_varlen_fwd.argtypes = [P] * 7 + [I, I, LL] + [P] * 3 + [I] * 6 + [P, Z, P]
    L.gdn2_varlen_fwd.restype = I
    L.gdn2_varlen_bwd.argtypes = [P] * 7 + [I, I, LL] + [P] * 10 + [I] * 6 + [P, Z, P]
    L.gdn2_varlen_bwd.restype = I
    L.gdn2_fwd_map.argtypes = [P] * 8 + [I] * 7 + [P, Z, P]
    L.gdn2_fwd_map.restype = I
    L.gdn2_bwd_map.argtypes = [P] * 9 + [I] * 7 + [P, Z, P]
    L.gdn2_bwd_map.restype = I
    L.gdn2_state_affine.argtypes = [P] * 4 + [I] * 4 + [P]
    L.gdn2_state_affine.restype = I
    L.gdn2_layer_gates_fwd.argtypes = [P] * 8 + [I] * 6 + [P]
    L.gdn2_layer_gates_fwd.restype = I
    L.gdn2_layer_gates_bwd.argtypes = [P] * 9 + [I] * 6 + [P]
    L.gdn2_layer_gates_bwd.restype = I
    F = ctypes.c_float
    L.gdn2_linear_workspace_size.argtypes = [I] * 7
    L.gdn2_linear_workspace_size.restype = Z
    L.gdn2_linear_varlen_workspace_size.argtypes = [I] * 3 + [LL] + [I] * 4
    L.gdn2_linear_varlen_workspace_size.restype = Z
    L.gdn2_linear_fwd.argtypes = [P] * 7 + [I] * 6 + [P, Z, P]
    L.gdn2_linear_fwd.restype = I
    L.gdn2_linear_bwd.argtypes = [P] * 11 + [I] * 6 + [P, Z, P]
    L.gdn2_linear_bwd.restype = I
    L.gdn2_linear_varlen_fwd.argtypes = [P] * 5 + [I, I, LL] + [P] * 3 + [I] * 4 + [P, Z, P]
    L.gdn2_linear_varlen_fwd.restype = I
    L.gdn2_linear_varlen_bwd.argtypes = [P] * 5 + [I, I, LL] + [P] * 7 + [I] * 4 + [P, Z, P]
    L.gdn2_linear_varlen_bwd.restype = I
    L.gdn2_linear_decode_step.argtypes = [P] * 6 + [I, P] + [I] * 5 + [P]
    L.gdn2_linear_decode_step.restype = I
    L.gdn2_qk_norm_rope_workspace_size.argtypes = [I]
    L.gdn2_qk_norm_rope_workspace_size.restype = Z
    rope = [P, I, I, P, P, I, I, I, F, P, P]   # positions .. k_weight
    L.gdn2_qk_norm_rope_fwd.argtypes = [P, P, LL, LL] + rope + [P] * 2 + [I] * 6 + [P]
    L.gdn2_qk_norm_rope_fwd.restype = I
    L.gdn2_qk_norm_rope_bwd.argtypes = [P, P, LL, LL, P, P] + rope + [P] * 4 + [I] * 6 + [P, Z, P]
    L.gdn2_qk_norm_rope_bwd.restype = I
    L.gdn2_device_status.argtypes = [P]
    L.gdn2_device_status.restype = I
    L.gdn2_trace_enable.argtypes = [I]
    L.gdn2_trace_enable.restype = None
    L.gdn2_trace_read.argtypes = [ctypes.c_char_p, Z, P, P, I]
    L.gdn2_trace_read.restype = I
    if path is None:
        _lib = L
    return L


def _check(fn, rc):
    if rc != 0:
        raise Gdn2Error(fn, rc, lib().gdn2_last_error().decode(errors="replace"))


def _dt(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return GDN2_BF16
    if t.dtype == torch.float32:
        return GDN2_F32
    raise TypeError("dtype %s is not supported (float32 or bfloat16)" % t.dtype)


def _ptr(t: Optional[torch.Tensor]):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("tensors must be on a CUDA device")
    if not t.is_contiguous():
        raise ValueError("tensors must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


def _stream(device) -> ctypes.c_void_p:
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _state(t, like, B, H, Dk, Dv):
    if t is None:
        return None
    if t.dtype != torch.float32 or tuple(t.shape) != (B, H, Dk, Dv):
        raise ValueError("states must be float32 [B, H, Dk, Dv] = %s" % ((B, H, Dk, Dv),))
    return t


def gdn2_workspace_size(op: int, B: int, T: int, H: int, Dk: int, Dv: int, chunk: int, dt: int) -> int:
    return int(lib().gdn2_workspace_size(op, B, T, H, Dk, Dv, chunk, dt))


def gdn2_fwd(q, k, v, log_alpha, b, w, S0=None, chunk: int = 64, want_state: bool = True,
             save_states: bool = False, ws: Optional[torch.Tensor] = None, o=None, ST=None):
    """Forward. Tensors [B, T, H, D] (bf16 or fp32), S0 [B, H, Dk, Dv] fp32 or None.

    Returns ``(o, ST)`` (``ST`` is None unless ``want_state``). ``ws`` is a uint8
    CUDA tensor of at least ``gdn2_workspace_size(GDN2_OP_FWD[_SAVE], ...)`` bytes,
    allocated if not given. With ``save_states`` the chunk-start states are kept in
    it for a later :func:`gdn2_bwd` with ``states_saved=True``.
    """
    B, T, H, Dk = q.shape
    Dv = v.shape[-1]
    dt = _dt(q)
    for name, t, D in (("k", k, Dk), ("v", v, Dv), ("log_alpha", log_alpha, Dk), ("b", b, Dk), ("w", w, Dv)):
        if t.dtype != q.dtype or tuple(t.shape) != (B, T, H, D):
            raise ValueError("%s must be %s [%d, %d, %d, %d]" % (name, q.dtype, B, T, H, D))
    _state(S0, q, B, H, Dk, Dv)
    if o is None:
        o = torch.empty((B, T, H, Dv), dtype=q.dtype, device=q.device)
    if ST is None and want_state:
        ST = torch.empty((B, H, Dk, Dv), dtype=torch.float32, device=q.device)
    ws_bytes = 0
    need = gdn2_workspace_size(GDN2_OP_FWD_SAVE if save_states else GDN2_OP_FWD, B, T, H, Dk, Dv, chunk, dt)
    if need and ws is None:
        ws = torch.empty(need, dtype=torch.uint8, device=q.device)
    if ws is not None:
        ws_bytes = ws.numel()
    rc = lib().gdn2_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha), _ptr(b), _ptr(w), _ptr(S0), _ptr(o),
                        _ptr(ST), B, T, H, Dk, Dv, chunk, dt, int(save_states), _ptr(ws), ws_bytes,
                        _stream(q.device))
    _check("gdn2_fwd", rc)
    return o, ST


def gdn2_bwd(q, k, v, log_alpha, b, w, dout, S0=None, dST=None, chunk: int = 64, want_dS0: bool = True,
             states_saved: bool = False, ws: Optional[torch.Tensor] = None, grads=None):
    """Gate-aware backward for L = <dout, o> + <dST, S_T>.

    Returns a dict with dq, dk, dv, dlog_alpha, db, dw (input dtype) and dS0 (fp32 or None).
    """
    B, T, H, Dk = q.shape
    Dv = v.shape[-1]
    dt = _dt(q)
    _state(S0, q, B, H, Dk, Dv)
    _state(dST, q, B, H, Dk, Dv)
    if tuple(dout.shape) != (B, T, H, Dv) or dout.dtype != q.dtype:
        raise ValueError("dout must be %s [%d, %d, %d, %d]" % (q.dtype, B, T, H, Dv))
    if grads is None:
        grads = {n: torch.empty_like(q) for n in ("dq", "dk", "dlog_alpha", "db")}
        grads.update({n: torch.empty_like(v) for n in ("dv", "dw")})
        grads["dS0"] = torch.empty((B, H, Dk, Dv), dtype=torch.float32, device=q.device) if want_dS0 else None
    need = gdn2_workspace_size(GDN2_OP_BWD, B, T, H, Dk, Dv, chunk, dt)
    if ws is None:
        ws = torch.empty(max(need, 256), dtype=torch.uint8, device=q.device)
    g = grads
    rc = lib().gdn2_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha), _ptr(b), _ptr(w), _ptr(S0), _ptr(dout),
                        _ptr(dST), _ptr(g["dq"]), _ptr(g["dk"]), _ptr(g["dv"]), _ptr(g["dlog_alpha"]),
                        _ptr(g["db"]), _ptr(g["dw"]), _ptr(g.get("dS0")), B, T, H, Dk, Dv, chunk, dt,
                        int(states_saved), _ptr(ws), ws.numel(), _stream(q.device))
    _check("gdn2_bwd", rc)
    return grads


def _map_ws(q, v, chunk, ws):
    B, T, H, Dk = q.shape
    need = gdn2_workspace_size(GDN2_OP_MAP, B, T, H, Dk, v.shape[-1], chunk, _dt(q))
    if ws is None:
        ws = torch.empty(max(need, 256), dtype=torch.uint8, device=q.device)
    return ws


def gdn2_fwd_map(q, k, v, log_alpha, b, w, chunk: int = 64, ws: Optional[torch.Tensor] = None):
    """Affine map of a sequence piece, ``S_end = M S_start + N``: returns ``(M, N)``, fp32
    ``[B, H, Dk, Dk]`` and ``[B, H, Dk, Dv]``."""
    B, T, H, Dk = q.shape
    Dv = v.shape[-1]
    M = torch.empty((B, H, Dk, Dk), dtype=torch.float32, device=q.device)
    N = torch.empty((B, H, Dk, Dv), dtype=torch.float32, device=q.device)
    ws = _map_ws(q, v, chunk, ws)
    rc = lib().gdn2_fwd_map(_ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha), _ptr(b), _ptr(w), _ptr(M), _ptr(N),
                            B, T, H, Dk, Dv, chunk, _dt(q), _ptr(ws), ws.numel(), _stream(q.device))
    _check("gdn2_fwd_map", rc)
    return M, N


def gdn2_bwd_map(q, k, v, log_alpha, b, w, dout, chunk: int = 64, ws: Optional[torch.Tensor] = None):
    """Reverse affine map of a sequence piece, ``dS_start = A dS_end + B``: returns ``(A, B)``."""
    B, T, H, Dk = q.shape
    Dv = v.shape[-1]
    A = torch.empty((B, H, Dk, Dk), dtype=torch.float32, device=q.device)
    Bm = torch.empty((B, H, Dk, Dv), dtype=torch.float32, device=q.device)
    ws = _map_ws(q, v, chunk, ws)
    rc = lib().gdn2_bwd_map(_ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha), _ptr(b), _ptr(w), _ptr(dout), _ptr(A),
                            _ptr(Bm), B, T, H, Dk, Dv, chunk, _dt(q), _ptr(ws), ws.numel(), _stream(q.device))
    _check("gdn2_bwd_map", rc)
    return A, Bm


def gdn2_state_affine(M, N, S_in, out=None):
    """``M S_in + N`` per (batch, head) in fp32 (``N`` or ``S_in`` may be None: zero)."""
    B, H, Dk, _ = M.shape
    ref = N if N is not None else S_in
    Dv = ref.shape[-1] if ref is not None else Dk
    if out is None:
        out = torch.empty((B, H, Dk, Dv), dtype=torch.float32, device=M.device)
    rc = lib().gdn2_state_affine(_ptr(M), _ptr(N), _ptr(S_in), _ptr(out), B, H, Dk, Dv, _stream(M.device))
    _check("gdn2_state_affine", rc)
    return out


def gdn2_layer_gates_fwd(z, Dk: int, Dv: int, a_bias=None):
    """Operator inputs from the layer's pre-activations ``z [B, T, H, 4 Dk + 2 Dv]``: returns
    ``(q, k, v, b, w, log_alpha)`` in z's dtype (``a_bias``: fp32 [H, Dk] decay bias or None)."""
    B, T, H, W = z.shape
    if W != 4 * Dk + 2 * Dv:
        raise ValueError("z must be [B, T, H, 4 Dk + 2 Dv]")
    if a_bias is not None and (a_bias.dtype != torch.float32 or tuple(a_bias.shape) != (H, Dk)):
        raise ValueError("a_bias must be float32 [H, Dk]")
    mk = lambda D: torch.empty((B, T, H, D), dtype=z.dtype, device=z.device)
    q, k, v, b, w, la = mk(Dk), mk(Dk), mk(Dv), mk(Dk), mk(Dv), mk(Dk)
    rc = lib().gdn2_layer_gates_fwd(_ptr(z), _ptr(a_bias), _ptr(q), _ptr(k), _ptr(v), _ptr(b), _ptr(w), _ptr(la),
                                    B, T, H, Dk, Dv, _dt(z), _stream(z.device))
    _check("gdn2_layer_gates_fwd", rc)
    return q, k, v, b, w, la


def gdn2_layer_gates_bwd(z, dq, dk, dv, db, dw, dlog_alpha, Dk: int, Dv: int, a_bias=None):
    """dz (z's layout) from z and the gradients of the six operator inputs."""
    B, T, H, _ = z.shape
    dz = torch.empty_like(z)
    rc = lib().gdn2_layer_gates_bwd(_ptr(z), _ptr(a_bias), _ptr(dq), _ptr(dk), _ptr(dv), _ptr(db), _ptr(dw),
                                    _ptr(dlog_alpha), _ptr(dz), B, T, H, Dk, Dv, _dt(z), _stream(z.device))
    _check("gdn2_layer_gates_bwd", rc)
    return dz


def gdn2_beta_workspace_size(gate: int, op: int, B: int, T: int, H: int, Dk: int, Dv: int, chunk: int,
                             dt: int) -> int:
    return int(lib().gdn2_beta_workspace_size(gate, op, B, T, H, Dk, Dv, chunk, dt))


def gdn2_beta_fwd(gate, q, k, v, log_alpha, beta, S0=None, chunk: int = 64, want_state: bool = True,
                  save_states: bool = False, ws: Optional[torch.Tensor] = None, o=None, ST=None):
    """KDA (gate=GDN2_GATE_KDA, log_alpha [B,T,H,Dk]) or Gated DeltaNet (GDN2_GATE_GDN, log_alpha [B,T,H])
    forward through the Gated Delta Rule-2 kernels; beta [B,T,H]. Returns ``(o, ST)``."""
    B, T, H, Dk = q.shape
    Dv = v.shape[-1]
    dt = _dt(q)
    la_shape = (B, T, H, Dk) if gate == GDN2_GATE_KDA else (B, T, H)
    for name, t, shp in (("k", k, (B, T, H, Dk)), ("v", v, (B, T, H, Dv)), ("log_alpha", log_alpha, la_shape),
                         ("beta", beta, (B, T, H))):
        if t.dtype != q.dtype or tuple(t.shape) != shp:
            raise ValueError("%s must be %s %s" % (name, q.dtype, shp))
    _state(S0, q, B, H, Dk, Dv)
    if o is None:
        o = torch.empty((B, T, H, Dv), dtype=q.dtype, device=q.device)
    if ST is None and want_state:
        ST = torch.empty((B, H, Dk, Dv), dtype=torch.float32, device=q.device)
    op = GDN2_OP_FWD_SAVE if save_states else GDN2_OP_FWD
    need = gdn2_beta_workspace_size(gate, op, B, T, H, Dk, Dv, chunk, dt)
    if ws is None:
        ws = torch.empty(max(need, 256), dtype=torch.uint8, device=q.device)
    rc = lib().gdn2_beta_fwd(gate, _ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha), _ptr(beta), _ptr(S0), _ptr(o),
                             _ptr(ST), B, T, H, Dk, Dv, chunk, dt, int(save_states), _ptr(ws), ws.numel(),
                             _stream(q.device))
    _check("gdn2_beta_fwd", rc)
    return o, ST


def gdn2_beta_bwd(gate, q, k, v, log_alpha, beta, dout, S0=None, dST=None, chunk: int = 64, want_dS0: bool = True,
                  states_saved: bool = False, ws: Optional[torch.Tensor] = None, grads=None):
    """Backward of :func:`gdn2_beta_fwd`: dict with dq, dk, dv, dlog_alpha (shape of log_alpha), dbeta
    [B,T,H] and dS0."""
    B, T, H, Dk = q.shape
    Dv = v.shape[-1]
    dt = _dt(q)
    _state(S0, q, B, H, Dk, Dv)
    _state(dST, q, B, H, Dk, Dv)
    if grads is None:
        grads = {"dq": torch.empty_like(q), "dk": torch.empty_like(q), "dv": torch.empty_like(v),
                 "dlog_alpha": torch.empty_like(log_alpha), "dbeta": torch.empty_like(beta),
                 "dS0": torch.empty((B, H, Dk, Dv), dtype=torch.float32, device=q.device) if want_dS0 else None}
    need = gdn2_beta_workspace_size(gate, GDN2_OP_BWD, B, T, H, Dk, Dv, chunk, dt)
    if ws is None:
        ws = torch.empty(max(need, 256), dtype=torch.uint8, device=q.device)
    g = grads
    rc = lib().gdn2_beta_bwd(gate, _ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha), _ptr(beta), _ptr(S0), _ptr(dout),
                             _ptr(dST), _ptr(g["dq"]), _ptr(g["dk"]), _ptr(g["dv"]), _ptr(g["dlog_alpha"]),
                             _ptr(g["dbeta"]), _ptr(g.get("dS0")), B, T, H, Dk, Dv, chunk, dt, int(states_saved),
                             _ptr(ws), ws.numel(), _stream(q.device))
    _check("gdn2_beta_bwd", rc)
    return grads


def gdn2_varlen_workspace_size(op: int, N: int, Tmax: int, H: int, Dk: int, Dv: int, chunk: int, dt: int) -> int:
    return int(lib().gdn2_varlen_workspace_size(op, N, Tmax, H, Dk, Dv, chunk, dt))


def gdn2_varlen_fwd(q, k, v, log_alpha, b, w, cu_seqlens, Tmax: int, S0=None, chunk: int = 64,
                    want_state: bool = True, save_states: bool = False, ws: Optional[torch.Tensor] = None):
    """Packed sequences: tensors [Ttot, H, D], cu_seqlens int32 [N + 1] on the device, Tmax >= every length.
    Returns ``(o [Ttot, H, Dv], ST [N, H, Dk, Dv] or None)``."""
    Ttot, H, Dk = q.shape
    Dv = v.shape[-1]
    N = cu_seqlens.numel() - 1
    dt = _dt(q)
    if cu_seqlens.dtype != torch.int32 or not cu_seqlens.is_cuda:
        raise ValueError("cu_seqlens must be an int32 CUDA tensor")
    _state(S0, q, N, H, Dk, Dv)
    o = torch.empty((Ttot, H, Dv), dtype=q.dtype, device=q.device)
    ST = torch.empty((N, H, Dk, Dv), dtype=torch.float32, device=q.device) if want_state else None
    need = gdn2_varlen_workspace_size(GDN2_OP_FWD_SAVE if save_states else GDN2_OP_FWD, N, Tmax, H, Dk, Dv, chunk, dt)
    if ws is None:
        ws = torch.empty(max(need, 256), dtype=torch.uint8, device=q.device)
    rc = lib().gdn2_varlen_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha), _ptr(b), _ptr(w), _ptr(cu_seqlens), N,
                               Tmax, Ttot, _ptr(S0), _ptr(o), _ptr(ST), H, Dk, Dv, chunk, dt, int(save_states),
                               _ptr(ws), ws.numel(), _stream(q.device))
    _check("gdn2_varlen_fwd", rc)
    return o, ST


def gdn2_varlen_bwd(q, k, v, log_alpha, b, w, dout, cu_seqlens, Tmax: int, S0=None, dST=None, chunk: int = 64,
                    want_dS0: bool = True, states_saved: bool = False, ws: Optional[torch.Tensor] = None):
    """Backward of :func:`gdn2_varlen_fwd`: dict of packed dq, dk, dv, dlog_alpha, db, dw and dS0 [N, ...]."""
    Ttot, H, Dk = q.shape
    Dv = v.shape[-1]
    N = cu_seqlens.numel() - 1
    dt = _dt(q)
    _state(S0, q, N, H, Dk, Dv)
    _state(dST, q, N, H, Dk, Dv)
    g = {n: torch.empty_like(q) for n in ("dq", "dk", "dlog_alpha", "db")}
    g.update({n: torch.empty_like(v) for n in ("dv", "dw")})
    g["dS0"] = torch.empty((N, H, Dk, Dv), dtype=torch.float32, device=q.device) if want_dS0 else None
    need = gdn2_varlen_workspace_size(GDN2_OP_BWD, N, Tmax, H, Dk, Dv, chunk, dt)
    if ws is None:
        ws = torch.empty(max(need, 256), dtype=torch.uint8, device=q.device)
    rc = lib().gdn2_varlen_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha), _ptr(b), _ptr(w), _ptr(cu_seqlens), N,
                               Tmax, Ttot, _ptr(S0), _ptr(dout), _ptr(dST), _ptr(g["dq"]), _ptr(g["dk"]), _ptr(g["dv"]),
                               _ptr(g["dlog_alpha"]), _ptr(g["db"]), _ptr(g["dw"]), _ptr(g["dS0"]), H, Dk, Dv, chunk,
                               dt, int(states_saved), _ptr(ws), ws.numel(), _stream(q.device))
    _check("gdn2_varlen_bwd", rc)
    return g


def gdn2_decode_step(q, k, v, log_alpha, b, w, S, o=None):
    """One decode step: inputs [B, H, D]; S [B, H, Dk, Dv] fp32 is updated in place. Returns o."""
    B, H, Dk = q.shape
    Dv = v.shape[-1]
    _state(S, q, B, H, Dk, Dv)
    if o is None:
        o = torch.empty((B, H, Dv), dtype=q.dtype, device=q.device)
    rc = lib().gdn2_decode_step(_ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha), _ptr(b), _ptr(w), _ptr(S), _ptr(o),
                                B, H, Dk, Dv, _dt(q), _stream(q.device))
    _check("gdn2_decode_step", rc)
    return o


# ------------------------------------------------------------------ linear attention with a decay per head

# A call of one token takes the GPU a few microseconds, so the checks of these calls are made of cheap questions: a
# tensor's device by index, shapes read once.

def _on(t: torch.Tensor, device: int, name: str) -> int:
    """Device pointer of a contiguous tensor on the call's device (as an int: ctypes converts it by the argtypes)."""
    if t.get_device() != device:
        raise ValueError("%s must be on cuda:%d, not on %s" % (name, device, t.device))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    return t.data_ptr()


def _opt(t: Optional[torch.Tensor], device: int, name: str, dtype, shape):
    if t is None:
        return None
    if t.dtype != dtype or t.shape != shape:
        raise ValueError("%s must be %s %s" % (name, dtype, list(shape)))
    return _on(t, device, name)


# the current stream's handle without the Stream object around it, which costs more than a launch
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (lambda i: torch.cuda.current_stream(i).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _here(t: torch.Tensor, call):
    """``call(device, stream)`` with t's device current (launches go to the current device) and its current stream."""
    if not t.is_cuda:
        raise ValueError("tensors must be on a CUDA device")
    dev = t.get_device()
    if dev == _current_device():
        return call(dev, _raw_stream(dev))
    with torch.cuda.device(dev):
        return call(dev, _raw_stream(dev))


def gdn2_linear_workspace_size(op: int, N: int, T: int, H: int, Dk: int, Dv: int, dt: int) -> int:
    return int(lib().gdn2_linear_workspace_size(op, N, T, H, Dk, Dv, dt))


def gdn2_linear_varlen_workspace_size(op: int, N: int, Tmax: int, Ttot: int, H: int, Dk: int, Dv: int, dt: int) -> int:
    return int(lib().gdn2_linear_varlen_workspace_size(op, N, min(Tmax, Ttot), Ttot, H, Dk, Dv, dt))


def _linear(fn, q, k, v, log_decay, S0, dout, dST, cu, Tmax, want_end, ws, outs, ends):
    """Shared by the four whole-sequence calls: checks, outputs, workspace, the call. Returns (outs, end state)."""
    packed = cu is not None
    qs, vs = q.shape, v.shape
    if len(qs) != (3 if packed else 4) or len(vs) != len(qs):
        raise ValueError("q and v must be [%sH, D]" % ("Ttot, " if packed else "B, T, "))
    *lead, H, Dk = qs
    Dv = vs[-1]
    dt, code = q.dtype, _dt(q)
    if k.dtype != dt or k.shape != qs:
        raise ValueError("k must be %s %s" % (dt, list(qs)))
    if v.dtype != dt or vs[:-1] != qs[:-1]:
        raise ValueError("v must be %s %s" % (dt, lead + [H, "Dv"]))
    if dout is not None and (dout.dtype != dt or dout.shape != vs):
        raise ValueError("dout must be %s %s" % (dt, list(vs)))
    if log_decay.dtype != torch.float32 or log_decay.dim() != 1 or log_decay.shape[0] != H:
        raise ValueError("log_decay must be float32 [%d]" % H)
    if packed:
        if cu.dtype != torch.int32 or cu.dim() != 1 or cu.numel() < 2:
            raise ValueError("cu_seqlens must be int32 [N + 1]")
        N, T = cu.numel() - 1, min(int(Tmax), lead[0])   # no sequence is longer than the tensor
    else:
        N, T = lead
    bwd = dout is not None
    state = (N, H, Dk, Dv)
    f32 = torch.float32

    def call(dev, stream):
        nonlocal ws
        args = [_on(q, dev, "q"), _on(k, dev, "k"), _on(v, dev, "v"), _on(log_decay, dev, "log_decay")]
        made = []
        for name, t, like in outs:   # (contiguous, as q, k and v are)
            if t is None:
                t = torch.empty_like(like)
            elif t.dtype != dt or t.shape != like.shape:
                raise ValueError("%s must be %s %s" % (name, dt, list(like.shape)))
            made.append(t)
        name, end = ends
        if end is None and want_end:
            end = q.new_empty(state, dtype=f32)
        L = lib()
        op = GDN2_OP_BWD if bwd else GDN2_OP_FWD
        need = (L.gdn2_linear_varlen_workspace_size(op, N, T, lead[0], H, Dk, Dv, code) if packed else
                L.gdn2_linear_workspace_size(op, N, T, H, Dk, Dv, code))
        if ws is None and need:
            ws = q.new_empty(need, dtype=torch.uint8)
        if packed:
            args += [_on(cu, dev, "cu_seqlens"), N, T, lead[0]]
        args.append(_opt(S0, dev, "S0", f32, state))
        if bwd:
            args += [_on(dout, dev, "dout"), _opt(dST, dev, "dST", f32, state)]
        args += [_on(t, dev, o[0]) for t, o in zip(made, outs)]
        args.append(_opt(end, dev, name, f32, state))
        if not packed:
            args += [N, T]
        rc = getattr(L, fn)(*args, H, Dk, Dv, code, None if ws is None else _on(ws, dev, "ws"),
                            0 if ws is None else ws.numel() * ws.element_size(), stream)
        if rc:
            _check(fn, rc)
        return made, end

    return _here(q, call)


def gdn2_linear_fwd(q, k, v, log_decay, S0=None, want_state: bool = True, ws: Optional[torch.Tensor] = None, o=None, ST=None):
    """Linear attention with a fixed decay per head, ``S_t = exp(log_decay_h) S_{t-1} + k_t v_t^T``, ``o_t = S_t^T q_t``.

    q, k [B, T, H, Dk], v [B, T, H, Dv] (bf16 or fp32), log_decay [H] fp32 (<= 0), S0 [B, H, Dk, Dv] fp32 or None.
    Returns ``(o, ST)`` (``ST`` is None unless ``want_state`` or given). ``ws`` is a uint8 CUDA tensor of at least
    ``gdn2_linear_workspace_size(GDN2_OP_FWD, ...)`` bytes, allocated if not given.
    """
    (o,), ST = _linear("gdn2_linear_fwd", q, k, v, log_decay, S0, None, None, None, None, want_state, ws,
                       (("o", o, v),), ("ST", ST))
    return o, ST


def gdn2_linear_bwd(q, k, v, log_decay, dout, S0=None, dST=None, want_dS0: bool = True,
                    ws: Optional[torch.Tensor] = None, grads=None):
    """Backward of :func:`gdn2_linear_fwd` for L = <dout, o> + <dST, S_T>: dict with dq, dk, dv (input dtype) and dS0
    (fp32 or None)."""
    g = grads or {}
    (dq, dk, dv), dS0 = _linear("gdn2_linear_bwd", q, k, v, log_decay, S0, dout, dST, None, None, want_dS0, ws,
                                (("dq", g.get("dq"), q), ("dk", g.get("dk"), k), ("dv", g.get("dv"), v)),
                                ("dS0", g.get("dS0")))
    return {"dq": dq, "dk": dk, "dv": dv, "dS0": dS0}


def gdn2_linear_varlen_fwd(q, k, v, log_decay, cu_seqlens, Tmax: int, S0=None, want_state: bool = True,
                           ws: Optional[torch.Tensor] = None, o=None, ST=None):
    """Packed sequences: q, k, v [Ttot, H, D], cu_seqlens int32 [N + 1] on the device, Tmax >= every length (a bound above
    Ttot counts as Ttot). ``ws``: at least ``gdn2_linear_varlen_workspace_size(GDN2_OP_FWD, ...)`` bytes.
    Returns ``(o [Ttot, H, Dv], ST [N, H, Dk, Dv] or None)``; rows of ``o`` behind the last sequence are not written."""
    (o,), ST = _linear("gdn2_linear_varlen_fwd", q, k, v, log_decay, S0, None, None, cu_seqlens, Tmax, want_state, ws,
                       (("o", o, v),), ("ST", ST))
    return o, ST


def gdn2_linear_varlen_bwd(q, k, v, log_decay, dout, cu_seqlens, Tmax: int, S0=None, dST=None, want_dS0: bool = True,
                           ws: Optional[torch.Tensor] = None, grads=None):
    """Backward of :func:`gdn2_linear_varlen_fwd`: dict of packed dq, dk, dv and dS0 [N, ...]."""
    g = grads or {}
    (dq, dk, dv), dS0 = _linear("gdn2_linear_varlen_bwd", q, k, v, log_decay, S0, dout, dST, cu_seqlens, Tmax, want_dS0, ws,
                                (("dq", g.get("dq"), q), ("dk", g.get("dk"), k), ("dv", g.get("dv"), v)),
                                ("dS0", g.get("dS0")))
    return {"dq": dq, "dk": dk, "dv": dv, "dS0": dS0}


def gdn2_linear_decode_step(q, k, v, log_decay, S, slots=None, o=None):
    """One token of :func:`gdn2_linear_fwd` for every row: q, k, v [B, H, D]; S [num_slots, H, Dk, Dv] fp32, updated in
    place. ``slots`` (int32 [B] on the device) names each row's state, a negative one an idle row (its o is zero);
    None: row b has S[b]. Returns o."""
    qs, vs, ss = q.shape, v.shape, S.shape
    if len(qs) != 3 or len(vs) != 3:
        raise ValueError("q and v must be [B, H, D]")
    B, H, Dk = qs
    Dv = vs[2]
    dt, code = q.dtype, _dt(q)
    if k.dtype != dt or k.shape != qs or v.dtype != dt or vs[0] != B or vs[1] != H:
        raise ValueError("k and v must be %s [%d, %d, D]" % (dt, B, H))
    if log_decay.dtype != torch.float32 or log_decay.dim() != 1 or log_decay.shape[0] != H:
        raise ValueError("log_decay must be float32 [%d]" % H)
    if S.dtype != torch.float32 or len(ss) != 4 or ss[1] != H or ss[2] != Dk or ss[3] != Dv:
        raise ValueError("S must be float32 [num_slots, %d, %d, %d]" % (H, Dk, Dv))
    if o is not None and (o.dtype != dt or o.shape != vs):
        raise ValueError("o must be %s [%d, %d, %d]" % (dt, B, H, Dv))

    def call(dev, stream):
        vp = _on(v, dev, "v")
        out = torch.empty_like(v) if o is None else o
        rc = lib().gdn2_linear_decode_step(
            _on(q, dev, "q"), _on(k, dev, "k"), vp, _on(log_decay, dev, "log_decay"), _on(S, dev, "S"),
            _opt(slots, dev, "slots", torch.int32, (B,)), ss[0], _on(out, dev, "o"), B, H, Dk, Dv, code, stream)
        if rc:
            _check("gdn2_linear_decode_step", rc)
        return out

    return _here(q, call)


class DecayLinearAttention(torch.autograd.Function):
    """autograd wrapper of the linear attention calls (dense, or packed with cu_seqlens)."""

    @staticmethod
    def forward(ctx, q, k, v, log_decay, S0, cu_seqlens, Tmax):
        ctx.set_materialize_grads(False)
        if cu_seqlens is None:
            o, ST = gdn2_linear_fwd(q, k, v, log_decay, S0)
        else:
            # rows behind the last sequence are nobody's: zeros, so that what follows can take the whole tensor
            o, ST = gdn2_linear_varlen_fwd(q, k, v, log_decay, cu_seqlens, Tmax, S0, o=torch.zeros_like(v))
        ctx.save_for_backward(q, k, v, log_decay, S0, cu_seqlens)
        ctx.Tmax = Tmax
        return o, ST

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, do, dST):
        q, k, v, log_decay, S0, cu = ctx.saved_tensors
        if do is None and dST is None:
            return (None,) * 7
        do = torch.zeros_like(v) if do is None else do.contiguous()
        dST = None if dST is None else dST.contiguous()
        want = ctx.needs_input_grad[4]
        if cu is None:
            g = gdn2_linear_bwd(q, k, v, log_decay, do, S0, dST, want_dS0=want)
        else:
            grads = {"dq": torch.zeros_like(q), "dk": torch.zeros_like(k), "dv": torch.zeros_like(v)}
            g = gdn2_linear_varlen_bwd(q, k, v, log_decay, do, cu, ctx.Tmax, S0, dST, want_dS0=want, grads=grads)
        return g["dq"], g["dk"], g["dv"], None, g["dS0"], None, None


def decay_linear_attention(q, k, v, log_decay, S0=None, cu_seqlens=None, Tmax: Optional[int] = None):
    """Differentiable linear attention with a fixed decay per head. Returns ``(o, S_T)``. With ``cu_seqlens`` (and
    ``Tmax``) the tensors are packed [Ttot, H, D]; ``o`` and the gradients are zero behind the last sequence."""
    if log_decay.requires_grad:
        raise ValueError("log_decay has no gradient: pass it detached")
    if (cu_seqlens is None) != (Tmax is None):
        raise ValueError("cu_seqlens and Tmax come together")
    return DecayLinearAttention.apply(q, k, v, log_decay, S0, cu_seqlens, Tmax)


# ------------------------------------------------------------------ query/key norm and rotation

def rope_axes(sections, device="cuda") -> torch.Tensor:
    """The ``axes`` argument for pairs laid out axis after axis, ``sections[i]`` pairs turning by axis i."""
    return torch.cat([torch.full((int(n),), i, dtype=torch.int32) for i, n in enumerate(sections)]).to(device)


def _rows_of(t, name, B, T, H, D):
    """Pointer and token stride of [B, T, H, D] whose heads are contiguous and whose tokens are evenly spaced."""
    if t.is_contiguous():
        return t.data_ptr(), H * D
    sb, st, sh, sd = t.stride()
    if sd != 1 or (sh != D and H > 1) or (B > 1 and T > 1 and sb != T * st):
        raise ValueError("%s: a token's heads must be contiguous and the tokens evenly spaced" % name)
    return t.data_ptr(), (st if T > 1 else sb if B > 1 else H * D)


def _rope(q, k, positions, inv_freq, axes, q_weight, k_weight, eps, interleaved):
    """Checks of the arguments the forward and the backward share: (sizes, leading and positional C arguments)."""
    qs, ks, ps = q.shape, k.shape, positions.shape
    if len(qs) != 4 or len(ks) != 4 or qs[0] != ks[0] or qs[1] != ks[1] or qs[3] != ks[3]:
        raise ValueError("q and k must be [B, T, Hq, D] and [B, T, Hk, D]")
    B, T, Hq, D = qs
    Hk = ks[2]
    dev, dt = q.get_device(), q.dtype
    if k.dtype != dt or k.get_device() != dev:
        raise ValueError("q and k must be of one dtype and on one device")
    if positions.dtype not in (torch.int32, torch.int64):
        raise TypeError("positions must be int32 or int64")
    if len(ps) not in (2, 3) or ps[-2] != B or ps[-1] != T:
        raise ValueError("positions must be [B, T] or [axes, B, T] = [..., %d, %d]" % (B, T))
    num_axes = ps[0] if len(ps) == 3 else 1
    if inv_freq.dtype != torch.float32 or inv_freq.dim() != 1:
        raise ValueError("inv_freq must be float32 [pairs]")
    P = inv_freq.shape[0]
    if num_axes > 1 and axes is None:
        raise ValueError("positions of several axes need axes, the axis of each pair")
    norm = eps is not None
    if not norm and (q_weight is not None or k_weight is not None):
        raise ValueError("a weight needs a norm: give eps")
    f32 = torch.float32
    q_ptr, q_step = _rows_of(q, "q", B, T, Hq, D)
    k_ptr, k_step = _rows_of(k, "k", B, T, Hk, D)
    tail = (_on(positions, dev, "positions"), positions.element_size(), num_axes, _on(inv_freq, dev, "inv_freq"),
            _opt(axes, dev, "axes", torch.int32, (P,)), P, 1 if interleaved else 0, 1 if norm else 0, eps if norm else 0.0,
            _opt(q_weight, dev, "q_weight", f32, (D,)), _opt(k_weight, dev, "k_weight", f32, (D,)))
    return (B, T, Hq, Hk, D, _dt(q)), (q_ptr, k_ptr, q_step, k_step), tail


def gdn2_qk_norm_rope_fwd(q, k, positions, inv_freq, axes=None, q_weight=None, k_weight=None, eps: Optional[float] = 1e-6,
                          interleaved: bool = False, q_out=None, k_out=None):
    """RMS norm of every query and key head and the rotation of its channel pairs by the token's position.

    q [B, T, Hq, D], k [B, T, Hk, D] (bf16 or fp32; a token's heads contiguous, so slices of one projection's output
    are taken as they are), positions int32 or int64 [B, T], or [axes, B, T] with ``axes`` (int32 [pairs], see
    :func:`rope_axes`) naming each pair's axis, inv_freq fp32 [pairs], weights fp32 [D] or None. ``eps=None``: no norm.
    Pairs are channels (p, p + pairs), or (2p, 2p + 1) if ``interleaved``. Returns ``(q_out, k_out)``, contiguous.
    """
    def call(dev, stream):
        sizes, lead, tail = _rope(q, k, positions, inv_freq, axes, q_weight, k_weight, eps, interleaved)
        qo = torch.empty_like(q, memory_format=torch.contiguous_format) if q_out is None else q_out
        ko = torch.empty_like(k, memory_format=torch.contiguous_format) if k_out is None else k_out
        qo_ptr = qo.data_ptr() if q_out is None else _opt(qo, dev, "q_out", q.dtype, q.shape)
        ko_ptr = ko.data_ptr() if k_out is None else _opt(ko, dev, "k_out", q.dtype, k.shape)
        rc = lib().gdn2_qk_norm_rope_fwd(*lead, *tail, qo_ptr, ko_ptr, *sizes, stream)
        if rc:
            _check("gdn2_qk_norm_rope_fwd", rc)
        return qo, ko

    return _here(q, call)


def gdn2_qk_norm_rope_bwd(q, k, dq_out, dk_out, positions, inv_freq, axes=None, q_weight=None, k_weight=None,
                          eps: Optional[float] = 1e-6, interleaved: bool = False, ws: Optional[torch.Tensor] = None):
    """Backward of :func:`gdn2_qk_norm_rope_fwd`: dict with dq, dk and, for given weights, dq_weight, dk_weight (fp32;
    None otherwise)."""
    def call(dev, stream):
        nonlocal ws
        sizes, lead, tail = _rope(q, k, positions, inv_freq, axes, q_weight, k_weight, eps, interleaved)
        D, dt = q.shape[3], q.dtype
        g = {"dq": torch.empty_like(q, memory_format=torch.contiguous_format),
             "dk": torch.empty_like(k, memory_format=torch.contiguous_format),
             "dq_weight": None if q_weight is None else torch.empty_like(q_weight),
             "dk_weight": None if k_weight is None else torch.empty_like(k_weight)}
        if ws is None and (q_weight is not None or k_weight is not None):
            ws = q.new_empty(lib().gdn2_qk_norm_rope_workspace_size(D), dtype=torch.uint8)
        rc = lib().gdn2_qk_norm_rope_bwd(
            *lead, _opt(dq_out, dev, "dq_out", dt, q.shape), _opt(dk_out, dev, "dk_out", dt, k.shape), *tail,
            g["dq"].data_ptr(), g["dk"].data_ptr(), *(None if g[n] is None else g[n].data_ptr() for n in ("dq_weight", "dk_weight")),
            *sizes, None if ws is None else _on(ws, dev, "ws"), 0 if ws is None else ws.numel() * ws.element_size(), stream)
        if rc:
            _check("gdn2_qk_norm_rope_bwd", rc)
        return g

    return _here(q, call)


class QkNormRope(torch.autograd.Function):
    """autograd wrapper of the query/key norm and rotation."""

    @staticmethod
    def forward(ctx, q, k, positions, inv_freq, axes, q_weight, k_weight, eps, interleaved):
        out = gdn2_qk_norm_rope_fwd(q, k, positions, inv_freq, axes, q_weight, k_weight, eps, interleaved)
        ctx.save_for_backward(q, k, positions, inv_freq, axes, q_weight, k_weight)
        ctx.eps, ctx.interleaved = eps, interleaved
        return out

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dq_out, dk_out):
        q, k, positions, inv_freq, axes, q_weight, k_weight = ctx.saved_tensors
        g = gdn2_qk_norm_rope_bwd(q, k, dq_out.contiguous(), dk_out.contiguous(), positions, inv_freq, axes, q_weight,
                                  k_weight, ctx.eps, ctx.interleaved)
        return g["dq"], g["dk"], None, None, None, g["dq_weight"], g["dk_weight"], None, None


def qk_norm_rope(q, k, positions, inv_freq, axes=None, q_weight=None, k_weight=None, eps: Optional[float] = 1e-6,
                 interleaved: bool = False):
    """Differentiable :func:`gdn2_qk_norm_rope_fwd` (gradients of q, k and the weights). Returns ``(q_out, k_out)``."""
    if inv_freq.requires_grad and torch.is_grad_enabled():
        raise ValueError("inv_freq has no gradient: pass it detached")
    return QkNormRope.apply(q, k, positions, inv_freq, axes, q_weight, k_weight, eps, interleaved)


def gdn2_device_status(device=None) -> int:
    """Synchronise the current stream and return the kernels' device-side status since the previous call: 0,
    GDN2_ERR_TIMEOUT if a bounded wait gave up, or GDN2_ERR_INVALID if a kernel met arguments that are wrong (an
    inconsistent cu_seqlens, a bad slot or axis). The record is cleared; :func:`last_error` names all of it."""
    with torch.cuda.device(device):   # the record is the current device's
        return int(lib().gdn2_device_status(torch.cuda.current_stream().cuda_stream))


def last_error() -> str:
    return lib().gdn2_last_error().decode()


def trace_enable(on: bool = True) -> None:
    """Start (or stop) per-kernel event timing of the library's launches."""
    lib().gdn2_trace_enable(1 if on else 0)


def trace_read() -> dict:
    """{kernel name: (launches, summed device ms)} since the last read (waits for the events)."""
    n_max = 32
    names = ctypes.create_string_buffer(1024)
    launches = (ctypes.c_int * n_max)()
    ms = (ctypes.c_double * n_max)()
    n = lib().gdn2_trace_read(names, 1024, ctypes.cast(launches, ctypes.c_void_p), ctypes.cast(ms, ctypes.c_void_p), n_max)
    keys = names.value.decode().split(",") if n else []
    return {k: (int(launches[i]), float(ms[i])) for i, k in enumerate(keys)}


class GatedDeltaRule2(torch.autograd.Function):
    """autograd wrapper: forward keeps the chunk-start states for the backward."""

    @staticmethod
    def forward(ctx, q, k, v, log_alpha, b, w, S0, chunk):
        B, T, H, Dk = q.shape
        Dv = v.shape[-1]
        need = gdn2_workspace_size(GDN2_OP_BWD, B, T, H, Dk, Dv, chunk, _dt(q))
        ws = torch.empty(max(need, 256), dtype=torch.uint8, device=q.device)
        o, ST = gdn2_fwd(q, k, v, log_alpha, b, w, S0, chunk=chunk, save_states=True, ws=ws)
        ctx.save_for_backward(q, k, v, log_alpha, b, w, S0, ws)
        ctx.chunk = chunk
        return o, ST

    @staticmethod
    def backward(ctx, do, dST):
        q, k, v, log_alpha, b, w, S0, ws = ctx.saved_tensors
        g = gdn2_bwd(q, k, v, log_alpha, b, w, do.contiguous(), S0,
                     None if dST is None else dST.contiguous(), chunk=ctx.chunk,
                     want_dS0=S0 is not None, states_saved=True, ws=ws)
        return g["dq"], g["dk"], g["dv"], g["dlog_alpha"], g["db"], g["dw"], g["dS0"], None


def gated_delta_rule2(q, k, v, log_alpha, b, w, S0=None, chunk: int = 64):
    """Differentiable Gated Delta Rule-2 operator. Returns ``(o, S_T)``."""
    return GatedDeltaRule2.apply(q, k, v, log_alpha, b, w, S0, chunk)
