"""Thin Python binding of libkda.so (the C ABI in include/kda.h).

Argument marshalling only: every step of the computation runs in the HIP
kernels behind the C ABI.  torch supplies device memory and the current
stream.  There is no fallback: if libkda.so is missing or a call is rejected,
an exception is raised.
"""

from __future__ import annotations

import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libkda.so")

KDA_F32, KDA_BF16 = 0, 1
QK_L2NORM, BETA_SIGMOID, GATE_IN_KERNEL = 1, 2, 4
FLAGS_DEFAULT = 7
GATE_SOFTPLUS = 8  # with GATE_IN_KERNEL: the unbounded KDA v1 gate -exp(A_log) softplus(z)

EXPORTS = (
    "kda_safe_chunk_size", "kda_chunk_fwd_workspace", "kda_chunk_fwd", "kda_chunk_fwd_timed",
    "kda_chunk_fwd_kernel_count", "kda_chunk_fwd_noalloc", "kda_chunk_fwd_conv", "kda_layer_fwd_workspace",
    "kda_layer_fwd", "kda_step", "kda_chunk_fwd_grouped", "kda_step_grouped",
    "kda_segment_compose", "kda_segment_fixup", "kda_short_conv", "kda_output_gate",
    "kda_chunk_bwd_workspace", "kda_chunk_bwd", "kda_chunk_bwd_grouped_workspace", "kda_chunk_bwd_grouped",
    "kda_rotary_freqs", "kda_rotary", "kda_attn_fwd_workspace", "kda_attn_fwd", "kda_attn_bwd_workspace",
    "kda_attn_bwd", "kda_cache_append", "kda_attn_step_workspace", "kda_attn_step",
    "kda_cache_fork", "kda_cache_reserve", "kda_cache_free", "kda_cache_compact", "kda_cache_copy",
    "kda_attn_shared_workspace", "kda_attn_shared", "kda_state_reorder",
    "kda_beam_select_workspace", "kda_beam_select",
    "kda_status_string",
)

_lib = None


class KDAError(RuntimeError):
    def __init__(self, fn: str, status: int, msg: str):
        super().__init__(f"{fn} failed with status {status}: {msg}")
        self.status = status


def load() -> ctypes.CDLL:
    """Load libkda.so and declare the prototypes (raises if it is not built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                           "`python -m gated_delta_rule_82_amd.build` (hipcc, gfx950)")
    L = ctypes.CDLL(LIB_PATH)
    P, I, F, U, S = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_uint, ctypes.c_size_t
    L.kda_safe_chunk_size.argtypes = [F, I]
    L.kda_safe_chunk_size.restype = I
    L.kda_chunk_fwd_workspace.argtypes = [I, I, I, I, I, I, I]
    L.kda_chunk_fwd_workspace.restype = S
    L.kda_chunk_fwd.argtypes = [P] * 11 + [I] * 6 + [F, U, I, P, S, P]
    L.kda_chunk_fwd.restype = I
    L.kda_chunk_fwd_timed.argtypes = [P] * 11 + [I] * 6 + [F, U, I, P, S, P, P, I]
    L.kda_chunk_fwd_timed.restype = I
    L.kda_chunk_fwd_kernel_count.argtypes = [I] * 7
    L.kda_chunk_fwd_kernel_count.restype = I
    L.kda_chunk_fwd_noalloc.argtypes = [P] * 11 + [I] * 6 + [F, U, I, P]
    L.kda_chunk_fwd_noalloc.restype = I
    L.kda_chunk_fwd_conv.argtypes = [P] * 12 + [I] * 6 + [F, U, I, P, S, P]
    L.kda_chunk_fwd_conv.restype = I
    L.kda_layer_fwd_workspace.argtypes = [I, I, I, I, I, I, I]
    L.kda_layer_fwd_workspace.restype = S
    L.kda_layer_fwd.argtypes = [P] * 14 + [I] * 6 + [F, U, I, P, S, P]
    L.kda_layer_fwd.restype = I
    L.kda_step.argtypes = [P] * 8 + [I] * 4 + [F, U, I, P]
    L.kda_step.restype = I
    L.kda_segment_compose.argtypes = [I, P, P, P, P, I, I, I, I, P]
    L.kda_segment_compose.restype = I
    L.kda_segment_fixup.argtypes = [I, P, P, P, P, I, I, I, I, I, I, P]
    L.kda_segment_fixup.restype = I
    L.kda_short_conv.argtypes = [P] * 6 + [I] * 5 + [P]
    L.kda_short_conv.restype = I
    L.kda_output_gate.argtypes = [P] * 4 + [I] * 5 + [P]
    L.kda_output_gate.restype = I
    L.kda_chunk_fwd_grouped.argtypes = [P] * 12 + [I] * 7 + [F, U, I, P, S, P]
    L.kda_chunk_fwd_grouped.restype = I
    L.kda_step_grouped.argtypes = [P] * 9 + [I] * 5 + [F, U, I, P]
    L.kda_step_grouped.restype = I
    L.kda_chunk_bwd_workspace.argtypes = [I] * 5
    L.kda_chunk_bwd_workspace.restype = S
    L.kda_chunk_bwd.argtypes = [P] * 16 + [I] * 5 + [F, U, I, P, S, P]
    L.kda_chunk_bwd.restype = I
    L.kda_chunk_bwd_grouped_workspace.argtypes = [I] * 7
    L.kda_chunk_bwd_grouped_workspace.restype = S
    L.kda_chunk_bwd_grouped.argtypes = [P] * 18 + [I] * 6 + [F, U, I, P, S, P]
    L.kda_chunk_bwd_grouped.restype = I
    D = ctypes.c_double
    L.kda_rotary_freqs.argtypes = [P, P, I, D, I, D, I, D, D]
    L.kda_rotary_freqs.restype = I
    L.kda_rotary.argtypes = [P] * 6 + [I] * 10 + [F, U, I, P]
    L.kda_rotary.restype = I
    L.kda_attn_fwd_workspace.argtypes = [I] * 7
    L.kda_attn_fwd_workspace.restype = S
    L.kda_attn_fwd.argtypes = [P] * 7 + [I] * 9 + [F, I, I, I, P, S, P]
    L.kda_attn_fwd.restype = I
    L.kda_attn_bwd_workspace.argtypes = [I] * 7
    L.kda_attn_bwd_workspace.restype = S
    L.kda_attn_bwd.argtypes = [P] * 11 + [I] * 9 + [F, I, I, I, P, S, P]
    L.kda_attn_bwd.restype = I
    L.kda_cache_append.argtypes = [P] * 9 + [I] * 9 + [I, P]
    L.kda_cache_append.restype = I
    L.kda_attn_step_workspace.argtypes = [I] * 6
    L.kda_attn_step_workspace.restype = S
    L.kda_attn_step.argtypes = [P] * 9 + [I] * 9 + [F, I, I, P, S, P]
    L.kda_attn_step.restype = I
    L.kda_cache_fork.argtypes = [P] * 6 + [I] * 7 + [P]
    L.kda_cache_fork.restype = I
    L.kda_cache_reserve.argtypes = [P] * 7 + [I] * 5 + [P]
    L.kda_cache_reserve.restype = I
    L.kda_cache_free.argtypes = [P] * 4 + [I] * 4 + [P]
    L.kda_cache_free.restype = I
    L.kda_cache_compact.argtypes = [P] * 8 + [I] * 3 + [P]
    L.kda_cache_compact.restype = I
    L.kda_cache_copy.argtypes = [P] * 11 + [I] * 6 + [P]
    L.kda_cache_copy.restype = I
    L.kda_attn_shared_workspace.argtypes = [I] * 7
    L.kda_attn_shared_workspace.restype = S
    L.kda_attn_shared.argtypes = [P] * 11 + [I] * 10 + [F, I, I, P, S, P]
    L.kda_attn_shared.restype = I
    L.kda_state_reorder.argtypes = [P] * 3 + [I] * 3 + [S, P]
    L.kda_state_reorder.restype = I
    L.kda_beam_select_workspace.argtypes = [I] * 5
    L.kda_beam_select_workspace.restype = S
    L.kda_beam_select.argtypes = [P] * 6 + [I] * 7 + [P, S, P]
    L.kda_beam_select.restype = I
    L.kda_status_string.argtypes = [I]
    L.kda_status_string.restype = ctypes.c_char_p
    _lib = L
    return L


def status_string(status: int) -> str:
    return load().kda_status_string(status).decode()


def _check(fn: str, status: int):
    if status != 0:
        raise KDAError(fn, status, status_string(status))


def _dt(t: torch.dtype) -> int:
    if t == torch.float32:
        return KDA_F32
    if t == torch.bfloat16:
        return KDA_BF16
    raise TypeError(f"unsupported dtype {t}; use float32 or bfloat16")


def _ptr(t):
    if t is None:
        return None
    if not t.is_cuda or not t.is_contiguous():
        raise ValueError("tensors must be contiguous device tensors")
    return t.data_ptr()


def _stream(device) -> int:
    return torch.cuda.current_stream(device).cuda_stream


def safe_chunk_size(g_min: float = -5.0, dtype: torch.dtype = torch.bfloat16) -> int:
    return load().kda_safe_chunk_size(g_min, _dt(dtype))


def workspace_bytes(B, T, H, Dk, Dv, chunk=64, dtype=torch.bfloat16) -> int:
    return load().kda_chunk_fwd_workspace(B, T, H, Dk, Dv, chunk, _dt(dtype))


def kernel_count(B, T, H, Dk, Dv, chunk=64, dtype=torch.bfloat16) -> int:
    """Kernels one chunk_fwd call launches (intra and inter alternate over slices)."""
    return load().kda_chunk_fwd_kernel_count(B, T, H, Dk, Dv, chunk, _dt(dtype))


def _event_handles(events):
    for e in events:
        if e.cuda_event == 0:  # torch creates the HIP event on its first record
            e.record()
    return (ctypes.c_void_p * len(events))(*[e.cuda_event for e in events])


def chunk_fwd(q, k, v, z, beta_raw, A_log, S0=None, *, chunk=64, g_min=-5.0,
              flags=FLAGS_DEFAULT, want_M=False, want_P=False, o=None, S_out=None,
              M_out=None, P_out=None, workspace=None, events=None, dt_bias=None):
    """Chunkwise KDA forward.  Returns (o, S_out) plus M and/or P when asked.

    `events` (optional): a list of torch.cuda.Event(enable_timing=True), at
    least kernel_count(...) + 1 (kda_chunk_fwd_timed): events[0] is recorded
    before the first kernel and events[k + 1] after kernel k.
    Grouped value heads (v, z, beta_raw with HV = a multiple of q's H heads)
    or a gate bias `dt_bias` [HV, Dk] fp32 run kda_chunk_fwd_grouped.
    """
    B, T, Hq, Dk = q.shape
    H = v.shape[2]
    Dv = v.shape[-1]
    grouped = Hq != H or dt_bias is not None
    if grouped and events is not None:
        raise ValueError("grouped heads / dt_bias run the plain call only")
    dt = q.dtype
    dev = q.device
    if o is None:
        o = torch.empty(B, T, H, Dv, dtype=dt, device=dev)
    if S_out is None:
        S_out = torch.empty(B, H, Dk, Dv, dtype=torch.float32, device=dev)
    if want_M and M_out is None:
        M_out = torch.empty(B, H, Dk, Dk, dtype=torch.float32, device=dev)
    if want_P and P_out is None:
        P_out = torch.empty(B, T, H, Dk, dtype=dt, device=dev)
    need = workspace_bytes(B, T, H, Dk, Dv, chunk, dt)
    if workspace is None or workspace.numel() < need:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=dev)
    args = (_ptr(q), _ptr(k), _ptr(v), _ptr(z), _ptr(beta_raw), _ptr(A_log), _ptr(S0),
            _ptr(o), _ptr(S_out), _ptr(M_out), _ptr(P_out),
            B, T, H, Dk, Dv, chunk, g_min, flags, _dt(dt),
            _ptr(workspace), workspace.numel(), _stream(dev))
    if grouped:
        gargs = (_ptr(q), _ptr(k), _ptr(v), _ptr(z), _ptr(beta_raw), _ptr(A_log), _ptr(dt_bias), _ptr(S0),
                 _ptr(o), _ptr(S_out), _ptr(M_out), _ptr(P_out),
                 B, T, Hq, H, Dk, Dv, chunk, g_min, flags, _dt(dt),
                 _ptr(workspace), workspace.numel(), _stream(dev))
        _check("kda_chunk_fwd_grouped", load().kda_chunk_fwd_grouped(*gargs))
    elif events is None:
        _check("kda_chunk_fwd", load().kda_chunk_fwd(*args))
    else:
        evs = _event_handles(events)
        _check("kda_chunk_fwd_timed", load().kda_chunk_fwd_timed(*args, evs, len(events)))
    out = [o, S_out]
    if want_M:
        out.append(M_out)
    if want_P:
        out.append(P_out)
    return tuple(out)


def chunk_fwd_conv(q, k, v, z, beta_raw, A_log, conv_w, conv_b=None, conv_state=None, S0=None, *, chunk=64,
                   g_min=-5.0, flags=FLAGS_DEFAULT, o=None, S_out=None, workspace=None):
    """kda_chunk_fwd_conv: the core on SiLU(ShortConv_4(.)) of the raw q, k, v.
    conv_w [H*(2 Dk + Dv), 4] fp32 (q channels, then k, then v), conv_b the
    same channels or None, conv_state [B, 3, H*(2 Dk + Dv)] in the input
    dtype or None.  Returns (o, S_out)."""
    B, T, H, Dk = q.shape
    Dv = v.shape[-1]
    dt = q.dtype
    dev = q.device
    if o is None:
        o = torch.empty(B, T, H, Dv, dtype=dt, device=dev)
    if S_out is None:
        S_out = torch.empty(B, H, Dk, Dv, dtype=torch.float32, device=dev)
    need = workspace_bytes(B, T, H, Dk, Dv, chunk, dt)
    if workspace is None or workspace.numel() < need:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=dev)
    _check("kda_chunk_fwd_conv",
           load().kda_chunk_fwd_conv(_ptr(q), _ptr(k), _ptr(v), _ptr(z), _ptr(beta_raw), _ptr(A_log), _ptr(S0),
                                     _ptr(conv_w), _ptr(conv_b), _ptr(conv_state), _ptr(o), _ptr(S_out),
                                     B, T, H, Dk, Dv, chunk, g_min, flags, _dt(dt),
                                     _ptr(workspace), workspace.numel(), _stream(dev)))
    return o, S_out


def layer_workspace_bytes(B, T, H, Dk, Dv, chunk=64, dtype=torch.bfloat16) -> int:
    return int(load().kda_layer_fwd_workspace(B, T, H, Dk, Dv, chunk, _dt(dtype)))


def layer_fwd(q, k, v, z, beta_raw, A_log, gate, gate_weight=None, S0=None, *, conv_w=None, conv_b=None,
              conv_state=None, chunk=64, g_min=-5.0, flags=FLAGS_DEFAULT, y=None, S_out=None, workspace=None):
    """kda_layer_fwd: the layer body without its projections, with the output
    side sigmoid(gate) * HeadRMSNorm(o) * gate_weight applied inside the core's
    output stores (and the input-side convolution when conv_w is given, as in
    chunk_fwd_conv).  gate [B,T,H,Dv] in the input dtype, gate_weight [Dv] fp32
    or None.  Returns (y, S_out)."""
    B, T, H, Dk = q.shape
    Dv = v.shape[-1]
    dt = q.dtype
    dev = q.device
    if y is None:
        y = torch.empty(B, T, H, Dv, dtype=dt, device=dev)
    if S_out is None:
        S_out = torch.empty(B, H, Dk, Dv, dtype=torch.float32, device=dev)
    need = layer_workspace_bytes(B, T, H, Dk, Dv, chunk, dt)
    if workspace is None or workspace.numel() < need:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=dev)
    _check("kda_layer_fwd",
           load().kda_layer_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(z), _ptr(beta_raw), _ptr(A_log), _ptr(S0),
                                _ptr(conv_w), _ptr(conv_b), _ptr(conv_state), _ptr(gate), _ptr(gate_weight),
                                _ptr(y), _ptr(S_out), B, T, H, Dk, Dv, chunk, g_min, flags, _dt(dt),
                                _ptr(workspace), workspace.numel(), _stream(dev)))
    return y, S_out


def chunk_fwd_noalloc(q, k, v, z, beta_raw, A_log, S0=None, *, chunk=64, g_min=-5.0,
                      flags=FLAGS_DEFAULT, want_M=False, want_P=False, o=None, S_out=None,
                      M_out=None, P_out=None):
    """kda_chunk_fwd_noalloc: chunk_fwd without a workspace (the library's
    built-in device scratch; calls on one GPU must not overlap in time).
    Outputs not passed are allocated here by torch, before the call."""
    B, T, H, Dk = q.shape
    Dv = v.shape[-1]
    dt = q.dtype
    dev = q.device
    if o is None:
        o = torch.empty(B, T, H, Dv, dtype=dt, device=dev)
    if S_out is None:
        S_out = torch.empty(B, H, Dk, Dv, dtype=torch.float32, device=dev)
    if want_M and M_out is None:
        M_out = torch.empty(B, H, Dk, Dk, dtype=torch.float32, device=dev)
    if want_P and P_out is None:
        P_out = torch.empty(B, T, H, Dk, dtype=dt, device=dev)
    _check("kda_chunk_fwd_noalloc",
           load().kda_chunk_fwd_noalloc(_ptr(q), _ptr(k), _ptr(v), _ptr(z), _ptr(beta_raw), _ptr(A_log), _ptr(S0),
                                        _ptr(o), _ptr(S_out), _ptr(M_out), _ptr(P_out),
                                        B, T, H, Dk, Dv, chunk, g_min, flags, _dt(dt), _stream(dev)))
    out = [o, S_out]
    if want_M:
        out.append(M_out)
    if want_P:
        out.append(P_out)
    return tuple(out)


def step(q, k, v, z, beta_raw, A_log, S, *, g_min=-5.0, flags=FLAGS_DEFAULT, o=None, dt_bias=None):
    """One decode step; S [B,HV,Dk,Dv] fp32 is updated in place.  Returns o.
    q, k have H heads, v, z, beta_raw HV (a multiple of H; grouped heads and
    dt_bias run kda_step_grouped)."""
    B, Hq, Dk = q.shape
    H = v.shape[1]
    Dv = v.shape[-1]
    if o is None:
        o = torch.empty(B, H, Dv, dtype=q.dtype, device=q.device)
    if Hq != H or dt_bias is not None:
        st = load().kda_step_grouped(_ptr(q), _ptr(k), _ptr(v), _ptr(z), _ptr(beta_raw), _ptr(A_log),
                                     _ptr(dt_bias), _ptr(S), _ptr(o), B, Hq, H, Dk, Dv, g_min, flags,
                                     _dt(q.dtype), _stream(q.device))
        _check("kda_step_grouped", st)
        return o
    st = load().kda_step(_ptr(q), _ptr(k), _ptr(v), _ptr(z), _ptr(beta_raw), _ptr(A_log),
                         _ptr(S), _ptr(o), B, H, Dk, Dv, g_min, flags, _dt(q.dtype),
                         _stream(q.device))
    _check("kda_step", st)
    return o


def segment_compose(M, S_tilde, S_in=None, *, S_prefix=None):
    """Prefix scan S_s = M_s S_{s-1} + S_tilde_s; M [n,B,H,Dk,Dk], S_tilde [n,B,H,Dk,Dv]."""
    n, B, H, Dk, Dv = S_tilde.shape
    if S_prefix is None:
        S_prefix = torch.empty_like(S_tilde)
    st = load().kda_segment_compose(n, _ptr(M), _ptr(S_tilde), _ptr(S_in), _ptr(S_prefix),
                                    B, H, Dk, Dv, _stream(S_tilde.device))
    _check("kda_segment_compose", st)
    return S_prefix


def segment_fixup(P, S_prefix, o, S_in=None):
    """o[s] += P[s] @ S_prev[s] in place; P [n,B,Tseg,H,Dk], o [n,B,Tseg,H,Dv]."""
    n, B, Tseg, H, Dk = P.shape
    Dv = o.shape[-1]
    st = load().kda_segment_fixup(n, _ptr(P), _ptr(S_in), _ptr(S_prefix), _ptr(o), B, Tseg,
                                  H, Dk, Dv, _dt(P.dtype), _stream(P.device))
    _check("kda_segment_fixup", st)
    return o


def bwd_workspace_bytes(B, T, H, Dk, Dv):
    return load().kda_chunk_bwd_workspace(B, T, H, Dk, Dv)


def chunk_bwd(q, k, v, z, beta_raw, A_log, dout, S0=None, dS_T=None, *, g_min=-5.0, flags=FLAGS_DEFAULT,
              want_dS0=True, workspace=None, dt_bias=None):
    """Backward of chunk_fwd: gradients of L = sum(dout * o) + sum(dS_T * S_T).
    Returns a dict dq, dk, dv, dz, dbeta_raw (input dtype), dA_log [H] and,
    when asked, dS0 [B,H,Dk,Dv] (fp32).  Grouped value heads (v with more
    heads than q) or a gate bias `dt_bias` run kda_chunk_bwd_grouped, which
    adds ddt_bias [HV, Dk] (fp32) when a bias is given."""
    B, T, Hq, Dk = q.shape
    H = v.shape[2]
    Dv = v.shape[-1]
    dt = q.dtype
    dev = q.device
    grouped = Hq != H or dt_bias is not None
    g = {"dq": torch.empty_like(q), "dk": torch.empty_like(k), "dv": torch.empty_like(v),
         "dz": torch.empty_like(z), "dbeta_raw": torch.empty_like(beta_raw),
         "dA_log": torch.empty(H, dtype=torch.float32, device=dev)}
    g["dS0"] = torch.empty(B, H, Dk, Dv, dtype=torch.float32, device=dev) if want_dS0 else None
    if dt_bias is not None:
        g["ddt_bias"] = torch.empty(H, Dk, dtype=torch.float32, device=dev)
    if grouped:
        need = load().kda_chunk_bwd_grouped_workspace(B, T, Hq, H, Dk, Dv, 1 if dt_bias is not None else 0)
    else:
        need = bwd_workspace_bytes(B, T, H, Dk, Dv)
    if workspace is None or workspace.numel() < need:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=dev)
    if grouped:
        st = load().kda_chunk_bwd_grouped(
            _ptr(q), _ptr(k), _ptr(v), _ptr(z), _ptr(beta_raw), _ptr(A_log), _ptr(dt_bias), _ptr(S0), _ptr(dout),
            _ptr(dS_T), _ptr(g["dq"]), _ptr(g["dk"]), _ptr(g["dv"]), _ptr(g["dz"]), _ptr(g["dbeta_raw"]),
            _ptr(g["dA_log"]), _ptr(g.get("ddt_bias")), _ptr(g["dS0"]),
            B, T, Hq, H, Dk, Dv, g_min, flags, _dt(dt), _ptr(workspace), workspace.numel(), _stream(dev))
        _check("kda_chunk_bwd_grouped", st)
    else:
        st = load().kda_chunk_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(z), _ptr(beta_raw), _ptr(A_log), _ptr(S0),
                                  _ptr(dout), _ptr(dS_T), _ptr(g["dq"]), _ptr(g["dk"]), _ptr(g["dv"]), _ptr(g["dz"]),
                                  _ptr(g["dbeta_raw"]), _ptr(g["dA_log"]), _ptr(g["dS0"]),
                                  B, T, H, Dk, Dv, g_min, flags, _dt(dt), _ptr(workspace), workspace.numel(),
                                  _stream(dev))
        _check("kda_chunk_bwd", st)
    return g


def short_conv(x, w, bias=None, *, state_in=None, state_out=None, silu=True, y=None):
    """y = SiLU(ShortConv(x)) (silu=False: the convolution alone) for x [B,T,C]
    (or [B,T,H,D], flattened to C = H*D); w [C,4] fp32 (tap 3 is the current
    token), bias [C] fp32 or None.  state_in / state_out [B,3,C] in x's dtype
    carry the last three inputs between calls (state_out may be state_in when
    T <= 32).  Returns y shaped like x."""
    shape = x.shape
    B, T = shape[0], shape[1]
    C = 1
    for d in shape[2:]:
        C *= d
    if y is None:
        y = torch.empty_like(x)
    st = load().kda_short_conv(_ptr(x), _ptr(w), _ptr(bias), _ptr(state_in), _ptr(state_out), _ptr(y),
                               B, T, C, 1 if silu else 0, _dt(x.dtype), _stream(x.device))
    _check("kda_short_conv", st)
    return y


def output_gate(o, gate, weight=None, *, y=None):
    """y = sigmoid(gate) * HeadRMSNorm(o) * weight for o, gate [B,T,H,Dv];
    weight [Dv] fp32 or None.  y may be o or gate (in place)."""
    B, T, H, Dv = o.shape
    if y is None:
        y = torch.empty_like(o)
    st = load().kda_output_gate(_ptr(o), _ptr(gate), _ptr(weight), _ptr(y), B, T, H, Dv,
                                _dt(o.dtype), _stream(o.device))
    _check("kda_output_gate", st)
    return y


# ---------------------------------------------------------------- softmax attention

ROTARY_SCALINGS = {"none": 0, "linear": 1, "ntk": 2, "yarn": 3}
ROTARY_INTERLEAVED, ROTARY_INVERSE = 1, 2
INT_MAX = 2 ** 31 - 1   # the C ABI's sizes and strides; ctypes would drop the bits above without a word


def _int32(name, n):
    if not -INT_MAX <= n <= INT_MAX:
        raise ValueError(f"{name} = {n} does not fit in 32 bits")
    return n


def _launch(name, dev, *args):
    """Calls an entry point on the current stream of `dev`, which becomes the current
    device for the call (a null stream handle names the current device's stream)."""
    fn = getattr(_lib or load(), name)
    if torch._C._cuda_getDevice() == dev.index:
        st = fn(*args, torch._C._cuda_getCurrentRawStream(dev.index))
    else:
        with torch.cuda.device(dev):
            st = fn(*args, torch._C._cuda_getCurrentRawStream(dev.index))
    if st:
        _check(name, st)


def _expect(name, t, shape, dtype, dev):
    """Checks an argument's shape, type and device; None passes."""
    if t is None or (t.dtype is dtype and t.shape == shape and t.device == dev):
        return
    if t.dtype != dtype:
        raise TypeError(f"{name} must be a {dtype} tensor, not {t.dtype}")
    if t.device != dev:
        raise ValueError(f"{name} is on {t.device}, expected {dev}")
    raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")


def _like(t):
    """A contiguous tensor of t's shape, type and device (the quickest way to allocate one)."""
    return torch.empty_like(t, memory_format=torch.contiguous_format)


def _rows(name, t):
    """(pointer, row stride in elements, 0: contiguous) of a [B,T,H,D] device tensor
    whose heads are packed and whose tokens lie one stride apart throughout."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if t.numel() > INT_MAX and max(t.shape) > INT_MAX:
        raise ValueError(f"{name} has {max(t.shape)} elements along an axis, more than 32 bits hold")
    if t.is_contiguous():
        return t.data_ptr(), 0
    B, T, H, D = t.shape
    sb, st, sh, sd = t.stride()
    if (D > 1 and sd != 1) or (H > 1 and sh != D):
        raise ValueError(f"the heads of {name} must be contiguous")
    ld = st if T > 1 else sb if B > 1 else H * D
    if ld < H * D or (T > 1 and B > 1 and sb != T * st):
        raise ValueError(f"the tokens of {name} must lie one stride apart")
    if ld > INT_MAX:
        raise ValueError(f"the tokens of {name} lie {ld} elements apart, more than 32 bits hold")
    return t.data_ptr(), ld


def _attn_shapes(q, k, v, q_len, kv_len):
    if q.dim() != 4 or k.dim() != 4:
        raise ValueError("q and k must be [B,T,H,D]")
    B, Tq, H, D = q.shape
    Tk, HK = k.shape[1], k.shape[2]
    _expect("k", k, (B, Tk, HK, D), q.dtype, q.device)
    _expect("v", v, (B, Tk, HK, D), q.dtype, q.device)
    _expect("q_len", q_len, (B,), torch.int32, q.device)
    _expect("kv_len", kv_len, (B,), torch.int32, q.device)
    return B, Tq, Tk, H, HK, D


def _workspace(need, given, dev):
    """The caller's workspace where it has `need` bytes, else (as for the chunkwise calls) one
    allocated for this call; None where none is needed.  One on another device is refused."""
    if given is not None:
        if given.device != dev:
            raise ValueError(f"workspace is on {given.device}, expected {dev}")
        if given.numel() * given.element_size() >= need:
            return given
    return torch.empty(need, dtype=torch.uint8, device=dev) if need else None


def _ws_args(ws):
    return (None, 0) if ws is None else (_ptr(ws), ws.numel() * ws.element_size())


def rotary_freqs(rot, *, base=10000.0, scaling="none", factor=1.0, trained=0, beta_fast=32.0, beta_slow=1.0,
                 device="cuda"):
    """kda_rotary_freqs: (inv_freq [rot/2] fp64 on `device`, scale) for `rotary`.
    scaling: "none", "linear", "ntk" or "yarn" (by parts; needs `trained`)."""
    rot, trained = _int32("rot", int(rot)), _int32("trained", trained)
    out = torch.empty(max(rot, 0) // 2, dtype=torch.float64)
    scale = ctypes.c_float()
    _check("kda_rotary_freqs",
           load().kda_rotary_freqs(out.data_ptr(), ctypes.addressof(scale), rot, base, ROTARY_SCALINGS[scaling], factor,
                                   trained, beta_fast, beta_slow))
    return out.to(device), scale.value


def rotary(q, k, inv_freq, positions=None, *, scale=1.0, interleaved=False, inverse=False, q_out=None, k_out=None):
    """kda_rotary: the rotary position encoding of q [B,T,H,D] and k [B,T,HK,D]
    (or None) in one pass; rot = 2 * inv_freq.numel().  positions [B,T] int32 or
    None (0 .. T-1).  inverse=True is the transposed map, which takes the
    gradients of the outputs to those of the inputs.  q_out / k_out may be q / k
    (in place).  q, k and the outputs may be parts of packed tensors.  Returns
    (q_out, k_out), or q_out without k."""
    B, T, H, D = q.shape
    dev, dt = q.device, q.dtype
    pairs = inv_freq.numel()
    _expect("inv_freq", inv_freq, (pairs,), torch.float64, dev)
    _expect("positions", positions, (B, T), torch.int32, dev)
    if q_out is None:
        q_out = _like(q)
    else:
        _expect("q_out", q_out, q.shape, dt, dev)
    qp, ldq = _rows("q", q)
    qo, ldqo = _rows("q_out", q_out)
    kp = ko = None
    HK = ldk = ldko = 0
    if k is not None:
        HK = k.shape[2]
        _expect("k", k, (B, T, HK, D), dt, dev)
        if k_out is None:
            k_out = _like(k)
        else:
            _expect("k_out", k_out, k.shape, dt, dev)
        kp, ldk = _rows("k", k)
        ko, ldko = _rows("k_out", k_out)
    _launch("kda_rotary", dev, qp, kp, qo, ko, _ptr(positions), _ptr(inv_freq), B, T, H, HK, D, 2 * pairs, ldq, ldk,
            ldqo, ldko, scale, (ROTARY_INTERLEAVED if interleaved else 0) | (ROTARY_INVERSE if inverse else 0), _dt(dt))
    return q_out if k is None else (q_out, k_out)


def attn_fwd_workspace_bytes(B, Tq, Tk, H, HK, D, dtype=torch.bfloat16) -> int:
    return load().kda_attn_fwd_workspace(B, Tq, Tk, H, HK, D, _dt(dtype))


def attn_fwd(q, k, v, *, scale=None, causal=True, window=0, q_len=None, kv_len=None, o=None, lse=None,
             workspace=None):
    """kda_attn_fwd: softmax attention of q [B,Tq,H,D] over k, v [B,Tk,HK,D]
    (H a multiple of HK; each may be part of a packed tensor).  scale None is
    1/sqrt(D).  causal aligns the last query with the last key; window > 0
    limits a query to that many keys; q_len, kv_len [B] int32 are the lengths of
    padded sequences.  A workspace of less than attn_fwd_workspace_bytes is not
    used.  Returns (o [B,Tq,H,D], lse [B,H,Tq] fp32)."""
    B, Tq, Tk, H, HK, D = _attn_shapes(q, k, v, q_len, kv_len)
    _int32("window", window)
    dev, dt = q.device, q.dtype
    if o is None:
        o = _like(q)
    else:
        _expect("o", o, (B, Tq, H, D), dt, dev)
    if lse is None:
        lse = torch.empty((B, H, Tq), dtype=torch.float32, device=dev)
    else:
        _expect("lse", lse, (B, H, Tq), torch.float32, dev)
    (qp, ldq), (kp, ldk), (vp, ldv) = _rows("q", q), _rows("k", k), _rows("v", v)
    ws = _workspace(attn_fwd_workspace_bytes(B, Tq, Tk, H, HK, D, dt), workspace, dev)
    _launch("kda_attn_fwd", dev, qp, kp, vp, _ptr(q_len), _ptr(kv_len), _ptr(o), _ptr(lse), B, Tq, Tk, H, HK, D, ldq,
            ldk, ldv, D ** -0.5 if scale is None else scale, 1 if causal else 0, window, _dt(dt), *_ws_args(ws))
    return o, lse


def attn_bwd_workspace_bytes(B, Tq, Tk, H, HK, D, dtype=torch.bfloat16) -> int:
    return load().kda_attn_bwd_workspace(B, Tq, Tk, H, HK, D, _dt(dtype))


def attn_bwd(q, k, v, o, lse, dout, *, scale=None, causal=True, window=0, q_len=None, kv_len=None, workspace=None):
    """kda_attn_bwd: gradients of sum(dout * o) from the inputs and results of
    attn_fwd (same scale, masks and lengths).  With causal=False and window=0 k
    and v may be a part of the keys that o and lse were formed with: its dk, dv
    and share of dq.  Returns a dict dq [B,Tq,H,D], dk, dv [B,Tk,HK,D] in the
    input dtype."""
    B, Tq, Tk, H, HK, D = _attn_shapes(q, k, v, q_len, kv_len)
    _int32("window", window)
    dev, dt = q.device, q.dtype
    _expect("o", o, (B, Tq, H, D), dt, dev)
    _expect("lse", lse, (B, H, Tq), torch.float32, dev)
    _expect("dout", dout, (B, Tq, H, D), dt, dev)
    g = {"dq": _like(q), "dk": _like(k), "dv": _like(k)}
    (qp, ldq), (kp, ldk), (vp, ldv) = _rows("q", q), _rows("k", k), _rows("v", v)
    ws = _workspace(attn_bwd_workspace_bytes(B, Tq, Tk, H, HK, D, dt), workspace, dev)
    _launch("kda_attn_bwd", dev, qp, kp, vp, _ptr(q_len), _ptr(kv_len), _ptr(o), _ptr(lse), _ptr(dout), _ptr(g["dq"]),
            _ptr(g["dk"]), _ptr(g["dv"]), B, Tq, Tk, H, HK, D, ldq, ldk, ldv, D ** -0.5 if scale is None else scale, 1
            if causal else 0, window, _dt(dt), *_ws_args(ws))
    return g


def new_cache(n_pages, HK, D, page=64, device="cuda"):
    """Buffers of an 8-bit key/value cache of n_pages pages: (k_cache
    [n_pages,HK,page,D], v_cache [n_pages,HK,D,page], k_scale, v_scale
    [n_pages,HK]).  Nothing needs to start at zero: what was not appended is not read."""
    return (torch.empty((n_pages, HK, page, D), dtype=torch.uint8, device=device),
            torch.empty((n_pages, HK, D, page), dtype=torch.uint8, device=device),
            torch.empty((n_pages, HK), dtype=torch.float32, device=device),
            torch.empty((n_pages, HK), dtype=torch.float32, device=device))


def _cache_fits(k_cache, v_cache, k_scale, v_scale, n_pages, HK, page, D, dev):
    """Whether the four buffers are a cache of that size on `dev`: one test, since each of these calls' latency
    is mostly that of looking at its arguments."""
    return (k_cache.dtype is torch.uint8 and v_cache.dtype is torch.uint8 and k_scale.dtype is torch.float32
            and v_scale.dtype is torch.float32 and k_cache.shape == (n_pages, HK, page, D)
            and v_cache.shape == (n_pages, HK, D, page) and k_scale.shape == v_scale.shape == (n_pages, HK)
            and k_cache.device == v_cache.device == k_scale.device == v_scale.device == dev)


def _expect_cache(k_cache, v_cache, k_scale, v_scale, n_pages, HK, page, D, dev):
    if _cache_fits(k_cache, v_cache, k_scale, v_scale, n_pages, HK, page, D, dev):
        return
    _expect("k_cache", k_cache, (n_pages, HK, page, D), torch.uint8, dev)
    _expect("v_cache", v_cache, (n_pages, HK, D, page), torch.uint8, dev)
    _expect("k_scale", k_scale, (n_pages, HK), torch.float32, dev)
    _expect("v_scale", v_scale, (n_pages, HK), torch.float32, dev)


def _cache_shapes(k_cache, v_cache, k_scale, v_scale, block_table, cache_len, new_len, B, D, dev):
    n_pages, HK, page = k_cache.shape[:3]
    _expect_cache(k_cache, v_cache, k_scale, v_scale, n_pages, HK, page, D, dev)
    _expect("block_table", block_table, (B, block_table.shape[-1]), torch.int32, dev)
    _expect("cache_len", cache_len, (B,), torch.int32, dev)
    _expect("new_len", new_len, (B,), torch.int32, dev)
    return n_pages, HK, page, _int32("block_table's pages", block_table.shape[1])


def cache_append(k, v, k_cache, v_cache, k_scale, v_scale, block_table, cache_len, new_len=None):
    """kda_cache_append: k, v [B,T,HK,D] go, as 8-bit codes, behind the
    cache_len[b] tokens of each sequence (new_len[b] of them, None: T), into the
    pages block_table [B,max_pages] int32 names.  The caches and scales are
    updated in place; cache_len is not.  Sequences of one call must not write the
    same page."""
    B, T, HK, D = k.shape
    dev = k.device
    _expect("v", v, k.shape, k.dtype, dev)
    n_pages, hk, page, max_pages = _cache_shapes(k_cache, v_cache, k_scale, v_scale, block_table, cache_len, new_len,
                                                 B, D, dev)
    if hk != HK:
        raise ValueError(f"the cache has {hk} heads, k has {HK}")
    (kp, ldk), (vp, ldv) = _rows("k", k), _rows("v", v)
    _launch("kda_cache_append", dev, kp, vp, _ptr(k_cache), _ptr(v_cache), _ptr(k_scale), _ptr(v_scale),
            _ptr(block_table), _ptr(cache_len), _ptr(new_len), n_pages, max_pages, B, T, HK, D, page, ldk, ldv,
            _dt(k.dtype))


def attn_step_workspace_bytes(B, Tq, H, HK, D, max_len) -> int:
    return load().kda_attn_step_workspace(B, Tq, H, HK, D, max_len)


def attn_step(q, k_cache, v_cache, k_scale, v_scale, block_table, cache_len, new_len=None, *, scale=None, window=0,
              o=None, workspace=None):
    """kda_attn_step: attention of the newest tokens' q [B,Tq,H,D] over the
    cache, after their cache_append (the same cache_len and new_len: query i of
    sequence b stands at position cache_len[b] + i).  Returns o [B,Tq,H,D]."""
    B, Tq, H, D = q.shape
    _int32("window", window)
    dev, dt = q.device, q.dtype
    n_pages, HK, page, max_pages = _cache_shapes(k_cache, v_cache, k_scale, v_scale, block_table, cache_len, new_len,
                                                 B, D, dev)
    if o is None:
        o = _like(q)
    else:
        _expect("o", o, (B, Tq, H, D), dt, dev)
    qp, ldq = _rows("q", q)
    ws = _workspace(attn_step_workspace_bytes(B, Tq, H, HK, D, max_pages * page), workspace, dev)
    _launch("kda_attn_step", dev, qp, _ptr(k_cache), _ptr(v_cache), _ptr(k_scale), _ptr(v_scale), _ptr(block_table),
            _ptr(cache_len), _ptr(new_len), _ptr(o), n_pages, max_pages, B, Tq, H, HK, D, page, ldq, D ** -0.5 if
            scale is None else scale, window, _dt(dt), *_ws_args(ws))
    return o


# ---------------------------------------------------------------- one prompt, several continuations

def _ints(name, shape, given, dev):
    """The caller's int32 tensor of that shape, or a new one."""
    if given is None:
        return torch.empty(shape if len(shape) > 1 else shape[0], dtype=torch.int32, device=dev)   # quicker without a tuple
    _expect(name, given, shape, torch.int32, dev)
    return given


def _table(block_table, refs):
    """(rows, pages of a row, pages of the cache, device) of a table and the cache's references."""
    if block_table.dim() != 2 or refs.dim() != 1:
        raise ValueError("block_table must be [B,max_pages] and refs [n_pages]")
    dev = block_table.device
    if block_table.dtype is not torch.int32 or refs.dtype is not torch.int32 or refs.device != dev:
        _expect("block_table", block_table, block_table.shape, torch.int32, dev)
        _expect("refs", refs, refs.shape, torch.int32, dev)
    B, width = block_table.shape
    return B, _int32("block_table's pages", width), _int32("refs' pages", refs.shape[0]), dev


def cache_fork(block_table, cache_len, parent, refs, *, page, keep=False, table_out=None, len_out=None):
    """kda_cache_fork: R requests of K_in sequences (block_table [R*K_in,max_pages],
    cache_len [R*K_in] int32) become R of K_out, row c of request r sharing the pages
    of row parent[r,c] (parent [R,K_out] int32, an index within the request; one outside
    makes an empty row).  refs [n_pages] int32 is updated: the old rows' references are
    dropped unless `keep`.  Returns (table_out [R*K_out,max_pages], len_out [R*K_out])."""
    B, width, n_pages, dev = _table(block_table, refs)
    if parent.dim() != 2 or (parent.shape[0] == 0 and B > 0) or (parent.shape[0] > 0 and B % parent.shape[0] != 0):
        raise ValueError(f"parent must be [R,K_out] with R a divisor of the table's {B} rows")
    R, K_out = parent.shape
    _int32("page", page)
    _expect("cache_len", cache_len, (B,), torch.int32, dev)
    _expect("parent", parent, (R, K_out), torch.int32, dev)
    table_out, len_out = _ints("table_out", (R * K_out, width), table_out, dev), _ints("len_out", (R * K_out,), len_out, dev)
    _launch("kda_cache_fork", dev, _ptr(block_table), _ptr(cache_len), _ptr(parent), _ptr(table_out), _ptr(len_out),
            _ptr(refs), _int32("R", R), B // R if R else 0, K_out, width, n_pages, page, 1 if keep else 0)
    return table_out, len_out


def cache_reserve(block_table, cache_len, refs, new_len=None, *, T=1, page, src=None, dst=None, info=None):
    """kda_cache_reserve: pages for new_len[b] (None: T; at most T) tokens behind
    cache_len[b], before their cache_append; block_table and refs are updated in place.
    Returns (src, dst, info): cache_copy's page to copy for each sequence and where to (-1:
    none), and [entries that got no page, free pages left]."""
    B, width, n_pages, dev = _table(block_table, refs)
    _int32("T", T), _int32("page", page)
    _expect("cache_len", cache_len, (B,), torch.int32, dev)
    _expect("new_len", new_len, (B,), torch.int32, dev)
    src = _like(cache_len) if src is None else _ints("src", (B,), src, dev)
    dst = _like(cache_len) if dst is None else _ints("dst", (B,), dst, dev)
    info = _ints("info", (2,), info, dev)
    _launch("kda_cache_reserve", dev, _ptr(block_table), _ptr(refs), _ptr(cache_len), _ptr(new_len), _ptr(src), _ptr(dst),
            _ptr(info), B, T, width, n_pages, page)
    return src, dst, info


def cache_free(block_table, refs, keep_from=None, keep_to=None, *, page):
    """kda_cache_free: gives back the pages of each sequence that hold none of its tokens
    keep_from[b] .. keep_to[b]-1 (int32 [B]; None: 0): all of them without either.
    block_table and refs are updated in place."""
    B, width, n_pages, dev = _table(block_table, refs)
    _int32("page", page)
    _expect("keep_from", keep_from, (B,), torch.int32, dev)
    _expect("keep_to", keep_to, (B,), torch.int32, dev)
    _launch("kda_cache_free", dev, _ptr(block_table), _ptr(refs), _ptr(keep_from), _ptr(keep_to), B, width, n_pages, page)


def cache_compact(block_table, refs, *, table_out=None, refs_out=None):
    """kda_cache_compact: the used pages' new numbers, the first ones of the cache.
    table_out / refs_out may be block_table / refs (in place).  Returns (table_out, refs_out,
    remap [n_pages], src, dst [n_pages // 2], info): remap is a page's new number (-1: free),
    info [copies, used pages].  cache_copy(..., src, dst, count=info) moves the data."""
    B, width, n_pages, dev = _table(block_table, refs)
    table_out = _like(block_table) if table_out is None else _ints("table_out", (B, width), table_out, dev)
    refs_out = _like(refs) if refs_out is None else _ints("refs_out", (n_pages,), refs_out, dev)
    remap, info, src = _like(refs), _ints("info", (2,), None, dev), _ints("src", (n_pages // 2,), None, dev)
    dst = _like(src)
    _launch("kda_cache_compact", dev, _ptr(block_table), _ptr(refs), _ptr(table_out), _ptr(refs_out), _ptr(remap),
            _ptr(src), _ptr(dst), _ptr(info), B, width, n_pages)
    return table_out, refs_out, remap, src, dst, info


def _cache_buffers(k_cache, v_cache, k_scale, v_scale, dev):
    n_pages, HK, page, D = k_cache.shape
    _expect_cache(k_cache, v_cache, k_scale, v_scale, n_pages, HK, page, D, dev)
    return n_pages, HK, page, D


def cache_copy(k_cache, v_cache, k_scale, v_scale, src, dst, *, to=None, count=None):
    """kda_cache_copy: page src[i] of the cache becomes page dst[i] (int32 [n]; -1: none) of
    the cache `to` (its four buffers; None: the same cache), for the first count[0]
    entries where count (int32) is given.  No page may be written twice, nor read by
    the call that writes it."""
    dev = k_cache.device
    n_pages, HK, page, D = _cache_buffers(k_cache, v_cache, k_scale, v_scale, dev)
    n_dst = n_pages
    if to is not None:
        n_dst = to[0].shape[0]
        if _cache_buffers(*to, dev)[1:] != (HK, page, D):
            raise ValueError("the caches' pages differ in shape")
    kt, vt, kst, vst = (k_cache, v_cache, k_scale, v_scale) if to is None else to
    _expect("src", src, (src.numel(),), torch.int32, dev)
    _expect("dst", dst, (src.numel(),), torch.int32, dev)
    if count is not None:
        _expect("count", count, count.shape, torch.int32, dev)
        if count.numel() < 1:
            raise ValueError("count holds no number")
    _launch("kda_cache_copy", dev, _ptr(k_cache), _ptr(v_cache), _ptr(k_scale), _ptr(v_scale), _ptr(kt), _ptr(vt),
            _ptr(kst), _ptr(vst), _ptr(src), _ptr(dst), _ptr(count), _int32("src", src.numel()), n_pages, n_dst, HK, D, page)


def attn_shared_workspace_bytes(B, Tq, H, HK, D, n_groups, max_len) -> int:
    return load().kda_attn_shared_workspace(B, Tq, H, HK, D, n_groups, max_len)


def attn_shared(q, k_cache, v_cache, k_scale, v_scale, block_table, cache_len, group_first, prefix_len, new_len=None, *,
                scale=None, window=0, o=None, workspace=None):
    """kda_attn_shared: attn_step where the sequences group_first[g] .. group_first[g+1]-1
    (int32 [n_groups+1]) have their first prefix_len[g] tokens (int32 [n_groups]) in common:
    their whole pages are read once a group, through its first sequence's row of block_table,
    which has to name them as long as any sequence of the group sees them.
    Returns o [B,Tq,H,D]."""
    B, Tq, H, D = q.shape
    _int32("window", window)
    dev, dt = q.device, q.dtype
    n_pages, HK, page, max_pages = _cache_shapes(k_cache, v_cache, k_scale, v_scale, block_table, cache_len, new_len,
                                                 B, D, dev)
    n_groups = prefix_len.shape[0]
    _expect("prefix_len", prefix_len, (n_groups,), torch.int32, dev)
    _expect("group_first", group_first, (n_groups + 1,), torch.int32, dev)
    if o is None:
        o = _like(q)
    else:
        _expect("o", o, (B, Tq, H, D), dt, dev)
    qp, ldq = _rows("q", q)
    ws = _workspace(attn_shared_workspace_bytes(B, Tq, H, HK, D, n_groups, max_pages * page), workspace, dev)
    _launch("kda_attn_shared", dev, qp, _ptr(k_cache), _ptr(v_cache), _ptr(k_scale), _ptr(v_scale), _ptr(block_table),
            _ptr(cache_len), _ptr(new_len), _ptr(group_first), _ptr(prefix_len), _ptr(o), n_groups, n_pages, max_pages, B, Tq,
            H, HK, D, page, ldq, D ** -0.5 if scale is None else scale, window, _dt(dt), *_ws_args(ws))
    return o


def state_reorder(state, parent, *, out=None):
    """kda_state_reorder: row c of request r of the result is row parent[r,c] of request
    r of state [R*K_in, ...] (parent [R,K_out] int32, an index within the request; zeros for
    one outside).  out=state reorders in place (K_in = K_out, at most 64).  Returns it."""
    if parent.dim() != 2 or state.dim() < 1:
        raise ValueError("parent must be [R,K_out] and state have rows")
    R, K_out = parent.shape
    dev, rows = state.device, state.shape[0]
    if (R == 0 and rows > 0) or (R > 0 and rows % R != 0):
        raise ValueError(f"state's {rows} rows are not those of {R} requests")
    _expect("parent", parent, (R, K_out), torch.int32, dev)
    shape = torch.Size((R * K_out, *state.shape[1:]))
    if out is None:
        out = torch.empty(shape, dtype=state.dtype, device=dev)
    else:
        _expect("out", out, shape, state.dtype, dev)
    row_bytes = state.element_size()
    for n in state.shape[1:]:
        row_bytes *= n
    _launch("kda_state_reorder", dev, _ptr(state), _ptr(out), _ptr(parent), _int32("R", R), rows // R if R else 0,
            _int32("K_out", K_out), row_bytes)
    return out


def beam_select_workspace_bytes(R, K, V, M, dtype=torch.bfloat16) -> int:
    return load().kda_beam_select_workspace(R, K, V, M, _dt(dtype))


def beam_select(logits, scores=None, M=None, *, done=None, end=-1, scores_out=None, parent=None, token=None, workspace=None):
    """kda_beam_select: the M (None: K) best continuations of each request over its K beams
    and V tokens, by scores [R,K] fp32 (None: 0) + log-softmax of logits [R,K,V] (whose rows
    may lie further apart than V; the first one is 16-byte aligned).  Equal ones are in the order of (beam, token).  done [R,K]
    uint8: finished beams, which continue with `end` at no cost.  Returns (scores [R,M]
    fp32, parent [R,M], token [R,M] int32), -infinity, -1, -1 where there are fewer."""
    if logits.dim() != 3:
        raise ValueError("logits must be [R,K,V]")
    R, K, V = logits.shape
    M = K if M is None else _int32("M", M)
    _int32("end", end)
    dev, dt = logits.device, logits.dtype
    if not logits.is_cuda:
        raise ValueError("logits must be a device tensor")
    sr, sk, sv = logits.stride()
    ld = sk if K > 1 else sr if R > 1 else V
    if logits.numel() and ((V > 1 and sv != 1) or ld < V or (R > 1 and K > 1 and sr != K * sk)):
        raise ValueError("the rows of logits must be contiguous and lie one stride apart")
    _expect("scores", scores, (R, K), torch.float32, dev)
    _expect("done", done, (R, K), torch.uint8, dev)
    if scores_out is None:
        scores_out = torch.empty((R, M), dtype=torch.float32, device=dev)
    else:
        _expect("scores_out", scores_out, (R, M), torch.float32, dev)
    parent = torch.empty_like(scores_out, dtype=torch.int32) if parent is None else _ints("parent", (R, M), parent, dev)
    token = _like(parent) if token is None else _ints("token", (R, M), token, dev)
    ws = _workspace(beam_select_workspace_bytes(_int32("R", R), _int32("K", K), _int32("V", V), M, dt), workspace, dev)
    _launch("kda_beam_select", dev, logits.data_ptr(), _ptr(scores), _ptr(done), _ptr(scores_out), _ptr(parent), _ptr(token),
            R, K, V, M, _int32("the rows' stride", ld), end, _dt(dt), *_ws_args(ws))
    return scores_out, parent, token
