"""ctypes binding of include/q3_block.h: argument marshalling only.

The operators between two packed products and behind the last one: products of
many tokens, the gated feed-forward block, residual norms (each with the
gradients of its inputs), the attention sublayer over a paged cache, sampling and
log probabilities.  Every function forwards to the C entry point of the same
name; outputs and workspaces that are not given are allocated here.  A call runs
on the current stream of its tensors' device.

No call is recorded by autograd: results carry no graph, also where an input
requires a gradient.  The backward calls give the gradients and are chained by
hand (or in the backward of a torch.autograd.Function).
"""
from __future__ import annotations

import ctypes
from dataclasses import dataclass
from typing import Optional

import torch

from . import _lib
from ._lib import PackedMatrix, Q3Matrix, c_i32, c_i64, c_vp

c_f32 = ctypes.c_float


class Q3ResidualNormGrads(ctypes.Structure):
    _fields_ = [("dx", c_vp), ("ld_dx", c_i64), ("dr_out", c_vp), ("ld_dr_out", c_i64), ("dr", c_vp),
                ("ld_dr", c_i64), ("dy", c_vp), ("ld_dy", c_i64), ("dgate", c_vp), ("ld_dgate", c_i64),
                ("dpost_weight", c_vp), ("dpre_weight", c_vp)]


class Q3FfnNorms(ctypes.Structure):
    _fields_ = [("pre_weight", c_vp), ("post_weight", c_vp), ("next_weight", c_vp), ("gate", c_vp),
                ("ld_gate", c_i64), ("scale", c_f32), ("eps", c_f32)]


class Q3PagedCache(ctypes.Structure):
    _fields_ = [("k", c_vp), ("v", c_vp), ("pages", c_i64), ("page_stride", c_i64), ("page_size", c_i32),
                ("heads", c_i32), ("head_dim", c_i32)]


class Q3PagedBatch(ctypes.Structure):
    _fields_ = [("sequences", c_i64), ("q_start", c_vp), ("kv_len", c_vp), ("page_table", c_vp), ("ld_table", c_i64),
                ("table_pages", c_i64)]


class Q3HeadNorms(ctypes.Structure):
    _fields_ = [("heads_q", c_i32), ("heads_kv", c_i32), ("head_dim", c_i32), ("rotated", c_i32),
                ("interleaved", c_i32), ("eps", c_f32), ("q_weight", c_vp), ("k_weight", c_vp), ("inv_freq", c_vp)]


class Q3QkvGrads(ctypes.Structure):
    _fields_ = [("d_type", c_i32), ("dq", c_vp), ("ld_dq", c_i64), ("dk", c_vp), ("ld_dk", c_i64), ("dv", c_vp),
                ("ld_dv", c_i64), ("dqkv", c_vp), ("ld_dqkv", c_i64), ("dq_weight", c_vp), ("dk_weight", c_vp)]


_int = ctypes.c_int
_cache = ctypes.POINTER(Q3PagedCache)
_batch = ctypes.POINTER(Q3PagedBatch)
_heads = ctypes.POINTER(Q3HeadNorms)
_mat = ctypes.POINTER(Q3Matrix)

# name -> (restype, argtypes); the same list include/q3_block.h declares.
SIGNATURES = {
    "q3_gemm_workspace_bytes": (c_i64, [c_i64, c_i64, c_i64]),
    "q3_gemm": (_int, [_mat, c_vp, c_i64, c_i64, c_vp, c_i64, c_vp, c_i64, c_vp]),
    "q3_gemm_backward_workspace_bytes": (c_i64, [c_i64, c_i64, c_i64]),
    "q3_gemm_backward": (_int, [_mat, c_vp, c_i64, c_i64, c_vp, c_i64, c_vp, c_i64, c_vp]),
    "q3_glu_workspace_bytes": (c_i64, [c_i64, c_i64, c_i64]),
    "q3_glu": (_int, [_mat, c_vp, c_i64, c_i64, c_i32, c_vp, c_i64, c_vp, c_i64, c_vp, c_i64, c_vp]),
    "q3_glu_backward": (_int, [c_vp, c_i64, c_vp, c_i64, c_i32, c_i64, c_i64, c_vp, c_i64, c_vp]),
    "q3_residual_norm": (_int, [c_vp, c_i64, c_vp, c_vp, c_i64, c_f32, c_vp, c_i64, c_vp, c_i64, c_i32, c_vp, c_vp,
                                c_i64, c_f32, c_i64, c_i64, c_vp]),
    "q3_residual_norm_backward_workspace_bytes": (c_i64, [c_i64, c_i64]),
    "q3_residual_norm_backward": (_int, [c_vp, c_i64, c_vp, c_vp, c_i64, c_f32, c_vp, c_i64, c_i32, c_vp, c_f32,
                                         c_i64, c_i64, ctypes.POINTER(Q3ResidualNormGrads), c_vp, c_i64, c_vp]),
    "q3_ffn_workspace_bytes": (c_i64, [c_i64, c_i64, c_i64]),
    "q3_ffn": (_int, [_mat, _mat, c_i32, ctypes.POINTER(Q3FfnNorms), c_vp, c_i64, c_vp, c_i64, c_i32, c_vp, c_i64,
                      c_i64, c_vp, c_i64, c_vp]),
    "q3_qk_norm_rope": (_int, [_heads, c_vp, c_i64, c_vp, c_vp, c_i64, c_vp, c_i64, c_vp, c_i64, _cache, _batch, c_i64,
                               c_vp]),
    "q3_qk_norm_rope_backward_workspace_bytes": (c_i64, [c_i64, c_i32]),
    "q3_qk_norm_rope_backward": (_int, [_heads, c_vp, c_i64, c_vp, c_i64, ctypes.POINTER(Q3QkvGrads), c_vp, c_i64,
                                        c_vp]),
    "q3_paged_attention_workspace_bytes": (c_i64, [c_i64, c_i64, c_i32, c_i32, c_i32]),
    "q3_paged_attention": (_int, [c_vp, c_i64, c_i32, _cache, _batch, c_f32, c_i32, c_vp, c_i64, c_vp, c_i64, c_vp,
                                  c_i64, c_vp]),
    "q3_logprobs_workspace_bytes": (c_i64, [c_i64, c_i64, c_i32]),
    "q3_logprobs": (_int, [c_vp, c_i64, c_i64, c_i64, c_vp, c_f32, c_i32, c_vp, c_vp, c_vp, c_vp, c_vp, c_vp, c_i64,
                           c_vp]),
    "q3_logprobs_backward": (_int, [c_vp, c_i64, c_i64, c_i64, c_vp, c_f32, c_vp, c_vp, c_vp, c_vp, c_i64, c_i32,
                                    c_vp]),
    "q3_sample_workspace_bytes": (c_i64, [c_i64, c_i64]),
    "q3_sample": (_int, [c_vp, c_i64, c_i64, c_i64, c_vp, c_vp, c_vp, c_vp, c_vp, c_vp, c_i64, c_vp, c_vp, c_vp]),
}

ACTS = {"silu": 0, "gelu": 1}
_R_TYPES = {torch.float32: 0, torch.bfloat16: 1}

_bound = None


def lib():
    """libq3.so with this header's entry points bound."""
    global _bound
    L = _lib.lib()
    if _bound is not L:
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _bound = L
    return L


def _call(name, device, *args):
    """The entry point on the device's current stream, with that device current."""
    fn = getattr(lib(), name)
    index = device.index
    # The raw handle: a Stream object costs 2 us of host time per call.
    stream = torch._C._cuda_getCurrentRawStream(index)
    if index == torch._C._cuda_getDevice():
        status = fn(*args, stream)
    else:
        with torch.cuda.device(device):
            status = fn(*args, stream)
    if status:
        raise _lib.Q3Error(name, status)


def _rows(t, shape, dtype, device, name):
    """A device tensor of exactly this shape and type with contiguous rows that
    do not overlap; returns it."""
    if type(t) is torch.Tensor and t.dtype is dtype and t.shape == shape and t.device == device and t.is_contiguous():
        return t
    if not isinstance(t, torch.Tensor) or t.device != device:
        raise ValueError(f"{name} must be a tensor on {device} (the inputs' device)")
    if t.dtype != dtype or t.shape != shape:
        raise ValueError(f"{name} must be {dtype} of shape {tuple(shape)}, got {t.dtype} {tuple(t.shape)}")
    if shape[-1] > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name} must have contiguous rows")
    if len(shape) == 2 and shape[0] > 1 and t.stride(0) < shape[1]:
        raise ValueError(f"{name} rows overlap (row pitch below the row length)")
    return t


def _vector(t, n, dtype, device, name):
    return None if t is None else _rows(t, (n,), dtype, device, name)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _pitch(t):
    if t is None:
        return 0
    m, n = t.shape
    return n if m <= 1 or n == 0 else t.stride(0)


def _pitch8(t):
    """The row pitch of bf16 token rows; a single row's pitch is what it would
    be padded to (nothing behind the row is read as values)."""
    return t.stride(0) if t.shape[0] > 1 and t.shape[1] else (t.shape[1] + 7) // 8 * 8


def _ws(workspace, nbytes, device):
    if workspace is None:
        return torch.empty(nbytes, dtype=torch.uint8, device=device) if nbytes else None
    return _lib._workspace(workspace, device)


def _ws_args(ws):
    return (None, 0) if ws is None else (ws.data_ptr(), ws.numel() * ws.element_size())


def _matrix(w: PackedMatrix, device):
    for t, name in ((w.code_plane, "code_plane"), (w.scale_plane, "scale_plane"), (w.codebook, "codebook")):
        if t.device != device:
            raise ValueError(f"{name} must be on {device} (the inputs' device)")
    return ctypes.byref(w.desc())


def _tokens(x, cols, name):
    if not isinstance(x, torch.Tensor) or not x.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if x.dim() != 2 or x.shape[1] != cols or x.dtype != torch.bfloat16:
        raise ValueError(f"{name} must be bfloat16 [m][{cols}], got {x.dtype} {tuple(x.shape)}")
    if cols > 1 and x.stride(1) != 1:
        raise ValueError(f"{name} rows must be contiguous")
    if x.shape[0] > 1 and x.stride(0) < cols:
        raise ValueError(f"{name} rows overlap (row pitch below the row length)")
    return x


def _act(act):
    if act not in ACTS:
        raise ValueError(f"act must be one of {sorted(ACTS)}, got {act!r}")
    return ACTS[act]


# ------------------------------------------------------------------ products

def q3_gemm_workspace_bytes(n: int, k: int, m: int) -> int:
    return lib().q3_gemm_workspace_bytes(n, k, m)


def q3_gemm(w: PackedMatrix, x: torch.Tensor, y: torch.Tensor = None, workspace: torch.Tensor = None) -> torch.Tensor:
    """y[m][n] = x[m] . w[n] for any number of tokens (x bfloat16, y float32).
    Not recorded by autograd: q3_gemm_backward gives x's gradient."""
    _tokens(x, w.k, "x")
    m, dev = x.shape[0], x.device
    y = torch.empty((m, w.n), dtype=torch.float32, device=dev) if y is None else \
        _rows(y, (m, w.n), torch.float32, dev, "y")
    ws = _ws(workspace, lib().q3_gemm_workspace_bytes(w.n, w.k, m), dev)
    _call("q3_gemm", dev, _matrix(w, dev), x.data_ptr(), m, _pitch(x), y.data_ptr(), _pitch(y), *_ws_args(ws))
    return y


def q3_gemm_backward_workspace_bytes(n: int, k: int, m: int) -> int:
    return lib().q3_gemm_backward_workspace_bytes(n, k, m)


def q3_gemm_backward(w: PackedMatrix, dy: torch.Tensor, dx: torch.Tensor = None,
                     workspace: torch.Tensor = None) -> torch.Tensor:
    """dx[m][k] = sum_n dy[m][n] w[n][k], the gradient of q3_gemm's x (dy
    bfloat16 with rows pitched to a multiple of 8, dx float32)."""
    _tokens(dy, w.n, "dy")
    m, dev = dy.shape[0], dy.device
    dx = torch.empty((m, w.k), dtype=torch.float32, device=dev) if dx is None else \
        _rows(dx, (m, w.k), torch.float32, dev, "dx")
    ws = _ws(workspace, lib().q3_gemm_backward_workspace_bytes(w.n, w.k, m), dev)
    _call("q3_gemm_backward", dev, _matrix(w, dev), dy.data_ptr(), m, _pitch8(dy), dx.data_ptr(), _pitch(dx),
          *_ws_args(ws))
    return dx


# ------------------------------------------------------------------ gated block

def q3_glu_workspace_bytes(n_gu: int, k: int, m: int) -> int:
    return lib().q3_glu_workspace_bytes(n_gu, k, m)


def q3_glu(gate_up: PackedMatrix, x: torch.Tensor, act: str = "silu", save_pre: bool = False, h: torch.Tensor = None,
           pre: torch.Tensor = None, workspace: torch.Tensor = None):
    """h = act(x . gate) * (x . up) in bfloat16 [m][I] for gate_up = [gate I rows;
    up I rows]; with save_pre (or pre given) -> (h, pre), the pre-activations
    [g; u] float32 [m][2I] that q3_glu_backward takes.  Not recorded by autograd:
    q3_glu_backward, then q3_gemm_backward give x's gradient."""
    _tokens(x, gate_up.k, "x")
    code = _act(act)
    m, dev, inter = x.shape[0], x.device, gate_up.n // 2
    if h is None:
        h = torch.empty((m, inter), dtype=torch.bfloat16, device=dev)
    else:
        _rows(h, (m, inter), torch.bfloat16, dev, "h")
    if pre is not None:
        _rows(pre, (m, gate_up.n), torch.float32, dev, "pre")
    elif save_pre:
        pre = torch.empty((m, gate_up.n), dtype=torch.float32, device=dev)
    ws = _ws(workspace, lib().q3_glu_workspace_bytes(gate_up.n, gate_up.k, m), dev)
    _call("q3_glu", dev, _matrix(gate_up, dev), x.data_ptr(), m, _pitch(x), code, h.data_ptr(), _pitch(h), _ptr(pre),
          _pitch(pre), *_ws_args(ws))
    return h if pre is None else (h, pre)


def q3_glu_backward(pre: torch.Tensor, dh: torch.Tensor, act: str = "silu", dpre: torch.Tensor = None) -> torch.Tensor:
    """The gradient of q3_glu's pre-activations, bfloat16 [m][2I], from pre and
    dh (float32 [m][I]); q3_gemm_backward(gate_up, dpre) is then that of x."""
    code = _act(act)
    if not isinstance(pre, torch.Tensor) or not pre.is_cuda or pre.dim() != 2 or pre.shape[1] % 2:
        raise ValueError("pre must be a device tensor float32 [m][2I]")
    m, two, dev = pre.shape[0], pre.shape[1], pre.device
    _rows(pre, (m, two), torch.float32, dev, "pre")
    _rows(dh, (m, two // 2), torch.float32, dev, "dh")
    dpre = torch.empty((m, two), dtype=torch.bfloat16, device=dev) if dpre is None else \
        _rows(dpre, (m, two), torch.bfloat16, dev, "dpre")
    _call("q3_glu_backward", dev, pre.data_ptr(), _pitch(pre), dh.data_ptr(), _pitch(dh), code, m, two // 2,
          dpre.data_ptr(), _pitch(dpre))
    return dpre


# ------------------------------------------------------------------ residual norms

def _norm_args(r, pre_weight, y, post_weight, gate):
    if not isinstance(r, torch.Tensor) or not r.is_cuda or r.dim() != 2 or r.dtype not in _R_TYPES:
        raise ValueError("r must be a float32 or bfloat16 device tensor [m][n]")
    (m, n), dev = r.shape, r.device
    if not r.is_contiguous():
        _rows(r, (m, n), r.dtype, dev, "r")
    if pre_weight is not None:
        _rows(pre_weight, (n,), torch.float32, dev, "pre_weight")
    if post_weight is not None:
        _rows(post_weight, (n,), torch.float32, dev, "post_weight")
    if y is None and (post_weight is not None or gate is not None):
        raise ValueError("post_weight and gate need y")
    if y is not None:
        _rows(y, (m, n), torch.float32, dev, "y")
    ld_gate = 0
    if gate is not None and gate.dim() == 1:
        _vector(gate, n, torch.float32, dev, "gate")
    elif gate is not None:
        _rows(gate, (m, n), torch.float32, dev, "gate")
        ld_gate = _pitch(gate)
    return m, n, dev, ld_gate


def _next_x(x, want_x, weight, weight_name, r):
    """The caller's bfloat16 output x, or None where it is not wanted."""
    if want_x:
        return _rows(x, r.shape, torch.bfloat16, r.device, "x")
    if x is not None or weight is not None:
        raise ValueError(f"want_x=False takes neither x nor {weight_name}")
    return None


def q3_residual_norm(r: torch.Tensor, pre_weight: torch.Tensor = None, y: torch.Tensor = None,
                     post_weight: torch.Tensor = None, gate: torch.Tensor = None, scale: float = 1.0,
                     eps: float = 1e-6, r_out: torch.Tensor = None, x: torch.Tensor = None, want_x: bool = True):
    """r' = r + scale * gate * norm(y; post_weight) and x = norm(r'; pre_weight)
    -> (r', x): r' in r's type, x bfloat16 (None, and not computed, with want_x
    False).  y None: r' is r itself.  post_weight None: y is not normed.  gate
    float32 [m][n], or [n] for all tokens.  r_out may be r.  Not recorded by
    autograd: q3_residual_norm_backward gives the gradients."""
    m, n, dev, ld_gate = _norm_args(r, pre_weight, y, post_weight, gate)
    if r_out is not None:
        _rows(r_out, (m, n), r.dtype, dev, "r_out")
    elif y is not None:
        r_out = r.new_empty((m, n))
    if want_x and x is None:
        x = r.new_empty((m, n), dtype=torch.bfloat16)
    else:
        x = _next_x(x, want_x, pre_weight, "pre_weight", r)
    if x is None and r_out is None:
        raise ValueError("want_x=False without y or r_out: nothing to compute")
    _call("q3_residual_norm", dev, _ptr(y), _pitch(y), _ptr(post_weight), _ptr(gate), ld_gate, scale, r.data_ptr(),
          _pitch(r), _ptr(r_out), _pitch(r_out), _R_TYPES[r.dtype], _ptr(pre_weight), _ptr(x), _pitch(x), eps, m, n)
    return (r if r_out is None else r_out), x


@dataclass
class ResidualNormGrads:
    """Gradients of q3_residual_norm's inputs (None where there is no such input)."""
    dr: torch.Tensor                         # r's type [m][n]
    dpre_weight: torch.Tensor                # float32 [n]
    dy: Optional[torch.Tensor] = None        # bfloat16 [m][n]
    dgate: Optional[torch.Tensor] = None     # float32, gate's shape
    dpost_weight: Optional[torch.Tensor] = None


def q3_residual_norm_backward(r_out: torch.Tensor, pre_weight: torch.Tensor = None, dx: torch.Tensor = None,
                              dr_out: torch.Tensor = None, y: torch.Tensor = None, post_weight: torch.Tensor = None,
                              gate: torch.Tensor = None, scale: float = 1.0, eps: float = 1e-6,
                              workspace: torch.Tensor = None) -> ResidualNormGrads:
    """From the kept r' (r_out), the gradients dx (float32) of x and dr_out (r's
    type) of r' from later blocks; either may be None (zero)."""
    m, n, dev, ld_gate = _norm_args(r_out, pre_weight, y, post_weight, gate)
    if dx is not None:
        _rows(dx, (m, n), torch.float32, dev, "dx")
    if dr_out is not None:
        _rows(dr_out, (m, n), r_out.dtype, dev, "dr_out")
    # The gradients summed over the tokens share one allocation; bf16 rows are
    # pitched so that q3_gemm_backward takes them as they are.
    wide = (n + 7) // 8 * 8
    sums = torch.empty((3, n), dtype=torch.float32, device=dev).unbind(0)
    g = ResidualNormGrads(r_out.new_empty((m, n)), sums[0])
    if y is not None:
        dy = r_out.new_empty((m, wide), dtype=torch.bfloat16)
        g.dy = dy if wide == n else dy[:, :n]
    if gate is not None:
        g.dgate = y.new_empty((m, n)) if gate.dim() == 2 else sums[2]
    if post_weight is not None:
        g.dpost_weight = sums[1]
    ws = _ws(workspace, lib().q3_residual_norm_backward_workspace_bytes(m, n), dev)
    grads = Q3ResidualNormGrads(_ptr(dx), _pitch(dx), _ptr(dr_out), _pitch(dr_out), g.dr.data_ptr(), n, _ptr(g.dy),
                                wide, _ptr(g.dgate), n, _ptr(g.dpost_weight), g.dpre_weight.data_ptr())
    _call("q3_residual_norm_backward", dev, _ptr(y), _pitch(y), _ptr(post_weight), _ptr(gate), ld_gate, scale,
          r_out.data_ptr(), _pitch(r_out), _R_TYPES[r_out.dtype], _ptr(pre_weight), eps, m, n, ctypes.byref(grads),
          *_ws_args(ws))
    return g


# ------------------------------------------------------------------ feed-forward sublayer

def q3_ffn_workspace_bytes(n_gu: int, k: int, m: int) -> int:
    return lib().q3_ffn_workspace_bytes(n_gu, k, m)


def q3_ffn(gate_up: PackedMatrix, down: PackedMatrix, r: torch.Tensor, pre_weight: torch.Tensor = None,
           post_weight: torch.Tensor = None, gate: torch.Tensor = None, scale: float = 1.0,
           next_weight: torch.Tensor = None, act: str = "silu", eps: float = 1e-6, r_out: torch.Tensor = None,
           x: torch.Tensor = None, workspace: torch.Tensor = None, want_x: bool = True):
    """r' = r + scale * gate * norm(down . h; post_weight), h the gated block of
    norm(r; pre_weight), and x = norm(r'; next_weight) -> (r', x), as the separate
    calls give them; with want_x False x is None and not computed.  r_out may be r.
    For inference: neither h's pre-activations nor the down product are kept, and
    the call is not recorded by autograd; training takes the separate calls."""
    code = _act(act)
    # y, the down product, is the call's own: r's shape stands for it in the checks
    m, n, dev, _ = _norm_args(r, pre_weight, None, None, None)
    _vector(post_weight, n, torch.float32, dev, "post_weight")
    _vector(next_weight, n, torch.float32, dev, "next_weight")
    if n != gate_up.k or down.n != n or 2 * down.k != gate_up.n:
        raise ValueError(f"r [m][{n}], gate_up [{gate_up.n}][{gate_up.k}] and down [{down.n}][{down.k}] do not chain")
    ld_gate = 0
    if gate is not None:
        _rows(gate, (n,) if gate.dim() == 1 else (m, n), torch.float32, dev, "gate")
        ld_gate = _pitch(gate) if gate.dim() == 2 else 0
    r_out = r.new_empty((m, n)) if r_out is None else _rows(r_out, (m, n), r.dtype, dev, "r_out")
    if want_x and x is None:
        x = r.new_empty((m, n), dtype=torch.bfloat16)
    else:
        x = _next_x(x, want_x, next_weight, "next_weight", r)
    ws = _ws(workspace, lib().q3_ffn_workspace_bytes(gate_up.n, n, m), dev)
    norms = Q3FfnNorms(_ptr(pre_weight), _ptr(post_weight), _ptr(next_weight), _ptr(gate), ld_gate, scale, eps)
    _call("q3_ffn", dev, _matrix(gate_up, dev), _matrix(down, dev), code, ctypes.byref(norms), r.data_ptr(), _pitch(r),
          r_out.data_ptr(), _pitch(r_out), _R_TYPES[r.dtype], _ptr(x), _pitch(x), m, *_ws_args(ws))
    return r_out, x


# ------------------------------------------------------------------ attention sublayer

class PagedCache:
    """A layer's keys and values in pages: bfloat16 [pages][heads][page_size][head_dim],
    contiguous inside a page (the pages may lie apart)."""

    def __init__(self, k: torch.Tensor, v: torch.Tensor):
        if not isinstance(k, torch.Tensor) or not k.is_cuda or k.dim() != 4 or k.dtype != torch.bfloat16:
            raise ValueError("k must be a device tensor bfloat16 [pages][heads][page_size][head_dim]")
        if not isinstance(v, torch.Tensor) or v.device != k.device or v.dtype != k.dtype or v.shape != k.shape:
            raise ValueError("v must be a tensor of k's type, shape and device")
        pages, heads, size, dim = k.shape
        if pages < 1 or heads < 1 or size < 1 or dim < 1:
            raise ValueError(f"a cache of shape {tuple(k.shape)} holds nothing")
        for t, name in ((k, "k"), (v, "v")):
            if not (t.is_contiguous() or t[0].is_contiguous()) or (pages > 1 and t.stride(0) < heads * size * dim):
                raise ValueError(f"{name}'s pages must be contiguous and must not overlap")
        stride = k.stride(0) if pages > 1 else heads * size * dim
        if pages > 1 and v.stride(0) != stride:
            raise ValueError("k's and v's pages must have one pitch")
        self.k, self.v, self.heads, self.page_size, self.head_dim, self.device = k, v, heads, size, dim, k.device
        self._desc = Q3PagedCache(k.data_ptr(), v.data_ptr(), pages, stride, size, heads, dim)

    def desc(self):
        return ctypes.byref(self._desc)


class PagedBatch:
    """New tokens of several sequences: rows q_start[s]..q_start[s + 1] of a call's
    rows are the last of sequence s's kv_len[s] positions (the new ones included),
    whose position p lives in page page_table[s][p // page_size].  int32 device
    tensors [sequences + 1], [sequences] and [sequences][pages]; entries are read
    when a call runs."""

    def __init__(self, q_start: torch.Tensor, kv_len: torch.Tensor, page_table: torch.Tensor):
        if not isinstance(page_table, torch.Tensor) or not page_table.is_cuda or page_table.dim() != 2:
            raise ValueError("page_table must be a device tensor int32 [sequences][pages]")
        (b, pages), dev = page_table.shape, page_table.device
        if b < 1 or pages < 1:
            raise ValueError(f"a page table of shape {tuple(page_table.shape)} names nothing")
        _rows(page_table, (b, pages), torch.int32, dev, "page_table")
        _rows(q_start, (b + 1,), torch.int32, dev, "q_start")
        _rows(kv_len, (b,), torch.int32, dev, "kv_len")
        self.q_start, self.kv_len, self.page_table, self.sequences, self.device = q_start, kv_len, page_table, b, dev
        self._desc = Q3PagedBatch(b, q_start.data_ptr(), kv_len.data_ptr(), page_table.data_ptr(), _pitch(page_table),
                                  pages)

    def desc(self):
        return ctypes.byref(self._desc)


def _on(obj, kind, device, name):
    if not isinstance(obj, kind) or obj.device != device:
        raise ValueError(f"{name} must be a {kind.__name__} on {device} (the inputs' device)")
    return obj.desc()


def _heads_of(qkv, heads_q, heads_kv, inv_freq, q_weight, k_weight, eps, interleaved):
    """The head descriptor of float32 rows [m][(heads_q + 2 heads_kv) head_dim]."""
    if not isinstance(qkv, torch.Tensor) or not qkv.is_cuda or qkv.dim() != 2:
        raise ValueError("qkv must be a device tensor float32 [m][(heads_q + 2 heads_kv) * head_dim]")
    dev, all_heads = qkv.device, heads_q + 2 * heads_kv
    if heads_q < 1 or heads_kv < 1 or qkv.shape[1] % all_heads:
        raise ValueError(f"qkv rows of {qkv.shape[1]} do not hold {heads_q} + 2 * {heads_kv} heads")
    _rows(qkv, qkv.shape, torch.float32, dev, "qkv")
    dim = qkv.shape[1] // all_heads
    _vector(q_weight, dim, torch.float32, dev, "q_weight")
    _vector(k_weight, dim, torch.float32, dev, "k_weight")
    turned = 0
    if inv_freq is not None:
        turned = 2 * inv_freq.numel()
        _rows(inv_freq, (turned // 2,), torch.float32, dev, "inv_freq")
        if turned > dim:
            raise ValueError(f"inv_freq of {turned // 2} turns more than a head of {dim}")
    return dim, Q3HeadNorms(heads_q, heads_kv, dim, turned, bool(interleaved), eps, _ptr(q_weight), _ptr(k_weight),
                            _ptr(inv_freq) if turned else None)


def q3_qk_norm_rope(qkv: torch.Tensor, heads_q: int, heads_kv: int, inv_freq: torch.Tensor = None,
                    positions: torch.Tensor = None, q_weight: torch.Tensor = None, k_weight: torch.Tensor = None,
                    eps: float = 1e-6, interleaved: bool = False, cache: PagedCache = None, batch: PagedBatch = None,
                    q: torch.Tensor = None, k: torch.Tensor = None, v: torch.Tensor = None):
    """The norms of each query and key head (q_weight, k_weight; None: not normed)
    and the rotation of its first 2 len(inv_freq) values by position * inv_freq, in
    pairs (j, j + len(inv_freq)), or adjacent ones with interleaved -> (q, k, v)
    bfloat16 rows.  With cache and batch, k and v go to the new tokens' places in
    the cache instead (and are returned as None); positions (int32 [m]) default to
    the batch's.  Rows that belong to no sequence of the batch are not written.  Not
    recorded by autograd: q3_qk_norm_rope_backward gives the gradients."""
    dim, desc = _heads_of(qkv, heads_q, heads_kv, inv_freq, q_weight, k_weight, eps, interleaved)
    m, dev = qkv.shape[0], qkv.device
    _vector(positions, m, torch.int32, dev, "positions")
    nq, nk = heads_q * dim, heads_kv * dim
    q = torch.empty((m, nq), dtype=torch.bfloat16, device=dev) if q is None else \
        _rows(q, (m, nq), torch.bfloat16, dev, "q")
    paged = (None, None)
    if cache is not None or batch is not None:
        if k is not None or v is not None:
            raise ValueError("k and v go to the cache: no rows for them")
        paged = _on(cache, PagedCache, dev, "cache"), _on(batch, PagedBatch, dev, "batch")
    else:
        if positions is None and desc.rotated:
            raise ValueError("positions are needed where there is no batch")
        k = torch.empty((m, nk), dtype=torch.bfloat16, device=dev) if k is None else \
            _rows(k, (m, nk), torch.bfloat16, dev, "k")
        v = torch.empty((m, nk), dtype=torch.bfloat16, device=dev) if v is None else \
            _rows(v, (m, nk), torch.bfloat16, dev, "v")
    _call("q3_qk_norm_rope", dev, ctypes.byref(desc), qkv.data_ptr(), _pitch(qkv), _ptr(positions), q.data_ptr(),
          _pitch(q), _ptr(k), _pitch(k), _ptr(v), _pitch(v), *paged, m)
    return q, k, v


@dataclass
class QkNormRopeGrads:
    """Gradients of q3_qk_norm_rope's inputs (None where there is no such input)."""
    dqkv: torch.Tensor                       # bfloat16, qkv's shape
    dq_weight: Optional[torch.Tensor] = None   # float32 [head_dim]
    dk_weight: Optional[torch.Tensor] = None


def q3_qk_norm_rope_backward_workspace_bytes(m: int, head_dim: int) -> int:
    return lib().q3_qk_norm_rope_backward_workspace_bytes(m, head_dim)


def q3_qk_norm_rope_backward(qkv: torch.Tensor, heads_q: int, heads_kv: int, inv_freq: torch.Tensor = None,
                             positions: torch.Tensor = None, dq: torch.Tensor = None, dk: torch.Tensor = None,
                             dv: torch.Tensor = None, q_weight: torch.Tensor = None, k_weight: torch.Tensor = None,
                             eps: float = 1e-6, interleaved: bool = False,
                             workspace: torch.Tensor = None) -> QkNormRopeGrads:
    """From the kept qkv rows and the gradients dq, dk, dv (all float32 or all
    bfloat16; each may be None: zero) of q3_qk_norm_rope's rows."""
    dim, desc = _heads_of(qkv, heads_q, heads_kv, inv_freq, q_weight, k_weight, eps, interleaved)
    m, dev = qkv.shape[0], qkv.device
    _vector(positions, m, torch.int32, dev, "positions")
    if positions is None and desc.rotated:
        raise ValueError("positions are needed for the rotation")
    dtype = next((t.dtype for t in (dq, dk, dv) if isinstance(t, torch.Tensor)), torch.bfloat16)
    if dtype not in _R_TYPES:
        raise ValueError("dq, dk and dv must be float32 or bfloat16")
    for t, name, heads in ((dq, "dq", heads_q), (dk, "dk", heads_kv), (dv, "dv", heads_kv)):
        if t is not None:
            _rows(t, (m, heads * dim), dtype, dev, name)
    g = QkNormRopeGrads(torch.empty(qkv.shape, dtype=torch.bfloat16, device=dev))
    if q_weight is not None or k_weight is not None:
        sums = torch.empty((2, dim), dtype=torch.float32, device=dev)
        g.dq_weight = None if q_weight is None else sums[0]
        g.dk_weight = None if k_weight is None else sums[1]
    ws = _ws(workspace, lib().q3_qk_norm_rope_backward_workspace_bytes(m, dim), dev)
    grads = Q3QkvGrads(_R_TYPES[dtype], _ptr(dq), _pitch(dq), _ptr(dk), _pitch(dk), _ptr(dv), _pitch(dv),
                       g.dqkv.data_ptr(), qkv.shape[1], _ptr(g.dq_weight), _ptr(g.dk_weight))
    _call("q3_qk_norm_rope_backward", dev, ctypes.byref(desc), qkv.data_ptr(), _pitch(qkv), _ptr(positions), m,
          ctypes.byref(grads), *_ws_args(ws))
    return g


def q3_paged_attention_workspace_bytes(m: int, sequences: int, heads_q: int, heads: int, head_dim: int) -> int:
    return lib().q3_paged_attention_workspace_bytes(m, sequences, heads_q, heads, head_dim)


def q3_paged_attention(q: torch.Tensor, cache: PagedCache, batch: PagedBatch, scale: float = None, window: int = 0,
                       want_lse: bool = False, out: torch.Tensor = None, lse: torch.Tensor = None,
                       workspace: torch.Tensor = None):
    """Attention of the batch's new tokens (q bfloat16 [m][heads_q * head_dim])
    over the cache, in which their own keys and values stand already: a token sees
    its own position and those before it, with window > 0 the last `window` of
    them.  scale defaults to head_dim ** -0.5.  -> out bfloat16 like q; with
    want_lse (or lse given) -> (out, lse), lse float32 [m][heads_q].  Tokens that see
    nothing get zeros and -inf; rows that belong to no sequence are not written.
    For inference: not recorded by autograd."""
    if not 0 <= window < 1 << 31:   # the C call's 32 bits would take another one
        raise ValueError(f"window must be 0..2^31 - 1, got {window}")
    if not isinstance(q, torch.Tensor) or not q.is_cuda or q.dim() != 2:
        raise ValueError("q must be a device tensor bfloat16 [m][heads_q * head_dim]")
    (m, n), dev = q.shape, q.device
    _rows(q, (m, n), torch.bfloat16, dev, "q")
    paged = _on(cache, PagedCache, dev, "cache"), _on(batch, PagedBatch, dev, "batch")
    heads, rest = divmod(n, cache.head_dim)
    if rest or heads < 1 or heads % cache.heads:
        raise ValueError(f"q rows of {n} do not hold a multiple of the cache's {cache.heads} heads of "
                         f"{cache.head_dim}")
    out = torch.empty((m, n), dtype=torch.bfloat16, device=dev) if out is None else \
        _rows(out, (m, n), torch.bfloat16, dev, "out")
    if lse is not None:
        _rows(lse, (m, heads), torch.float32, dev, "lse")
        if not lse.is_contiguous():
            raise ValueError("lse must be contiguous")
    elif want_lse:
        lse = torch.empty((m, heads), dtype=torch.float32, device=dev)
    ws = _ws(workspace, lib().q3_paged_attention_workspace_bytes(m, batch.sequences, heads, cache.heads,
                                                                 cache.head_dim), dev)
    _call("q3_paged_attention", dev, q.data_ptr(), _pitch(q), heads, *paged,
          cache.head_dim ** -0.5 if scale is None else scale, window, out.data_ptr(), _pitch(out), _ptr(lse), m,
          *_ws_args(ws))
    return out if lse is None else (out, lse)


# ------------------------------------------------------------------ sampling

def sample_workspace(m: int, n: int, device) -> torch.Tensor:
    """Workspace for q3_sample (reusable across calls in stream order)."""
    nbytes = lib().q3_sample_workspace_bytes(m, n)
    if nbytes <= 0:
        raise ValueError("unsupported sampling shape")
    return torch.empty(nbytes, dtype=torch.uint8, device=device)


def q3_sample(logits: torch.Tensor, u: torch.Tensor, temperature: torch.Tensor = None, top_k: torch.Tensor = None,
              top_p: torch.Tensor = None, min_p: torch.Tensor = None, workspace: torch.Tensor = None,
              tokens: torch.Tensor = None, logprobs: torch.Tensor = None):
    """One token per row of float32 logits [m][n] from the random numbers u
    (float32 [m] in [0, 1)) -> (tokens int32 [m], logprobs float32 [m]).  The
    settings are float32 [m] (top_k int32 [m]) or None (off)."""
    if not isinstance(logits, torch.Tensor) or not logits.is_cuda or logits.dim() != 2:
        raise ValueError("logits must be a device tensor float32 [m][n]")
    (m, n), dev = logits.shape, logits.device
    _rows(logits, (m, n), torch.float32, dev, "logits")
    _rows(u, (m,), torch.float32, dev, "u")
    _vector(temperature, m, torch.float32, dev, "temperature")
    _vector(top_k, m, torch.int32, dev, "top_k")
    _vector(top_p, m, torch.float32, dev, "top_p")
    _vector(min_p, m, torch.float32, dev, "min_p")
    tokens = torch.empty(m, dtype=torch.int32, device=dev) if tokens is None else \
        _rows(tokens, (m,), torch.int32, dev, "tokens")
    logprobs = torch.empty(m, dtype=torch.float32, device=dev) if logprobs is None else \
        _rows(logprobs, (m,), torch.float32, dev, "logprobs")
    ws = _ws(workspace, lib().q3_sample_workspace_bytes(m, n), dev)
    _call("q3_sample", dev, logits.data_ptr(), m, n, _pitch(logits), _ptr(temperature), _ptr(top_k), _ptr(top_p),
          _ptr(min_p), u.data_ptr(), *_ws_args(ws), tokens.data_ptr(), logprobs.data_ptr())
    return tokens, logprobs


# ------------------------------------------------------------------ log probabilities

@dataclass
class Logprobs:
    """q3_logprobs' answers for each row."""
    logprobs: torch.Tensor                       # float32 [m]
    entropy: torch.Tensor                        # float32 [m]
    stats: torch.Tensor                          # float32 [m][4], for q3_logprobs_backward
    top_ids: Optional[torch.Tensor] = None       # int32 [m][top]
    top_logprobs: Optional[torch.Tensor] = None   # float32 [m][top]


def q3_logprobs_workspace_bytes(m: int, n: int, top: int = 0) -> int:
    return lib().q3_logprobs_workspace_bytes(m, n, top)


def _logits_of(logits):
    if not isinstance(logits, torch.Tensor) or not logits.is_cuda or logits.dim() != 2:
        raise ValueError("logits must be a device tensor float32 [m][n]")
    return _rows(logits, logits.shape, torch.float32, logits.device, "logits")


def q3_logprobs(logits: torch.Tensor, targets: torch.Tensor, temperature: float = 1.0, top: int = 0,
                workspace: torch.Tensor = None) -> Logprobs:
    """Log probabilities of the tokens `targets` (int32 [m]; outside [0, n): none, 0)
    under float32 logits [m][n] / temperature, the rows' entropy and their `top`
    (up to 32) largest entries.  Not recorded by autograd: q3_logprobs_backward gives
    the gradient."""
    _logits_of(logits)
    (m, n), dev = logits.shape, logits.device
    _rows(targets, (m,), torch.int32, dev, "targets")
    if not 0 <= top <= 32:
        raise ValueError(f"top must be 0..32, got {top}")
    rows = torch.empty((2, m), dtype=torch.float32, device=dev).unbind(0)
    r = Logprobs(rows[0], rows[1], torch.empty((m, 4), dtype=torch.float32, device=dev))
    if top:
        r.top_ids = torch.empty((m, top), dtype=torch.int32, device=dev)
        r.top_logprobs = torch.empty((m, top), dtype=torch.float32, device=dev)
    ws = _ws(workspace, lib().q3_logprobs_workspace_bytes(m, n, top), dev)
    _call("q3_logprobs", dev, logits.data_ptr(), m, n, _pitch(logits), targets.data_ptr(), temperature, top,
          r.logprobs.data_ptr(), r.entropy.data_ptr(), _ptr(r.top_ids), _ptr(r.top_logprobs), r.stats.data_ptr(),
          *_ws_args(ws))
    return r


def q3_logprobs_backward(logits: torch.Tensor, targets: torch.Tensor, stats: torch.Tensor,
                         dlogprobs: torch.Tensor = None, dentropy: torch.Tensor = None, temperature: float = 1.0,
                         dtype: torch.dtype = torch.bfloat16, dlogits: torch.Tensor = None) -> torch.Tensor:
    """The gradient of the logits from q3_logprobs' stats and the gradients dlogprobs
    and dentropy (float32 [m]; either may be None: zero): dtype bfloat16, rows
    pitched so that q3_gemm_backward takes them, or float32 (dlogits may then be
    the logits)."""
    _logits_of(logits)
    (m, n), dev = logits.shape, logits.device
    _rows(targets, (m,), torch.int32, dev, "targets")
    _rows(stats, (m, 4), torch.float32, dev, "stats")
    if not stats.is_contiguous():
        raise ValueError("stats must be contiguous")
    _vector(dlogprobs, m, torch.float32, dev, "dlogprobs")
    _vector(dentropy, m, torch.float32, dev, "dentropy")
    if dlogits is None:
        if dtype not in _R_TYPES:
            raise ValueError(f"dtype must be bfloat16 or float32, got {dtype}")
        wide = (n + 7) // 8 * 8
        dlogits = torch.empty((m, wide), dtype=dtype, device=dev)
        dlogits = dlogits if wide == n else dlogits[:, :n]
    else:
        if dlogits.dtype not in _R_TYPES:
            raise ValueError(f"dlogits must be bfloat16 or float32, got {dlogits.dtype}")
        _rows(dlogits, (m, n), dlogits.dtype, dev, "dlogits")
    _call("q3_logprobs_backward", dev, logits.data_ptr(), m, n, _pitch(logits), targets.data_ptr(), temperature,
          stats.data_ptr(), _ptr(dlogprobs), _ptr(dentropy), dlogits.data_ptr(), _pitch(dlogits),
          _R_TYPES[dlogits.dtype])
    return dlogits
