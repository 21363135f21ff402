"""ctypes binding of include/q3_block.h: argument marshalling only.

The operators between two packed products and behind the last one: products of
many tokens, the gated feed-forward block, residual norms (each with the
gradients of its inputs) and sampling.  Every function forwards to the C entry
point of the same name; outputs and workspaces that are not given are allocated
here.  A call runs on the current stream of its tensors' device.

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


_int = ctypes.c_int
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
