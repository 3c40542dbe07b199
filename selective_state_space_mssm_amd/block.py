"""ctypes binding of the operators around the scan (C ABI in include/mssm_block.h).

As binding.py: argument marshalling only, on torch's current HIP stream.
"""
from __future__ import annotations

import ctypes

import torch

from .binding import MSSM_BF16, MSSM_F32, MssmError, _check, _dtype_code, _opt, _ptr, _req, _stream, _workspace, lib

MSSM_F8 = 2
MAX_BEAMS = 16
MAX_BEAM_STATES = 16
ACTIVATIONS = {None: 0, "none": 0, "relu": 1, "silu": 2, "gelu": 3}
BLOCK_EXPORTS = ["mssm_add_rmsnorm", "mssm_add_rmsnorm_q8", "mssm_linear_workspace_bytes", "mssm_linear",
                 "mssm_beam_select_workspace_bytes", "mssm_beam_select", "mssm_beam_reorder"]


class NormProblem(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("dim", ctypes.c_int64), ("dtype", ctypes.c_int32),
                ("residual_dtype", ctypes.c_int32), ("eps", ctypes.c_float)]


class LinearProblem(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("in_dim", ctypes.c_int64), ("out_dim", ctypes.c_int64),
                ("dtype", ctypes.c_int32), ("out_dtype", ctypes.c_int32), ("activation", ctypes.c_int32)]


class BeamProblem(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int64), ("beams", ctypes.c_int64), ("vocab", ctypes.c_int64),
                ("dtype", ctypes.c_int32), ("end_token", ctypes.c_int32)]


class BeamState(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("layers", ctypes.c_int64), ("bytes", ctypes.c_int64)]


def _declare():
    sz, st, vp, i64 = ctypes.c_size_t, ctypes.c_int, ctypes.c_void_p, ctypes.c_int64
    NP, LP, BP = ctypes.POINTER(NormProblem), ctypes.POINTER(LinearProblem), ctypes.POINTER(BeamProblem)
    for name, args, res in (
            ("mssm_add_rmsnorm", [NP] + [vp] * 6, st),
            ("mssm_add_rmsnorm_q8", [NP] + [vp] * 7, st),
            ("mssm_linear_workspace_bytes", [LP], sz),
            ("mssm_linear", [LP] + [vp] * 7 + [vp, sz, vp], st),
            ("mssm_beam_select_workspace_bytes", [BP], sz),
            ("mssm_beam_select", [BP] + [vp] * 7 + [vp, sz, vp], st),
            ("mssm_beam_reorder", [i64, i64, vp, ctypes.c_int32, ctypes.POINTER(BeamState), vp], st)):
        getattr(lib, name).argtypes = args
        getattr(lib, name).restype = res


_declare()


def _norm_args(x, weight, residual, residual_out, eps):
    if x is None or x.dim() < 1:
        raise ValueError("x must have at least one dimension")
    D = x.shape[-1]
    _req(x, "x", x.shape, x.dtype)
    code = _dtype_code(x)
    _req(weight, "weight", (D,), torch.float32)
    kept = residual if residual is not None else residual_out
    rcode = _dtype_code(kept) if kept is not None else code
    if residual is not None:
        _req(residual, "residual", x.shape, residual.dtype)
        if residual_out is None:
            residual_out = torch.empty_like(residual)
    if residual_out is not None:
        _req(residual_out, "residual_out", x.shape, kept.dtype)
    if not eps >= 0.0:
        raise ValueError(f"eps = {eps} must not be negative")
    return NormProblem(x.numel() // D if D else 0, D, code, rcode, eps), residual_out


def add_rmsnorm(x, weight, residual=None, eps=1e-5, y=None, residual_out=None):
    """Residual addition and root-mean-square norm of the last dimension:
    h = x + residual, y = h / sqrt(mean(h^2) + eps) * weight.  x (..., D)
    float32 or bfloat16, residual as x in either type, weight (D) float32.
    Returns (y, residual_out): y in x's type, residual_out = h in the
    residual's (None without a residual, unless given).  residual_out may be
    residual and y may be x."""
    prob, residual_out = _norm_args(x, weight, residual, residual_out, eps)
    if y is None:
        y = torch.empty_like(x)
    _req(y, "y", x.shape, x.dtype)
    _check(lib.mssm_add_rmsnorm(ctypes.byref(prob), _ptr(x), _ptr(residual), _ptr(weight), _ptr(y),
                                _ptr(residual_out), _stream(x.device)))
    return y, residual_out


def add_rmsnorm_q8(x, weight, residual=None, eps=1e-5, q=None, scale=None, residual_out=None):
    """add_rmsnorm with y in 8 bits: q (..., D) float8_e4m3fn and scale (...)
    float32 with y ~ q * scale, scale = max(max|y|, 1e-30) / 448 of each row.
    Returns (q, scale, residual_out); linear() takes q and scale as x and
    x_scale."""
    prob, residual_out = _norm_args(x, weight, residual, residual_out, eps)
    if q is None:
        q = torch.empty(x.shape, dtype=torch.float8_e4m3fn, device=x.device)
    _req(q, "q", x.shape, torch.float8_e4m3fn)
    if scale is None:
        scale = torch.empty(x.shape[:-1], dtype=torch.float32, device=x.device)
    _req(scale, "scale", x.shape[:-1], torch.float32)
    _check(lib.mssm_add_rmsnorm_q8(ctypes.byref(prob), _ptr(x), _ptr(residual), _ptr(weight), _ptr(q), _ptr(scale),
                                   _ptr(residual_out), _stream(x.device)))
    return q, scale, residual_out


def linear(x, w, bias=None, residual=None, activation=None, x_scale=None, w_scale=None, out_dtype=None, y=None,
           workspace=None):
    """Projection with its epilogue: y = act(x wᵀ + bias) + residual, rounded
    once.  x (..., K) and w (N, K) both float32, both bfloat16 or both
    float8_e4m3fn; 8-bit operands come with x_scale (...) and w_scale (N)
    float32, one scale a row.  bias (N) float32; activation None, "relu",
    "silu" or "gelu" (by erf); residual (..., N) in the output's type.
    out_dtype: float32, or bfloat16 (not with float32 operands); x's type by
    default, bfloat16 with 8-bit operands.  y may be residual."""
    codes = {torch.float32: MSSM_F32, torch.bfloat16: MSSM_BF16, torch.float8_e4m3fn: MSSM_F8}
    if x is None or w is None or x.dim() < 1 or w.dim() != 2:
        raise ValueError("x must be (..., K) and w (N, K)")
    if x.dtype not in codes:
        raise TypeError(f"x must be float32, bfloat16 or float8_e4m3fn, got {x.dtype}")
    if activation not in ACTIVATIONS:
        raise ValueError(f"activation {activation!r} is not one of {sorted(k for k in ACTIVATIONS if k)}")
    lead, K, N = x.shape[:-1], x.shape[-1], w.shape[0]
    _req(x, "x", x.shape, x.dtype)
    _req(w, "w", (N, K), x.dtype)
    if out_dtype is None:
        out_dtype = torch.bfloat16 if x.dtype == torch.float8_e4m3fn else x.dtype
    if out_dtype not in (torch.float32, torch.bfloat16) or (x.dtype == torch.float32 and out_dtype != torch.float32):
        raise TypeError(f"out_dtype {out_dtype} is not available for {x.dtype} operands")
    if x.dtype == torch.float8_e4m3fn:
        _req(x_scale, "x_scale", lead, torch.float32)
        _req(w_scale, "w_scale", (N,), torch.float32)
    elif x_scale is not None or w_scale is not None:
        raise ValueError("x_scale and w_scale belong to 8-bit operands")
    _opt(bias, "bias", (N,), torch.float32)
    _opt(residual, "residual", (*lead, N), out_dtype)
    if y is None:
        y = torch.empty((*lead, N), dtype=out_dtype, device=x.device)
    _req(y, "y", (*lead, N), out_dtype)
    prob = LinearProblem(x.numel() // K if K else 0, K, N, codes[x.dtype], MSSM_F32 if out_dtype == torch.float32 else MSSM_BF16,
                         ACTIVATIONS[activation])
    nbytes = int(lib.mssm_linear_workspace_bytes(ctypes.byref(prob)))
    ws = _workspace(nbytes, x.device, workspace)
    _check(lib.mssm_linear(ctypes.byref(prob), _ptr(x), _ptr(x_scale), _ptr(w), _ptr(w_scale), _ptr(bias),
                           _ptr(residual), _ptr(y), _ptr(ws), nbytes, _stream(x.device)))
    return y


def beam_select(logits, scores, finished=None, end_token=None, scores_out=None, parent=None, token=None,
                finished_out=None, workspace=None):
    """One selection of beam search.  logits (B, K, V) float32 or bfloat16,
    scores (B, K) float32 (-inf: a beam not in use), finished (B, K) bool with
    end_token.  Of the K * V continuations scores + log_softmax(logits) of
    every batch row the K best, in descending order, ties to the lowest
    k * V + v.  Returns (scores_out, parent, token, finished_out): parent and
    token (B, K) int32; finished_out (B, K) bool, None without an end_token."""
    if logits is None or logits.dim() != 3:
        raise ValueError("logits must be (B, K, V)")
    B, K, V = logits.shape
    _req(logits, "logits", (B, K, V), logits.dtype)
    code = _dtype_code(logits)
    if K > MAX_BEAMS:
        raise ValueError(f"{K} beams: at most {MAX_BEAMS}")
    _req(scores, "scores", (B, K), torch.float32)
    _opt(finished, "finished", (B, K), torch.bool)
    if end_token is None:
        if finished is not None or finished_out is not None:
            raise ValueError("finished beams need an end_token")
    else:
        if not 0 <= end_token < V:
            raise ValueError(f"end_token {end_token} is not in 0..{V - 1}")
        if finished_out is None:
            finished_out = torch.empty((B, K), dtype=torch.bool, device=logits.device)
    _opt(finished_out, "finished_out", (B, K), torch.bool)
    if scores_out is None:
        scores_out = torch.empty((B, K), dtype=torch.float32, device=logits.device)
    _req(scores_out, "scores_out", (B, K), torch.float32)
    if parent is None:
        parent = torch.empty((B, K), dtype=torch.int32, device=logits.device)
    _req(parent, "parent", (B, K), torch.int32)
    if token is None:
        token = torch.empty((B, K), dtype=torch.int32, device=logits.device)
    _req(token, "token", (B, K), torch.int32)
    prob = BeamProblem(B, K, V, code, -1 if end_token is None else end_token)
    nbytes = int(lib.mssm_beam_select_workspace_bytes(ctypes.byref(prob)))
    ws = _workspace(nbytes, logits.device, workspace)
    _check(lib.mssm_beam_select(ctypes.byref(prob), _ptr(logits), _ptr(scores), _ptr(finished), _ptr(scores_out),
                                _ptr(parent), _ptr(token), _ptr(finished_out), _ptr(ws), nbytes,
                                _stream(logits.device)))
    return scores_out, parent, token, finished_out


def beam_reorder(parent, states):
    """The beams' states follow their parents, in place: for every tensor of
    states, (layers, B * K, ...) of any type, t[l, b * K + k] becomes
    t[l, b * K + parent[b, k]].  parent (B, K) int32, as beam_select returns
    it.  One state (B * K, ...) goes as state[None].  Returns states."""
    if parent is None or parent.dim() != 2:
        raise ValueError("parent must be (B, K)")
    B, K = parent.shape
    _req(parent, "parent", (B, K), torch.int32)
    if K > MAX_BEAMS:
        raise ValueError(f"{K} beams: at most {MAX_BEAMS}")
    each = [states] if isinstance(states, torch.Tensor) else list(states)
    if not 1 <= len(each) <= MAX_BEAM_STATES:
        raise ValueError(f"{len(each)} states: 1 to {MAX_BEAM_STATES} a call")
    entries = (BeamState * len(each))()
    for i, t in enumerate(each):
        if t is None or t.dim() < 2 or t.shape[1] != B * K:
            raise ValueError(f"states[{i}] must be (layers, {B * K}, ...)")
        _req(t, f"states[{i}]", t.shape, t.dtype)
        if t.numel() == 0:
            raise MssmError(-2, lib)
        entries[i] = BeamState(t.data_ptr(), t.shape[0], t[0, 0].numel() * t.element_size())
    _check(lib.mssm_beam_reorder(B, K, _ptr(parent), len(each), entries, _stream(parent.device)))
    return states
