"""ctypes binding of the operators around the scan (C ABI in include/mssm_block.h).

As binding.py: argument marshalling only, on the current HIP stream of the
tensors' device (the library launches on the current device, which is switched
for the call where it is another one).  These
are operators of serving: they have no backward, and what they return from
tensors that require gradients does not.  A
decode step makes these calls once a layer, with kernels of a few microseconds,
so the marshalling is kept short: problem descriptors and workspace sizes are
remembered by the sizes they follow from.
"""
from __future__ import annotations

import ctypes
import operator
from functools import lru_cache

import torch

from .binding import MSSM_BF16, MSSM_F32, MssmError, _dtype_code, _workspace, lib
from . import binding

MSSM_F8 = 2
_CODES = {torch.float32: MSSM_F32, torch.bfloat16: MSSM_BF16, torch.float8_e4m3fn: MSSM_F8}
MAX_BEAMS = 16
MAX_BEAM_STATES = 16
MAX_RANK = 128
ACTIVATIONS = {None: 0, "none": 0, "relu": 1, "silu": 2, "gelu": 3}
BLOCK_EXPORTS = ["mssm_add_rmsnorm", "mssm_add_rmsnorm_q8", "mssm_linear_workspace_bytes", "mssm_linear",
                 "mssm_lora_workspace_bytes", "mssm_lora", "mssm_beam_select_workspace_bytes", "mssm_beam_select",
                 "mssm_beam_reorder"]


class NormProblem(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("dim", ctypes.c_int64), ("dtype", ctypes.c_int32),
                ("residual_dtype", ctypes.c_int32), ("eps", ctypes.c_float)]


class LinearProblem(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("in_dim", ctypes.c_int64), ("out_dim", ctypes.c_int64),
                ("dtype", ctypes.c_int32), ("out_dtype", ctypes.c_int32), ("activation", ctypes.c_int32)]


class LoraProblem(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("in_dim", ctypes.c_int64), ("out_dim", ctypes.c_int64),
                ("rank", ctypes.c_int64), ("adapters", ctypes.c_int64), ("dtype", ctypes.c_int32),
                ("out_dtype", ctypes.c_int32)]


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
            ("mssm_lora_workspace_bytes", [ctypes.POINTER(LoraProblem)], sz),
            ("mssm_lora", [ctypes.POINTER(LoraProblem)] + [vp] * 7 + [vp, sz, vp], st),
            ("mssm_beam_select_workspace_bytes", [BP], sz),
            ("mssm_beam_select", [BP] + [vp] * 7 + [vp, sz, vp], st),
            ("mssm_beam_reorder", [i64, i64, vp, ctypes.c_int32, ctypes.POINTER(BeamState), vp], st)):
        getattr(lib, name).argtypes = args
        getattr(lib, name).restype = res


_declare()


def _req(t, name, shape, dtype, dev):
    """binding._req, which says what is wrong, for a tensor that is not right at first sight; dev: the index of
    the GPU that the call's first tensor is on."""
    if t is None or not (t.get_device() == dev and t.dtype == dtype and t.shape == shape and t.is_contiguous()):
        binding._req(t, name, shape, dtype)
        raise ValueError(f"{name} is on device {t.get_device()}, the call's other tensors on {dev}")


def _opt(t, name, shape, dtype, dev):
    if t is not None:
        _req(t, name, shape, dtype, dev)


def _ptr(t):
    return None if t is None else t.data_ptr()


# The current stream's handle by the call that torch's own code generators use; the public one builds an object each time.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (lambda i: torch.cuda.current_stream(i).cuda_stream)


def _new(shape, dtype, device):
    """torch.empty of a contiguous tensor; with its strides given, torch takes half the time for few dimensions."""
    if len(shape) == 1:
        return torch.empty_strided(shape, (1,), dtype=dtype, device=device)
    if len(shape) == 2:
        return torch.empty_strided(shape, (shape[1], 1), dtype=dtype, device=device)
    return torch.empty(shape, dtype=dtype, device=device)


_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _run(status: int):
    if status != 0:
        raise MssmError(status, lib)


@lru_cache(maxsize=1024)
def _norm_problem(rows, dim, code, rcode, eps):
    p = NormProblem(rows, dim, code, rcode, eps)
    return ctypes.byref(p), p


@lru_cache(maxsize=1024)
def _linear_problem(rows, k, n, code, ocode, act, device):
    p = LinearProblem(rows, k, n, code, ocode, act)
    with torch.cuda.device(device):
        return ctypes.byref(p), int(lib.mssm_linear_workspace_bytes(ctypes.byref(p))), p


@lru_cache(maxsize=1024)
def _lora_problem(rows, k, n, rank, adapters, code, ocode):
    p = LoraProblem(rows, k, n, rank, adapters, code, ocode)
    return ctypes.byref(p), int(lib.mssm_lora_workspace_bytes(ctypes.byref(p))), p


@lru_cache(maxsize=1024)
def _beam_problem(batch, beams, vocab, code, end):
    p = BeamProblem(batch, beams, vocab, code, end)
    return ctypes.byref(p), int(lib.mssm_beam_select_workspace_bytes(ctypes.byref(p))), p


def _norm_args(x, weight, residual, residual_out, eps):
    shape = () if x is None else x.shape
    if not shape:
        raise ValueError("x must have at least one dimension")
    D = shape[-1]
    code = _dtype_code(x)
    dev = x.get_device()
    if dev < 0:
        raise ValueError("x must be a GPU tensor")
    if not x.is_contiguous():
        raise ValueError("x must be contiguous")
    _req(weight, "weight", (D,), torch.float32, dev)
    kept = residual if residual is not None else residual_out
    rcode = _dtype_code(kept) if kept is not None else code
    if residual is not None:
        _req(residual, "residual", shape, residual.dtype, dev)
    if residual_out is not None:
        _req(residual_out, "residual_out", shape, kept.dtype, dev)
    elif residual is not None:
        residual_out = torch.empty_like(residual)
    if not eps >= 0.0:
        raise ValueError(f"eps = {eps} must not be negative")
    return _norm_problem(x.numel() // D if D else 0, D, code, rcode, float(eps))[0], residual_out, dev  # by its value


def add_rmsnorm(x, weight, residual=None, eps=1e-5, y=None, residual_out=None):
    """Residual addition and root-mean-square norm of the last dimension:
    h = x + residual, y = h / sqrt(mean(h^2) + eps) * weight.  x (..., D)
    float32 or bfloat16, residual as x in either type, weight (D) float32.
    Returns (y, residual_out): y in x's type, residual_out = h in the
    residual's (None without a residual, unless given).  residual_out may be
    residual and y may be x.  Forward only: no gradient is recorded."""
    prob, residual_out, dev = _norm_args(x, weight, residual, residual_out, eps)
    if y is None:
        y = torch.empty_like(x)
    else:
        _req(y, "y", x.shape, x.dtype, dev)
    if _current_device() != dev:
        with torch.cuda.device(dev):
            return add_rmsnorm(x, weight, residual, eps, y, residual_out)
    _run(lib.mssm_add_rmsnorm(prob, x.data_ptr(), _ptr(residual), weight.data_ptr(), y.data_ptr(), _ptr(residual_out),
                              _raw_stream(dev)))
    return y, residual_out


def add_rmsnorm_q8(x, weight, residual=None, eps=1e-5, q=None, scale=None, residual_out=None):
    """add_rmsnorm with y in 8 bits: q (..., D) float8_e4m3fn and scale (...)
    float32 with y ~ q * scale, scale = max(max|y|, 1e-30) / 448 of each row.
    Returns (q, scale, residual_out); linear() takes q and scale as x and
    x_scale.  Forward only: no gradient is recorded."""
    prob, residual_out, dev = _norm_args(x, weight, residual, residual_out, eps)
    if q is None:
        q = torch.empty_like(x, dtype=torch.float8_e4m3fn)
    else:
        _req(q, "q", x.shape, torch.float8_e4m3fn, dev)
    if scale is None:
        scale = _new(x.shape[:-1], torch.float32, x.device)
    else:
        _req(scale, "scale", x.shape[:-1], torch.float32, dev)
    if _current_device() != dev:
        with torch.cuda.device(dev):
            return add_rmsnorm_q8(x, weight, residual, eps, q, scale, residual_out)
    _run(lib.mssm_add_rmsnorm_q8(prob, x.data_ptr(), _ptr(residual), weight.data_ptr(), q.data_ptr(), scale.data_ptr(),
                                 _ptr(residual_out), _raw_stream(dev)))
    return q, scale, residual_out


def linear(x, w, bias=None, residual=None, activation=None, x_scale=None, w_scale=None, out_dtype=None, y=None,
           workspace=None):
    """Projection with its epilogue: y = act(x wᵀ + bias) + residual, rounded
    once.  x (..., K) and w (N, K) both float32, both bfloat16 or both
    float8_e4m3fn; 8-bit operands come with x_scale (...) and w_scale (N)
    float32, one scale a row.  bias (N) float32; activation None, "relu",
    "silu" or "gelu" (by erf); residual (..., N) in the output's type.
    out_dtype: float32, or bfloat16 (not with float32 operands); x's type by
    default, bfloat16 with 8-bit operands.  8-bit operands with a bfloat16
    output are summed by the 8-bit matrix instructions, within 2^-10 sum |x w|
    (typically 1.5e-5 of the sum); out_dtype=float32 sums them in float32 at
    half the rate, for sums that cancel.  y may be residual.  Forward only:
    no gradient is recorded."""
    if x is None or w is None or x.dim() < 1 or w.dim() != 2:
        raise ValueError("x must be (..., K) and w (N, K)")
    act = x.dtype
    if act not in _CODES:
        raise TypeError(f"x must be float32, bfloat16 or float8_e4m3fn, got {x.dtype}")
    if activation not in ACTIVATIONS:
        raise ValueError(f"activation {activation!r} is not one of {sorted(k for k in ACTIVATIONS if k)}")
    shape, N = x.shape, w.shape[0]
    lead, K = shape[:-1], shape[-1]
    dev = x.get_device()
    if dev < 0:
        raise ValueError("x must be a GPU tensor")
    if not x.is_contiguous():
        raise ValueError("x must be contiguous")
    _req(w, "w", (N, K), act, dev)
    if out_dtype is None:
        out_dtype = torch.bfloat16 if act == torch.float8_e4m3fn else act
    if out_dtype not in (torch.float32, torch.bfloat16) or (act == torch.float32 and out_dtype != torch.float32):
        raise TypeError(f"out_dtype {out_dtype} is not available for {act} operands")
    if act == torch.float8_e4m3fn:
        _req(x_scale, "x_scale", lead, torch.float32, dev)
        _req(w_scale, "w_scale", (N,), torch.float32, dev)
    elif x_scale is not None or w_scale is not None:
        raise ValueError("x_scale and w_scale belong to 8-bit operands")
    _opt(bias, "bias", (N,), torch.float32, dev)
    _opt(residual, "residual", (*lead, N), out_dtype, dev)
    if y is None:
        y = _new((*lead, N), out_dtype, x.device)
    else:
        _req(y, "y", (*lead, N), out_dtype, dev)
    prob, nbytes, _ = _linear_problem(x.numel() // K if K else 0, K, N, _CODES[act], _CODES[out_dtype],
                                      ACTIVATIONS[activation], dev)
    ws = _workspace(nbytes, x.device, workspace)
    if _current_device() != dev:
        with torch.cuda.device(dev):
            return linear(x, w, bias, residual, activation, x_scale, w_scale, out_dtype, y, ws)
    _run(lib.mssm_linear(prob, x.data_ptr(), _ptr(x_scale), w.data_ptr(), _ptr(w_scale), _ptr(bias), _ptr(residual),
                         y.data_ptr(), _ptr(ws), nbytes, _raw_stream(dev)))
    return y


def lora(x, a, b, index, y, scale=None, x_scale=None, workspace=None):
    """Low-rank adapters beside a shared projection, in place:
    y[m] += scale[i] (x[m] a[i]ᵀ) b[i]ᵀ with i = index[m], rounded once.
    x (..., K) float32, bfloat16 or float8_e4m3fn with x_scale (...) float32, one
    scale a row; a (S, R, K) and b (S, N, R) float32 with float32 x, else
    bfloat16; index (...) int32 in any order (a row whose index is not in
    0 .. S - 1 stays as it is); y (..., N) float32, or bfloat16 (not with float32
    x), as linear() returns it; scale (S) float32.  Returns y.  Forward only: no
    gradient is recorded."""
    if x is None or x.dim() < 1 or a is None or a.dim() != 3 or y is None or y.dim() < 1:
        raise ValueError("x must be (..., K), a (S, R, K) and y (..., N)")
    act = x.dtype
    if act not in _CODES:
        raise TypeError(f"x must be float32, bfloat16 or float8_e4m3fn, got {x.dtype}")
    lead, K, N = x.shape[:-1], x.shape[-1], y.shape[-1]
    S, R = a.shape[:2]
    dev = x.get_device()
    if dev < 0:
        raise ValueError("x must be a GPU tensor")
    if not x.is_contiguous():
        raise ValueError("x must be contiguous")
    if R > MAX_RANK:
        raise ValueError(f"rank {R}: at most {MAX_RANK}")
    weights = torch.float32 if act == torch.float32 else torch.bfloat16
    _req(a, "a", (S, R, K), weights, dev)
    _req(b, "b", (S, N, R), weights, dev)
    _req(index, "index", lead, torch.int32, dev)
    if y.dtype not in (torch.float32, torch.bfloat16) or (act == torch.float32 and y.dtype != torch.float32):
        raise TypeError(f"y of {y.dtype} is not available for {act} x")
    _req(y, "y", (*lead, N), y.dtype, dev)
    _opt(scale, "scale", (S,), torch.float32, dev)
    if act == torch.float8_e4m3fn:
        _req(x_scale, "x_scale", lead, torch.float32, dev)
    elif x_scale is not None:
        raise ValueError("x_scale belongs to 8-bit rows")
    prob, nbytes, _ = _lora_problem(x.numel() // K if K else 0, K, N, R, S, _CODES[act], _CODES[y.dtype])
    ws = _workspace(nbytes, x.device, workspace)
    if _current_device() != dev:
        with torch.cuda.device(dev):
            return lora(x, a, b, index, y, scale, x_scale, ws)
    _run(lib.mssm_lora(prob, x.data_ptr(), _ptr(x_scale), a.data_ptr(), b.data_ptr(), _ptr(scale), index.data_ptr(),
                       y.data_ptr(), _ptr(ws), nbytes, _raw_stream(dev)))
    return y


def beam_select(logits, scores, finished=None, end_token=None, scores_out=None, parent=None, token=None,
                finished_out=None, workspace=None):
    """One selection of beam search.  logits (B, K, V) float32 or bfloat16,
    scores (B, K) float32 (-inf: a beam not in use), finished (B, K) bool with
    end_token.  Of the K * V continuations scores + log_softmax(logits) of
    every batch row the K best, in descending order, ties to the lowest
    k * V + v.  Returns (scores_out, parent, token, finished_out): parent and
    token (B, K) int32; finished_out (B, K) bool, None without an end_token.
    Forward only: no gradient is recorded."""
    if logits is None or logits.dim() != 3:
        raise ValueError("logits must be (B, K, V)")
    B, K, V = logits.shape
    dev = logits.get_device()
    if dev < 0:
        raise ValueError("logits must be a GPU tensor")
    if not logits.is_contiguous():
        raise ValueError("logits must be contiguous")
    code = _dtype_code(logits)
    if K > MAX_BEAMS:
        raise ValueError(f"{K} beams: at most {MAX_BEAMS}")
    _req(scores, "scores", (B, K), torch.float32, dev)
    _opt(finished, "finished", (B, K), torch.bool, dev)
    if end_token is None:
        if finished is not None or finished_out is not None:
            raise ValueError("finished beams need an end_token")
    else:
        if not 0 <= end_token < V:
            raise ValueError(f"end_token {end_token} is not in 0..{V - 1}")
        if finished_out is None:
            finished_out = _new((B, K), torch.bool, logits.device)
    _opt(finished_out, "finished_out", (B, K), torch.bool, dev)
    if scores_out is None:
        scores_out = torch.empty_like(scores)
    else:
        _req(scores_out, "scores_out", (B, K), torch.float32, dev)
    if parent is None:
        parent = torch.empty_like(scores, dtype=torch.int32)
    else:
        _req(parent, "parent", (B, K), torch.int32, dev)
    if token is None:
        token = torch.empty_like(parent)
    else:
        _req(token, "token", (B, K), torch.int32, dev)
    prob, nbytes, _ = _beam_problem(B, K, V, code, -1 if end_token is None else operator.index(end_token))
    ws = _workspace(nbytes, logits.device, workspace)
    if _current_device() != dev:
        with torch.cuda.device(dev):
            return beam_select(logits, scores, finished, end_token, scores_out, parent, token, finished_out, ws)
    _run(lib.mssm_beam_select(prob, logits.data_ptr(), scores.data_ptr(), _ptr(finished), scores_out.data_ptr(),
                              parent.data_ptr(), token.data_ptr(), _ptr(finished_out), _ptr(ws), nbytes, _raw_stream(dev)))
    return scores_out, parent, token, finished_out


def beam_reorder(parent, states):
    """The beams' states follow their parents, in place: for every tensor of
    states, (layers, B * K, ...) of any type, t[l, b * K + k] becomes
    t[l, b * K + parent[b, k]].  parent (B, K) int32, as beam_select returns
    it.  One state (B * K, ...) goes as state[None].  Returns states.  Forward
    only: no gradient is recorded."""
    if parent is None or parent.dim() != 2:
        raise ValueError("parent must be (B, K)")
    B, K = parent.shape
    dev = parent.get_device()
    if dev < 0:
        raise ValueError("parent must be a GPU tensor")
    _req(parent, "parent", (B, K), torch.int32, dev)
    if K > MAX_BEAMS:
        raise ValueError(f"{K} beams: at most {MAX_BEAMS}")
    each = [states] if isinstance(states, torch.Tensor) else list(states)
    if not 1 <= len(each) <= MAX_BEAM_STATES:
        raise ValueError(f"{len(each)} states: 1 to {MAX_BEAM_STATES} a call")
    entries = (BeamState * len(each))()
    for i, t in enumerate(each):
        if t is None or t.dim() < 2 or t.shape[1] != B * K:
            raise ValueError(f"states[{i}] must be (layers, {B * K}, ...)")
        if t.get_device() != dev or not t.is_contiguous():
            _req(t, f"states[{i}]", t.shape, t.dtype, dev)
        if t.numel() == 0:
            raise MssmError(-2, lib)
        e = entries[i]
        e.data, e.layers, e.bytes = t.data_ptr(), t.shape[0], t.numel() // (t.shape[0] * B * K) * t.element_size()
    if _current_device() != dev:
        with torch.cuda.device(dev):
            beam_reorder(parent, each)
        return states
    _run(lib.mssm_beam_reorder(B, K, parent.data_ptr(), len(each), entries, _raw_stream(dev)))
    return states
