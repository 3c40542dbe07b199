"""ctypes binding of the gated delta rule (C ABI in include/mssm_gdr.h).

As binding.py: argument marshalling only, on the current HIP stream of the
tensors' device (the library launches on the current device, which is switched
for the call where it is another one).  Problem descriptors and workspace sizes
are remembered by the sizes they follow from.
"""
from __future__ import annotations

import ctypes
from functools import lru_cache

import torch

from . import block
from .binding import _dtype_code, _workspace, lib
from .block import _opt, _ptr, _raw_stream, _req, _run

GDR_MAX_KEY_DIM, GDR_MAX_VALUE_DIM = 128, 512
GDR_EXPORTS = ["mssm_gdr_fwd_workspace_bytes", "mssm_gdr_fwd", "mssm_gdr_ctx_bytes", "mssm_gdr_fwd_train",
               "mssm_gdr_bwd_saved_workspace_bytes", "mssm_gdr_bwd_saved", "mssm_gdr_bwd_workspace_bytes", "mssm_gdr_bwd",
               "mssm_gdr_step"]


class GdrProblem(ctypes.Structure):
    _fields_ = [("tokens", ctypes.c_int64), ("seqs", ctypes.c_int64), ("qk_heads", ctypes.c_int64),
                ("heads", ctypes.c_int64), ("key_dim", ctypes.c_int64), ("value_dim", ctypes.c_int64),
                ("dtype", ctypes.c_int32), ("norm_qk", ctypes.c_int32), ("scale", ctypes.c_float)]


def _declare():
    sz, st, vp, P = ctypes.c_size_t, ctypes.c_int, ctypes.c_void_p, ctypes.POINTER(GdrProblem)
    for name, args, res in (
            ("mssm_gdr_fwd_workspace_bytes", [P], sz),
            ("mssm_gdr_fwd", [P] + [vp] * 9 + [vp, sz, vp], st),
            ("mssm_gdr_ctx_bytes", [P], sz),
            ("mssm_gdr_fwd_train", [P] + [vp] * 9 + [vp, sz, vp], st),
            ("mssm_gdr_bwd_saved_workspace_bytes", [P], sz),
            ("mssm_gdr_bwd_saved", [P] + [vp] * 6 + [vp, sz] + [vp] * 8 + [vp, sz, vp], st),
            ("mssm_gdr_bwd_workspace_bytes", [P], sz),
            ("mssm_gdr_bwd", [P] + [vp] * 15 + [vp, sz, vp], st),
            ("mssm_gdr_step", [P] + [vp] * 9, st)):
        getattr(lib, name).argtypes = args
        getattr(lib, name).restype = res


_declare()


@lru_cache(maxsize=1024)
def _remembered(tokens, seqs, groups, heads, kdim, vdim, code, norm, scale, size_of):
    p = GdrProblem(tokens, seqs, groups, heads, kdim, vdim, code, norm, scale)
    return ctypes.byref(p), int(getattr(lib, size_of)(ctypes.byref(p))) if size_of else 0, p


def _problem(tokens, seqs, groups, heads, kdim, vdim, code, norm, scale, size_of):
    # by the scale's value: a tensor of one number is the same one when its value is another
    return _remembered(tokens, seqs, groups, heads, kdim, vdim, code, norm, kdim ** -0.5 if scale is None else float(scale), size_of)


def _first(t, name, dims):
    if t is None or t.dim() != len(dims):
        raise ValueError(f"{name} must be ({', '.join(dims)})")
    dev = t.get_device()
    if dev < 0:
        raise ValueError(f"{name} must be a GPU tensor")
    return dev


def _sequences(q, k, v, g, beta, offsets):
    """Checks the inputs of whole sequences; (device, element type, sizes)."""
    dev = _first(v, "v", ("B", "L", "H", "V"))
    code, act = _dtype_code(v), v.dtype
    B, L, H, V = v.shape
    if q is None or q.dim() != 4 or q.shape[2] < 1 or H % q.shape[2]:
        raise ValueError(f"q must be (B, L, G, K) with {H} heads of v a multiple of its G")
    G, K = q.shape[2:]
    _req(v, "v", (B, L, H, V), act, dev)
    _req(q, "q", (B, L, G, K), act, dev)
    _req(k, "k", (B, L, G, K), act, dev)
    _req(g, "g", (B, L, H), torch.float32, dev)
    _req(beta, "beta", (B, L, H), torch.float32, dev)
    N = B
    if offsets is not None:
        if B != 1:
            raise ValueError("packed sequences (offsets) come as one batch row")
        if offsets.dim() != 1 or offsets.shape[0] < 2:
            raise ValueError("offsets must be (sequences + 1)")
        N = offsets.shape[0] - 1
        _req(offsets, "offsets", (N + 1,), torch.int32, dev)
    return dev, act, (B * L, N, G, H, K, V, code)


def _forward(fn, size_of, q, k, v, g, beta, h0, offsets, scale, norm_qk, return_final_state, y, h_final, memory):
    dev, act, sizes = _sequences(q, k, v, g, beta, offsets)
    _, N, _, H, K, V, _ = sizes
    _opt(h0, "h0", (N, H, V, K), torch.float32, dev)
    if y is None:
        y = torch.empty_like(v)
    else:
        _req(y, "y", v.shape, act, dev)
    if h_final is not None:
        _req(h_final, "h_final", (N, H, V, K), torch.float32, dev)
    elif return_final_state:
        h_final = torch.empty((N, H, V, K), dtype=torch.float32, device=v.device)
    prob, nbytes, _ = _problem(*sizes, 1 if norm_qk else 0, scale, size_of)
    mem = _workspace(max(nbytes, 1), v.device, memory)
    if block._current_device() != dev:
        with torch.cuda.device(dev):
            return _forward(fn, size_of, q, k, v, g, beta, h0, offsets, scale, norm_qk, return_final_state, y, h_final, mem)
    _run(fn(prob, q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(), beta.data_ptr(), _ptr(h0), _ptr(offsets),
            y.data_ptr(), _ptr(h_final), mem.data_ptr(), mem.numel() * mem.element_size(), _raw_stream(dev)))
    return y, h_final, mem


def gdr_fwd(q, k, v, g, beta, h0=None, offsets=None, scale=None, norm_qk=False, return_final_state=True, y=None,
            h_final=None, workspace=None):
    """The gated delta rule over whole sequences:
    S_t = exp(g_t) S_{t-1} + beta_t (v_t - exp(g_t) S_{t-1} k_t) k_tᵀ,
    y_t = scale S_t q_t.  q, k (B, L, G, K) and v (B, L, H, V) all float32 or all
    bfloat16, H a multiple of G (head h of v goes with head h // (H // G) of q
    and k); g (log decay, <= 0) and beta (B, L, H) and the states (N, H, V, K)
    float32.  offsets (N + 1) int32: N sequences packed into one batch row, n
    from token offsets[n] to offsets[n + 1] - 1 (in ascending order; tokens of
    no sequence are left as they are); N = B without.  norm_qk: q and k divided
    by their lengths; scale: K ** -0.5 by default.  h_final may be h0.
    Returns (y, h_final) (h_final None unless requested).  No gradient is
    recorded, also of tensors that require one: gdr_bwd computes them."""
    return _forward(lib.mssm_gdr_fwd, "mssm_gdr_fwd_workspace_bytes", q, k, v, g, beta, h0, offsets, scale, norm_qk,
                    return_final_state, y, h_final, workspace)[:2]


def gdr_fwd_train(q, k, v, g, beta, h0=None, offsets=None, scale=None, norm_qk=False, return_final_state=True, y=None,
                  h_final=None, ctx=None):
    """gdr_fwd that also saves the training context for gdr_bwd_saved.  Returns
    (y, h_final, ctx); ctx is a uint8 device tensor (pass one to reuse it).  No
    gradient is recorded, also of tensors that require one: gdr_bwd_saved
    computes them."""
    return _forward(lib.mssm_gdr_fwd_train, "mssm_gdr_ctx_bytes", q, k, v, g, beta, h0, offsets, scale, norm_qk,
                    return_final_state, y, h_final, ctx)


def _backward(saved, q, k, v, g, beta, dy, h0, ctx, dh_final, offsets, scale, norm_qk, want_dh0, workspace):
    dev, act, sizes = _sequences(q, k, v, g, beta, offsets)
    _, N, _, H, K, V, _ = sizes
    state = (N, H, V, K)
    _req(dy, "dy", v.shape, act, dev)
    _opt(h0, "h0", state, torch.float32, dev)
    _opt(dh_final, "dh_final", state, torch.float32, dev)
    prob, nbytes, _ = _problem(*sizes, 1 if norm_qk else 0, scale,
                               "mssm_gdr_bwd_saved_workspace_bytes" if saved else "mssm_gdr_bwd_workspace_bytes")
    if saved:
        if ctx is None:
            raise ValueError("ctx is required")
        _workspace(max(_problem(*sizes, 1 if norm_qk else 0, scale, "mssm_gdr_ctx_bytes")[1], 1), v.device, ctx)
    ws = _workspace(max(nbytes, 1), v.device, workspace)
    if block._current_device() != dev:
        with torch.cuda.device(dev):
            return _backward(saved, q, k, v, g, beta, dy, h0, ctx, dh_final, offsets, scale, norm_qk, want_dh0, ws)
    d = {"dq": torch.empty_like(q), "dk": torch.empty_like(k), "dv": torch.empty_like(v), "dg": torch.empty_like(g),
         "dbeta": torch.empty_like(beta),
         "dh0": torch.empty(state, dtype=torch.float32, device=v.device) if want_dh0 else None}
    inputs = (q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(), beta.data_ptr())
    rest = (dy.data_ptr(), _ptr(dh_final), d["dq"].data_ptr(), d["dk"].data_ptr(), d["dv"].data_ptr(), d["dg"].data_ptr(),
            d["dbeta"].data_ptr(), _ptr(d["dh0"]), ws.data_ptr(), ws.numel() * ws.element_size(), _raw_stream(dev))
    if saved:
        _run(lib.mssm_gdr_bwd_saved(prob, *inputs, _ptr(offsets), ctx.data_ptr(), ctx.numel() * ctx.element_size(), *rest))
    else:
        _run(lib.mssm_gdr_bwd(prob, *inputs, _ptr(h0), _ptr(offsets), *rest))
    return d


def gdr_bwd(q, k, v, g, beta, dy, h0=None, dh_final=None, offsets=None, scale=None, norm_qk=False, want_dh0=True,
            workspace=None):
    """Gradients of sum(dy*y) + sum(dh_final*h_final) of gdr_fwd with the same
    arguments.  Returns a dict with dq, dk, dv (in their inputs' type), dg,
    dbeta, dh0 (float32; dh0 None unless wanted); gradients of tokens that
    belong to no sequence are left as they are (undefined)."""
    return _backward(False, q, k, v, g, beta, dy, h0, None, dh_final, offsets, scale, norm_qk, want_dh0, workspace)


def gdr_bwd_saved(q, k, v, g, beta, dy, ctx, dh_final=None, offsets=None, scale=None, norm_qk=False, want_dh0=True,
                  workspace=None):
    """gdr_bwd from the ctx that gdr_fwd_train returned for the same arguments
    (which holds h0), without recomputing the forward."""
    return _backward(True, q, k, v, g, beta, dy, None, ctx, dh_final, offsets, scale, norm_qk, want_dh0, workspace)


def gdr_step(q_t, k_t, v_t, g_t, beta_t, state, slots=None, scale=None, norm_qk=False, y=None):
    """One token of every row through its state, in place.  q_t, k_t (B, G, K),
    v_t (B, H, V), g_t, beta_t (B, H) as in gdr_fwd; state (S, H, V, K) float32.
    slots (B) int32: the state of every row (row b has state b without); a row
    whose slot is not in 0 .. S - 1 is not in use (its y is 0), and rows with the
    same slot go through their state in the order of the rows.  Returns y
    (B, H, V).  Forward only: no gradient is recorded."""
    dev = _first(v_t, "v_t", ("B", "H", "V"))
    code, act = _dtype_code(v_t), v_t.dtype
    B, H, V = v_t.shape
    if q_t is None or q_t.dim() != 3 or q_t.shape[1] < 1 or H % q_t.shape[1]:
        raise ValueError(f"q_t must be (B, G, K) with {H} heads of v_t a multiple of its G")
    G, K = q_t.shape[1:]
    _req(v_t, "v_t", (B, H, V), act, dev)
    _req(q_t, "q_t", (B, G, K), act, dev)
    _req(k_t, "k_t", (B, G, K), act, dev)
    _req(g_t, "g_t", (B, H), torch.float32, dev)
    _req(beta_t, "beta_t", (B, H), torch.float32, dev)
    if state is None or state.dim() != 4:
        raise ValueError("state must be (S, H, V, K)")
    S = state.shape[0]
    _req(state, "state", (S, H, V, K), torch.float32, dev)
    _opt(slots, "slots", (B,), torch.int32, dev)
    if slots is None and S < B:
        raise ValueError(f"{S} states for {B} rows")
    if y is None:
        y = torch.empty_like(v_t)
    else:
        _req(y, "y", (B, H, V), act, dev)
    if block._current_device() != dev:
        with torch.cuda.device(dev):
            return gdr_step(q_t, k_t, v_t, g_t, beta_t, state, slots, scale, norm_qk, y)
    _run(lib.mssm_gdr_step(_problem(B, S, G, H, K, V, code, 1 if norm_qk else 0, scale, None)[0], q_t.data_ptr(), k_t.data_ptr(),
                           v_t.data_ptr(), g_t.data_ptr(), beta_t.data_ptr(), _ptr(slots), state.data_ptr(), y.data_ptr(),
                           _raw_stream(dev)))
    return y
