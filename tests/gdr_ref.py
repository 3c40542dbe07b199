"""The gated delta rule in 64 bits, token by token from its definition, and the
bounds that the kernels' outputs are held to.

Bounds: a kernel's float32 value is a chain of sums of up to key_dim + 64
products of float32 values, through as many chunks as the sequence has.  One
rounding is 2^-24 of what is added; with the magnitudes of what is added up to a
few times the largest value M of the output, their errors add up like random
ones to about sqrt(192) * 2 of them a chunk, 28; four standard deviations are
112, and errors of earlier chunks enter later ones through a state that is
contracted (beta |k|^2 <= 2), at most as many times again as there are chunks.
So |value - exact| <= 128 chunks 2^-24 M forward; a gradient goes through two
such chains and is held to twice that.  An output in bfloat16 is rounded once, 2^-8 of
itself, and y is then summed from operands of 16 bits each (2^-15 of M in all).
"""
import numpy as np
import torch

EPS = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
NORM_EPS = 1e-6


def inputs(lengths, G, H, K, V, dtype="f32", seed=0, h0=True, unit=False, packed=True, device="cpu"):
    """Inputs as float64 that are exact in `dtype`; unit: q and k of length one (to be used without norm_qk)."""
    r = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(s, generator=r, dtype=torch.float64)  # noqa: E731
    T = sum(lengths)
    lead = (1, T) if packed else (len(lengths), lengths[0])
    x = {"q": n(*lead, G, K), "k": n(*lead, G, K), "v": n(*lead, H, V)}
    if unit:
        x["q"], x["k"] = (t / t.norm(dim=-1, keepdim=True) for t in (x["q"], x["k"]))
    x = {name: t.to(TYPES[dtype]).double() for name, t in x.items()}
    x["g"] = (-0.5 * torch.rand((*lead, H), generator=r, dtype=torch.float64) ** 3).float().double()
    x["beta"] = torch.rand((*lead, H), generator=r, dtype=torch.float64).float().double()
    x["h0"] = n(len(lengths), H, V, K).float().double() if h0 else None
    x["dy"] = n(*lead, H, V).to(TYPES[dtype]).double()
    x["dh_final"] = n(len(lengths), H, V, K).float().double()
    x["offsets"] = torch.tensor([0] + list(np.cumsum(lengths)), dtype=torch.int32) if packed else None
    return x


def on_gpu(x, dtype):
    out = {}
    for name, t in x.items():
        if t is None or name == "offsets":
            out[name] = None if t is None else t.cuda()
        else:
            out[name] = t.to(TYPES[dtype] if name in ("q", "k", "v", "dy") else torch.float32).cuda()
    return out


def unit(t):
    return t / torch.sqrt((t * t).sum(-1, keepdim=True) + NORM_EPS)


def sequence(q, k, v, g, beta, state, scale, norm):
    """One sequence: q, k (L, G, K), v (L, H, V), g, beta (L, H), state (H, V, K); (y, final state)."""
    rep = v.shape[1] // q.shape[1]
    if norm:
        q, k = unit(q), unit(k)
    q, k = q.repeat_interleave(rep, 1), k.repeat_interleave(rep, 1)
    ys = []
    for t in range(v.shape[0]):
        state = torch.exp(g[t])[:, None, None] * state
        e = v[t] - (state * k[t][:, None, :]).sum(-1)
        state = state + (beta[t][:, None] * e)[:, :, None] * k[t][:, None, :]
        ys.append(scale * (state * q[t][:, None, :]).sum(-1))
    return (torch.stack(ys) if ys else v.new_zeros(v.shape)), state


def forward(x, scale=None, norm=False):
    """(y, h_final) of the inputs, sequence by sequence; differentiable."""
    B, L, H, V = x["v"].shape
    K = x["q"].shape[3]
    scale = K ** -0.5 if scale is None else scale
    flat = {n: x[n].flatten(0, 1) for n in ("q", "k", "v", "g", "beta")}
    ends = x["offsets"].tolist() if x["offsets"] is not None else [L * i for i in range(B + 1)]
    ys, finals = [], []
    for n, (a, b) in enumerate(zip(ends, ends[1:])):
        s0 = x["h0"][n] if x["h0"] is not None else torch.zeros((H, V, K), dtype=torch.float64)
        y, s = sequence(*(flat[m][a:b] for m in ("q", "k", "v", "g", "beta")), s0, scale, norm)
        ys.append(y)
        finals.append(s)
    return torch.cat(ys).view(x["v"].shape), torch.stack(finals)


def gradients(x, scale=None, norm=False, dh_final=True):
    names = ["q", "k", "v", "g", "beta"] + (["h0"] if x["h0"] is not None else [])
    leaves = {n: x[n].clone().requires_grad_() for n in names}
    y, s = forward({**x, **leaves}, scale, norm)
    loss = (y * x["dy"]).sum() + ((s * x["dh_final"]).sum() if dh_final else 0.0)
    return y.detach(), s.detach(), dict(zip(["d" + n for n in names], torch.autograd.grad(loss, list(leaves.values()))))


def check(got, want, dtype, chunks, name, gradient=False):
    got, want = got.detach().double().cpu(), want.detach().double()
    m = float(want.abs().max()) if want.numel() else 0.0
    bound = 128 * chunks * (2 if gradient else 1) * 2.0 ** -24 * m
    if dtype == "bf16":
        bound = bound + EPS["bf16"] * want.abs() + 2.0 ** -15 * m
    else:
        bound = bound + EPS["f32"] * want.abs()
    off = (got - want).abs()
    assert torch.all(off <= bound), f"{name}: off by {float(off.max()):.3g} of {m:.3g}, {float((off / (bound + 1e-300)).max()):.2f} of the bound"
