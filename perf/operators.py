"""Cases of the operators that serve a Mamba block around its scan, for measurement.

Three operators, each in a plain form (elementary torch operations in float32, rounded once) and as the library's
calls (``own``):

* ``norm``    residual addition + root-mean-square norm, its output in 8 bits (e4m3 with one scale a row) or in the
              input's type;
* ``linear``  the projections: y = act(x wᵀ · scales + bias) + residual, for float32, bfloat16 and 8-bit operands;
* ``beam``    one beam-search step: the K best of K·V continuations of every batch row, then the beams' recurrent and
              convolution states reordered in place.
"""
import math

import torch

own = False

E4M3_MAX = 448.0      # the largest finite e4m3 value
SCALE_FLOOR = 1e-30   # a row whose largest magnitude is below this is scaled as if it were this

F32, BF16, FP8 = torch.float32, torch.bfloat16, torch.float8_e4m3fn
TYPES = {"f32": F32, "bf16": BF16, "fp8": FP8}
BYTES = {"f32": 4, "bf16": 2, "fp8": 1}


# ---- the cases ---------------------------------------------------------------------------------------------------

def _norm(name, rows, dim, dtype, residual, out):
    return {"name": name, "op": "norm", "rows": rows, "dim": dim, "dtype": dtype, "residual": residual, "out": out}


def _linear(name, rows, k, n, dtype, out, act="none", bias=False, residual=False):
    return {"name": name, "op": "linear", "rows": rows, "k": k, "n": n, "dtype": dtype, "out": out, "act": act,
            "bias": bias, "residual": residual}


def _beam(name, batch, beams, vocab, dtype, layers, dim, finished):
    return {"name": name, "op": "beam", "batch": batch, "beams": beams, "vocab": vocab, "dtype": dtype,
            "layers": layers, "dim": dim, "dstate": 16, "dconv": 4, "finished": finished}


def listed():
    return [
        # one decode step of 4 sequences at the 2.8B layer's model width (D = 5120 = 2 x 2560): latency alone
        _norm("norm 4 tokens to 8 bits", 4, 2560, "bf16", "f32", "fp8"),
        # the 2.8B layer's prefill (B = 4, L = 4096), float32 residual stream, feeding an 8-bit projection
        _norm("norm prefill to 8 bits", 16384, 2560, "bf16", "f32", "fp8"),
        # a ragged batch in float32: odd width, rows that start off a 16-byte boundary
        _norm("norm ragged f32", 2047, 1537, "f32", "f32", "f32"),
        # single-token decode through the 2.8B layer's input projection (u and z): a read of the weights
        _linear("in_proj 1 token bf16", 1, 2560, 10240, "bf16", "bf16"),
        # the logits of 8 sequences with 4 beams each: the largest weight, few rows
        _linear("logits 32 rows bf16", 32, 2560, 50280, "bf16", "f32"),
        # the 2.8B layer's input projection over a prefill, on the norm's 8-bit rows
        _linear("in_proj prefill 8 bits", 16384, 2560, 10240, "fp8", "bf16"),
        # its output projection with the float32 residual stream added in the epilogue
        _linear("out_proj prefill bf16", 16384, 5120, 2560, "bf16", "f32", residual=True),
        # everything odd at once: a K whose rows start off any vector boundary, ragged tiles, the whole epilogue
        _linear("linear ragged bf16", 300, 1537, 333, "bf16", "bf16", "gelu", bias=True, residual=True),
        # the 130M layer's projection to step size, B and C (48 + 2 x 16) in float32: a narrow output, many rows
        _linear("x_proj prefill f32", 16384, 1536, 80, "f32", "f32"),
        # one request with 4 beams on the 130M layer's states (24 layers): latency
        _beam("beam 1 x 4", 1, 4, 50280, "f32", 24, 1536, 0.0),
        # 8 requests with 4 beams on the 2.8B layer's states (64 layers): 734 MB of states to reorder
        _beam("beam 8 x 4, deep states", 8, 4, 50280, "f32", 64, 5120, 0.1),
        # the selection alone over a full serving batch
        _beam("beam 64 x 8, selection", 64, 8, 50280, "bf16", 0, 0, 0.1),
    ]


def _span(rng, lo, hi):
    """A size between lo and hi, spread over the logarithm; half of them odd."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    v = min(hi, max(lo, v | 1 if rng.random() < 0.5 else v))
    return v + 1 if v == 3 * 1024 else v


def _width(rng, lo, hi):
    """A model width: a multiple of 16 half of the time, any number otherwise."""
    v = _span(rng, lo, hi)
    v = max(lo, v // 16 * 16) if rng.random() < 0.5 else v
    return v + 16 if v == 3 * 1024 else v


def draw(rng):
    op = rng.choice(("norm", "linear", "linear", "beam"))
    if op == "norm":
        dtype = rng.choice(("f32", "bf16"))
        c = _norm("", _span(rng, 1, 16384), _width(rng, 16, 5120), dtype, rng.choice(("none", "f32", "bf16")),
                  rng.choice((dtype, "fp8")))
    elif op == "linear":
        dtype = rng.choice(("f32", "bf16", "fp8"))
        rows, k = _span(rng, 1, 16384), _width(rng, 16, 5120)
        n = _width(rng, 16, 50280 if rows <= 64 else 10240)
        if dtype == "f32" and rows * k * n > 2 ** 36:  # float32 products cost sixteen times as much
            rows = max(1, 2 ** 36 // (k * n))
        c = _linear("", rows, k, n, dtype, rng.choice(("f32", "bf16")) if dtype != "f32" else "f32",
                    rng.choice(("none", "relu", "silu", "gelu")), rng.random() < 0.5, rng.random() < 0.5)
    else:
        batch, beams = _span(rng, 1, 64), rng.randint(1, 8)
        layers = rng.choice((0, 1, 8, 24))
        dim = _width(rng, 64, 1536) if layers else 0
        c = _beam("", batch, beams, _span(rng, 100, 50280), rng.choice(("f32", "bf16")), layers, dim,
                  rng.choice((0.0, 0.1, 0.5)))
    del c["name"]
    return c


def work(case):
    c = case
    if c["op"] == "norm":
        per = BYTES[c["dtype"]] + BYTES[c["out"]] + (2 * BYTES[c["residual"]] if c["residual"] != "none" else 0)
        scales = 4 * c["rows"] if c["out"] == "fp8" else 0
        return {"bytes": c["rows"] * c["dim"] * per + 4 * c["dim"] + scales, "flops": 6 * c["rows"] * c["dim"]}
    if c["op"] == "linear":
        m, k, n, o = c["rows"], c["k"], c["n"], BYTES[c["out"]]
        b = (m * k + n * k) * BYTES[c["dtype"]] + m * n * o * (2 if c["residual"] else 1) + (4 * n if c["bias"] else 0)
        return {"bytes": b + (4 * (m + n) if c["dtype"] == "fp8" else 0), "flops": 2 * m * n * k}
    b, k = c["batch"], c["beams"]
    read = b * k * c["vocab"] * BYTES[c["dtype"]] + 17 * b * k
    seq = c["layers"] * c["dim"] * (4 * c["dstate"] + 2 * (c["dconv"] - 1))  # one beam's states
    # beams whose parent is another one are written; the distinct parents of those are read (parents spread evenly)
    moved = b * k * (1 - 1 / k)
    parents = b * k * (1 - (1 - 1 / k) ** (k - 1))
    return {"bytes": read + seq * (moved + parents), "flops": 4 * b * k * c["vocab"]}


# ---- inputs ------------------------------------------------------------------------------------------------------

def _randn(g, *shape, dtype=F32, scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def _rows8(t):
    """Rows in 8 bits with a scale each, as a program keeps its weights."""
    scale = t.abs().amax(1).clamp(min=SCALE_FLOOR) / E4M3_MAX
    return (t / scale[:, None]).to(FP8), scale


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(c)
    if c["op"] == "norm":
        # a block's output next to a residual stream that has grown over the layers; a few wide channels
        x = _randn(g, c["rows"], c["dim"])
        x[:, :: max(1, c["dim"] // 7)] *= 8.0
        s["x"] = x.to(TYPES[c["dtype"]])
        s["res"] = None if c["residual"] == "none" else _randn(g, c["rows"], c["dim"], dtype=TYPES[c["residual"]], scale=3.0)
        s["weight"] = 1.0 + _randn(g, c["dim"], scale=0.2)
        s["eps"] = 1e-5
    elif c["op"] == "linear":
        m, k, n = c["rows"], c["k"], c["n"]
        x, w = _randn(g, m, k), _randn(g, n, k, scale=k ** -0.5)
        s["xs"] = s["ws"] = None
        if c["dtype"] == "fp8":
            (s["x"], s["xs"]), (s["w"], s["ws"]) = _rows8(x), _rows8(w)
        else:
            s["x"], s["w"] = x.to(TYPES[c["dtype"]]), w.to(TYPES[c["dtype"]])
        s["bias_t"] = _randn(g, n) if c["bias"] else None
        s["res"] = _randn(g, m, n, dtype=TYPES[c["out"]]) if c["residual"] else None
    else:
        b, k, v = c["batch"], c["beams"], c["vocab"]
        s["logits"] = _randn(g, b, k, v, dtype=TYPES[c["dtype"]], scale=2.5)
        s["logits"][:, :, 1::97] = -math.inf  # tokens that the program bans
        s["scores"] = -2.0 + _randn(g, b, k, scale=0.5)
        s["done"] = torch.rand((b, k), generator=g, device="cuda") < c["finished"] if c["finished"] > 0 else None
        s["end"] = 2
        s["states"] = []
        if c["layers"]:
            s["states"] = [_randn(g, c["layers"], b * k, c["dim"], c["dstate"]),
                           _randn(g, c["layers"], b * k, c["dconv"] - 1, c["dim"], dtype=BF16)]
    return s


# ---- plain forms -------------------------------------------------------------------------------------------------

def _plain_norm(s):
    h = s["x"].float()
    res = None
    if s["res"] is not None:
        h = h + s["res"].float()
        res = h.to(s["res"].dtype)
    y = h * torch.rsqrt((h * h).mean(1, keepdim=True) + s["eps"]) * s["weight"]
    if s["out"] != "fp8":
        return {"y": y.to(TYPES[s["out"]]), "residual": res}
    scale = y.abs().amax(1).clamp(min=SCALE_FLOOR) / E4M3_MAX
    return {"y": (y / scale[:, None]).to(FP8), "scale": scale, "residual": res}


def _plain_linear(s):
    y = s["x"].float() @ s["w"].float().t()
    if s["xs"] is not None:
        y = y * s["xs"][:, None] * s["ws"]
    if s["bias_t"] is not None:
        y = y + s["bias_t"]
    if s["act"] == "relu":
        y = torch.where(y > 0, y, 0.0)
    elif s["act"] == "silu":
        y = y / (1.0 + torch.exp(-y))
    elif s["act"] == "gelu":
        y = 0.5 * y * (1.0 + torch.erf(y * 0.5 ** 0.5))
    if s["res"] is not None:
        y = y + s["res"].float()
    return {"y": y.to(TYPES[s["out"]])}


def _plain_beam(s):
    b, k, v = s["logits"].shape
    x = s["logits"].float()
    top = x.amax(2, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    total = torch.exp(x - top).sum(2, keepdim=True)
    cand = torch.where(x == -math.inf, x, s["scores"][:, :, None] + ((x - top) - torch.log(total)))
    if s["done"] is not None:  # a finished beam has one continuation: itself
        cand = torch.where(s["done"][:, :, None], -math.inf, cand)
        cand[:, :, s["end"]] = torch.where(s["done"], s["scores"], cand[:, :, s["end"]])
    best, at = torch.sort(cand.view(b, k * v), dim=1, descending=True, stable=True)
    scores, at = best[:, :k].contiguous(), at[:, :k]
    parent, token = (at // v).int(), (at % v).int()
    out = {"scores": scores, "parent": parent, "token": token, "states": s["states"]}
    if s["done"] is not None:
        out["finished"] = s["done"].gather(1, parent.long()) | (token == s["end"])
    rows = (torch.arange(b, device=parent.device)[:, None] * k + parent).view(-1)
    if s["states"]:
        s["states"][0].copy_(s["states"][0].index_select(1, rows))
        s["states"][1].copy_(s["states"][1].index_select(1, rows))
    return out


# ---- the library's calls -----------------------------------------------------------------------------------------

def _own_norm(s):
    import selective_state_space_mssm_amd as mssm
    if s["out"] != "fp8":
        y, res = mssm.add_rmsnorm(s["x"], s["weight"], s["res"], s["eps"])
        return {"y": y, "residual": res}
    y, scale, res = mssm.add_rmsnorm_q8(s["x"], s["weight"], s["res"], s["eps"])
    return {"y": y, "scale": scale, "residual": res}


def _own_linear(s):
    import selective_state_space_mssm_amd as mssm
    return {"y": mssm.linear(s["x"], s["w"], s["bias_t"], s["res"], activation=s["act"], x_scale=s["xs"], w_scale=s["ws"],
                             out_dtype=TYPES[s["out"]])}


def _own_beam(s):
    import selective_state_space_mssm_amd as mssm
    end = s["end"] if s["done"] is not None else None
    scores, parent, token, done = mssm.beam_select(s["logits"], s["scores"], finished=s["done"], end_token=end)
    if s["states"]:
        mssm.beam_reorder(parent, s["states"])
    out = {"scores": scores, "parent": parent, "token": token, "states": s["states"]}
    if done is not None:
        out["finished"] = done
    return out


def run(state):
    if own:
        return {"norm": _own_norm, "linear": _own_linear, "beam": _own_beam}[state["op"]](state)
    return {"norm": _plain_norm, "linear": _plain_linear, "beam": _plain_beam}[state["op"]](state)


# ---- from the definitions, in 64 bits ----------------------------------------------------------------------------

def _round_e4m3(v):
    """The nearest e4m3 values (ties to even): 3 mantissa bits down to 2^-6, steps of 2^-9 below."""
    _, e = torch.frexp(v)
    step = torch.ldexp(torch.ones_like(v), (e - 1).clamp(min=-6) - 3)
    return (torch.round(v / step) * step).clamp(-E4M3_MAX, E4M3_MAX)


def exact(case, seed):
    s = prepare(case, seed)
    if s["op"] == "norm":
        h = s["x"].double() + (0.0 if s["res"] is None else s["res"].double())
        y = h / torch.sqrt(h.pow(2).sum(1, keepdim=True) / h.shape[1] + s["eps"]) * s["weight"].double()
        res = None if s["res"] is None else h
        if s["out"] != "fp8":
            return {"y": y, "residual": res}
        scale = y.abs().max(1).values.clamp(min=SCALE_FLOOR) / E4M3_MAX
        return {"y": _round_e4m3(y / scale[:, None]), "scale": scale, "residual": res}
    if s["op"] == "linear":
        y = torch.mm(s["x"].double(), s["w"].double().t())
        if s["xs"] is not None:
            y = y * torch.outer(s["xs"].double(), s["ws"].double())
        y = y if s["bias_t"] is None else y + s["bias_t"].double()
        if s["act"] == "relu":
            y = y.clamp(min=0.0)
        elif s["act"] == "silu":
            y = y * (0.5 + 0.5 * torch.tanh(0.5 * y))
        elif s["act"] == "gelu":
            y = 0.5 * y * torch.special.erfc(-y / math.sqrt(2.0))
        return {"y": y if s["res"] is None else y + s["res"].double()}
    b, k, v = s["logits"].shape
    x = s["logits"].double()
    cand = x - torch.logsumexp(x, 2, keepdim=True) + s["scores"].double()[:, :, None]
    if s["done"] is not None:
        cand = cand.masked_fill(s["done"][:, :, None], -math.inf)
        at = s["done"].nonzero()
        cand[at[:, 0], at[:, 1], s["end"]] = s["scores"].double()[at[:, 0], at[:, 1]]
    scores, at = cand.view(b, k * v).topk(k, dim=1)
    rows = (at // v + k * torch.arange(b, device=at.device)[:, None]).view(-1)
    out = {"scores": scores, "parent": None, "token": None, "states": [t[:, rows].double() for t in s["states"]]}
    if s["done"] is not None:
        out["finished"] = None
    return out
