"""Cases of the gated delta rule and of low-rank adapters, for measurement.

Operators, each in a plain form (elementary torch operations in float32, rounded once) and as the library's calls
(``own``):

* ``prompt``   the gated delta rule over whole sequences, of one length or packed behind one another, from their
               initial to their final states:
               S_t = exp(g_t) S_{t-1} + beta_t (v_t - exp(g_t) S_{t-1} k_t) k_tᵀ,   y_t = scale S_t q_t,
               with q and k scaled to length one first;
* ``train``    the same and the gradients of everything that goes in;
* ``token``    one token of every sequence of a batch, the states (rows of a larger pool) moved on in place;
* ``adapters`` y += scale[i] (x A_iᵀ) B_iᵀ beside a shared projection, the adapter i of every row its own.
"""
import math
import random

import torch

own = False

F32, BF16, FP8 = torch.float32, torch.bfloat16, torch.float8_e4m3fn
TYPES = {"f32": F32, "bf16": BF16, "fp8": FP8}
BYTES = {"f32": 4, "bf16": 2, "fp8": 1}
E4M3_MAX = 448.0   # the largest finite e4m3 value
NORM_EPS = 1e-6    # added to the squared length of q and k
CHUNK = 64         # steps that the plain form takes at once


# ---- the cases ---------------------------------------------------------------------------------------------------

def _mix(op, name, seqs, tokens, ragged, groups, heads, k, v, dtype, initial):
    """tokens: of all sequences together; ragged: packed with different lengths; groups: heads of q and k."""
    return {"name": name, "op": op, "seqs": seqs, "tokens": tokens, "ragged": ragged, "groups": groups, "heads": heads,
            "k": k, "v": v, "dtype": dtype, "initial": initial}


def _token(name, rows, pool, groups, heads, k, v, dtype):
    """pool: states of which the rows take some in any order (0: exactly the rows' own)."""
    return {"name": name, "op": "token", "rows": rows, "pool": pool, "groups": groups, "heads": heads, "k": k, "v": v,
            "dtype": dtype}


def _adapters(name, rows, k, n, rank, adapters, order, dtype, out):
    """order: "runs" (packed prompts, one adapter each) or "any" (every row its own); some rows have none."""
    return {"name": name, "op": "adapters", "rows": rows, "k": k, "n": n, "rank": rank, "adapters": adapters,
            "order": order, "dtype": dtype, "out": out}


def listed():
    return [
        # a prefill at the 2.8B layer's width and sizes (B = 4, L = 4096, D = 5120 = 40 heads of 128), two value
        # heads to a head of q and k
        _mix("prompt", "prompt 4 x 4096 bf16", 4, 16384, False, 20, 40, 128, 128, "bf16", False),
        # a serving batch of prompts of different lengths, packed; sequences that continue from their states
        _mix("prompt", "prompt 37 packed bf16", 37, 8191, True, 8, 32, 128, 128, "bf16", True),
        # one long document: few heads, the chain over its length
        _mix("prompt", "prompt 1 x 32768 bf16", 1, 32768, False, 16, 16, 128, 128, "bf16", False),
        # the 130M layer's sizes in float32 (B = 8, L = 2048, D = 1536 = 24 heads of 64)
        _mix("prompt", "prompt 8 x 2048 f32", 8, 16384, False, 24, 24, 64, 64, "f32", False),
        # the training workload's sizes (B = 8, L = 2048, D = 1536) in float32
        _mix("train", "train 8 x 2048 f32", 8, 16384, False, 24, 24, 64, 64, "f32", False),
        # a training step of packed documents at wide heads, shared heads of q and k
        _mix("train", "train 9 packed bf16", 9, 8192, True, 16, 32, 128, 128, "bf16", True),
        # one decode step of 4 sequences at the 2.8B layer's width: latency
        _token("token 4 rows bf16", 4, 0, 20, 40, 128, 128, "bf16"),
        # a full serving batch (B = 256): 671 MB of states read and written
        _token("token 256 rows bf16", 256, 0, 20, 40, 128, 128, "bf16"),
        # an odd batch that takes its states from a pool, float32, heads of unequal sizes
        _token("token 33 rows of a pool f32", 33, 64, 6, 24, 48, 80, "f32"),
        # one decode step of 32 requests, an adapter each, beside the 2.8B layer's input projection: latency
        _adapters("adapters 32 rows bf16", 32, 2560, 10240, 16, 32, "any", "bf16", "bf16"),
        # packed prompts on the norm's 8-bit rows, the same projection
        _adapters("adapters prefill 8 bits", 16384, 2560, 10240, 64, 16, "runs", "fp8", "bf16"),
        # everything odd: rows off any vector boundary, float32, a rank that is no power of two
        _adapters("adapters ragged f32", 300, 1537, 333, 12, 7, "any", "f32", "f32"),
    ]


def _span(rng, lo, hi):
    """A size between lo and hi, spread over the logarithm; half of them odd."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return min(hi, max(lo, v | 1 if rng.random() < 0.5 else v))


def _heads(rng):
    groups = rng.choice((1, 2, 4, 8, 16))
    return groups, groups * rng.choice((1, 1, 2, 4)) if groups <= 8 else groups


def draw(rng):
    op = rng.choice(("prompt", "prompt", "train", "token", "adapters", "adapters"))
    if op in ("prompt", "train"):
        groups, heads = _heads(rng)
        seqs, ragged = _span(rng, 1, 64), rng.random() < 0.5
        tokens = max(seqs, _span(rng, 1, 16384 if op == "prompt" else 8192))
        if not ragged:
            tokens = tokens // seqs * seqs
        c = _mix(op, "", seqs, tokens, ragged, groups, heads, 16 * rng.randint(1, 8), 16 * rng.randint(1, 8),
                 rng.choice(("f32", "bf16", "bf16")), rng.random() < 0.5)
    elif op == "token":
        groups, heads = _heads(rng)
        rows = _span(rng, 1, 256)
        c = _token("", rows, rng.choice((0, rows + rng.randint(0, 64))), groups, heads, 16 * rng.randint(1, 8),
                   16 * rng.randint(1, 8), rng.choice(("f32", "bf16")))
    else:
        dtype = rng.choice(("f32", "bf16", "fp8"))
        rows = _span(rng, 1, 16384)
        order = "runs" if rows > 1024 else rng.choice(("runs", "any"))
        c = _adapters("", rows, _span(rng, 16, 5120), _span(rng, 16, 10240), _span(rng, 4, 128), rng.randint(1, 64), order,
                      dtype, "f32" if dtype == "f32" else rng.choice(("f32", "bf16")))
        if dtype == "f32" and c["rows"] * (c["k"] + c["n"]) * c["rank"] > 2 ** 32:  # float32 products cost much more
            c["rank"] = max(1, 2 ** 32 // (c["rows"] * (c["k"] + c["n"])))
    del c["name"]
    return c


def _rng(case):
    """Numbers that belong to the case (its lengths, its runs), whatever the seed of the inputs."""
    return random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))


def _lengths(c):
    if not c["ragged"]:
        return [c["tokens"] // c["seqs"]] * c["seqs"]
    r = _rng(c)
    cuts = sorted(r.randint(0, c["tokens"]) for _ in range(c["seqs"] - 1))  # some sequences may be empty
    return [b - a for a, b in zip([0] + cuts, cuts + [c["tokens"]])]


def work(case):
    c = case
    if c["op"] in ("prompt", "train"):
        t, e, n = c["tokens"], BYTES[c["dtype"]], c["seqs"]
        qk, hv, gates, state = 2 * t * c["groups"] * c["k"] * e, t * c["heads"] * c["v"] * e, 8 * t * c["heads"], \
            4 * n * c["heads"] * c["k"] * c["v"]
        # forward: q, k, v, g, beta, states in; y, states out.  The recurrence: S k, the rank-one update, S q.
        moved = qk + 2 * hv + gates + state * (2 if c["initial"] else 1)
        flops = 6 * t * c["heads"] * c["k"] * c["v"]
        if c["op"] == "train":  # with dy and the gradients; the adjoint has six such products to the forward's three
            moved += qk + 2 * hv + gates + state * (1 if c["initial"] else 0)
            flops *= 3
        return {"bytes": moved, "flops": flops}
    if c["op"] == "token":
        b, e = c["rows"], BYTES[c["dtype"]]
        return {"bytes": b * (2 * c["groups"] * c["k"] * e + c["heads"] * (2 * c["v"] * e + 8 + 8 * c["k"] * c["v"])),
                "flops": 6 * b * c["heads"] * c["k"] * c["v"]}
    m, k, n, r = c["rows"], c["k"], c["n"], c["rank"]
    index = _index(c)
    m_used, a_used = sum(i >= 0 for i in index), len({i for i in index if i >= 0})
    e, ew, eo = BYTES[c["dtype"]], BYTES["f32" if c["dtype"] == "f32" else "bf16"], BYTES[c["out"]]
    return {"bytes": m_used * (k * e + 2 * n * eo) + a_used * r * (k + n) * ew + 4 * m,
            "flops": 2 * m_used * r * (k + n)}


def _index(c):
    """The adapter of every row; -1: none."""
    r = _rng(c)
    if c["order"] == "any":
        return [r.randrange(c["adapters"]) if r.random() < 0.9 else -1 for _ in range(c["rows"])]
    out = []
    while len(out) < c["rows"]:
        i = r.randrange(c["adapters"]) if r.random() < 0.9 else -1
        out += [i] * r.randint(1, max(1, 2 * c["rows"] // 16))
    return out[:c["rows"]]


# ---- inputs ------------------------------------------------------------------------------------------------------

def _randn(g, *shape, dtype=F32, scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def _silu(t):
    return t / (1.0 + torch.exp(-t))


def _gates(g, *shape):
    """Log decays of heads that forget fast and slowly, and write strengths, as their projections give them."""
    rate = -torch.exp(torch.empty(shape[-1], device="cuda").uniform_(math.log(0.01), math.log(2.0), generator=g))
    return rate * torch.log1p(torch.exp(_randn(g, *shape) - 1.0)), torch.sigmoid(_randn(g, *shape))


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(c)
    if c["op"] in ("prompt", "train", "token"):
        t, dt = TYPES[c["dtype"]], c["dtype"]
        if c["op"] == "token":
            lead, states = (c["rows"],), c["pool"] or c["rows"]
        else:
            lead = (1, c["tokens"]) if c["ragged"] else (c["seqs"], c["tokens"] // c["seqs"])
            states = c["seqs"]
        # q, k and v behind a short convolution with SiLU
        s["q"], s["k_t"] = (_silu(_randn(g, *lead, c["groups"], c["k"])).to(t) for _ in range(2))
        s["v_t"] = _silu(_randn(g, *lead, c["heads"], c["v"], scale=1.5)).to(t)
        s["g"], s["beta"] = _gates(g, *lead, c["heads"])
        if c["op"] == "token":
            s["state"] = _randn(g, states, c["heads"], c["v"], c["k"], scale=0.5)
            order = random.Random(seed).sample(range(states), c["rows"])
            s["slots"] = torch.tensor(order, dtype=torch.int32, device="cuda") if c["pool"] else None
            return s
        s["h0"] = _randn(g, states, c["heads"], c["v"], c["k"], scale=0.5) if c["initial"] else None
        s["lengths"] = _lengths(c)
        ends = torch.tensor([0] + s["lengths"]).cumsum(0)
        s["offsets"] = ends.to(torch.int32).cuda() if c["ragged"] else None
        s["at"] = _positions(s["lengths"])
        if c["op"] == "train":
            s["dy"] = _randn(g, *lead, c["heads"], c["v"], dtype=t)
        return s
    m, k, n, r = c["rows"], c["k"], c["n"], c["rank"]
    x = _randn(g, m, k)
    s["x_scale"] = None
    if c["dtype"] == "fp8":
        s["x_scale"] = x.abs().amax(1) / E4M3_MAX
        x = x / s["x_scale"][:, None]
    s["x"] = x.to(TYPES[c["dtype"]])
    w = F32 if c["dtype"] == "f32" else BF16
    s["a"] = _randn(g, c["adapters"], r, k, scale=k ** -0.5).to(w)
    s["b"] = _randn(g, c["adapters"], n, r, scale=0.3 * r ** -0.5).to(w)
    s["scales"] = 1.0 + torch.rand(c["adapters"], generator=g, device="cuda")
    s["y"] = _randn(g, m, n).to(TYPES[c["out"]])  # the shared projection's output
    index = _index(c)
    s["index"] = torch.tensor(index, dtype=torch.int32, device="cuda")
    s["rows_of"] = {i: torch.tensor([j for j, v in enumerate(index) if v == i], device="cuda") for i in sorted(set(index)) if i >= 0}
    return s


def _positions(lengths):
    """Where the plain forms find the tokens of sequences padded to whole chunks: (seqs, padded), -1 behind the end."""
    most = max(1, -(-max(lengths) // CHUNK)) * CHUNK
    starts = torch.tensor([0] + lengths[:-1]).cumsum(0)
    t = torch.arange(most)
    return torch.where(t < torch.tensor(lengths)[:, None], starts[:, None] + t, -1).cuda()


# ---- plain forms -------------------------------------------------------------------------------------------------

def _unit(t):
    return t * torch.rsqrt((t * t).sum(-1, keepdim=True) + NORM_EPS)


def _padded(t, at):
    """(tokens, heads, ...) -> (seqs, heads, chunks, CHUNK, ...), zeros behind a sequence's end."""
    out = torch.where((at >= 0).view(*at.shape, *[1] * (t.dim() - 1)), t[at.clamp(min=0)], 0.0)
    return out.transpose(1, 2).unflatten(2, (-1, CHUNK))


def _plain_rule(q, k, v, g, beta, h0, at, tokens):
    """All in float32, tokens in one axis; y (tokens, heads, v) and the final states (seqs, heads, v, k)."""
    heads, rep = v.shape[1], v.shape[1] // q.shape[1]
    scale = q.shape[2] ** -0.5
    q, k = (_padded(_unit(t).repeat_interleave(rep, 1), at) for t in (q, k))
    v, g, beta = _padded(v, at), _padded(g, at), _padded(beta, at)[..., None]
    since = g.double().cumsum(-1)                     # log decay from the chunk's start
    step = torch.arange(CHUNK, device=q.device)
    span = since[..., :, None] - since[..., None, :]  # ... between two steps of it
    lower = step[:, None] >= step
    decay = torch.exp(torch.where(lower, span, 0.0)).float() * lower
    # u = (1 + A)^-1 beta (v - exp(since) S k): the inverse as the product (1 - A)(1 + A^2)(1 + A^4)...
    a = (beta * decay * (k @ k.transpose(-1, -2)) * (step[:, None] > step)).double()
    one = torch.eye(CHUNK, device=q.device, dtype=torch.float64)
    inverse, power, width = one - a, a @ a, 2
    while width < CHUNK:
        inverse, power, width = inverse @ (one + power), power @ power, 2 * width
    inverse = inverse.float()
    mixed = decay * (q @ k.transpose(-1, -2))
    since = torch.exp(since).float()[..., None]
    last = since[..., -1:, :]
    to_end = torch.exp((g.double().sum(-1, keepdim=True) - g.double().cumsum(-1))).float()[..., None]
    from_v, from_s = inverse @ (beta * v), inverse @ (beta * since * k)
    q_in, k_out = since * q, (to_end * k).transpose(-1, -2)
    state = torch.zeros((at.shape[0], heads, k.shape[-1], v.shape[-1]), device=q.device) if h0 is None else h0.transpose(2, 3)
    ys = []
    for c in range(q.shape[2]):
        u = from_v[:, :, c] - from_s[:, :, c] @ state
        ys.append(scale * (q_in[:, :, c] @ state + mixed[:, :, c] @ u))
        state = last[:, :, c] * state + k_out[:, :, c] @ u
    y = torch.stack(ys, 2).flatten(2, 3).transpose(1, 2)  # (seqs, padded, heads, v)
    keep = (at >= 0).view(-1).nonzero()[:, 0]
    return y.reshape(-1, *y.shape[2:])[keep], state.transpose(2, 3)


def _flat(s, *names):
    return [s[n].float().flatten(0, 1) for n in names]


def _plain_prompt(s):
    with torch.no_grad():
        y, state = _plain_rule(*_flat(s, "q", "k_t", "v_t", "g", "beta"), s["h0"], s["at"], s["tokens"])
    return {"y": y.view(s["v_t"].shape).to(s["v_t"].dtype), "h_final": state.contiguous()}


def _plain_train(s):
    leaves = [t.detach().requires_grad_() for t in _flat(s, "q", "k_t", "v_t", "g", "beta")]
    h0 = None if s["h0"] is None else s["h0"].detach().requires_grad_()
    y, state = _plain_rule(*leaves, h0, s["at"], s["tokens"])
    grads = torch.autograd.grad(y, leaves + ([] if h0 is None else [h0]), s["dy"].float().flatten(0, 1))
    out = {"y": y.detach().view(s["v_t"].shape).to(s["v_t"].dtype), "h_final": state.detach().contiguous()}
    for name, of, grad in zip(("dq", "dk", "dv", "dg", "dbeta"), ("q", "k_t", "v_t", "g", "beta"), grads):
        out[name] = grad.view(s[of].shape).to(s[of].dtype)
    out["dh0"] = None if h0 is None else grads[5]
    return out


def _plain_token(s):
    rep = s["heads"] // s["groups"]
    q, k = (_unit(t.float()).repeat_interleave(rep, 1)[:, :, None] for t in (s["q"], s["k_t"]))  # (rows, heads, 1, k)
    state = s["state"] if s["slots"] is None else s["state"][s["slots"].long()]
    state = torch.exp(s["g"])[:, :, None, None] * state
    u = s["beta"][:, :, None, None] * (s["v_t"].float()[..., None] - (state * k).sum(-1, keepdim=True))
    state = state + u * k
    y = (state * q).sum(-1) * s["k"] ** -0.5
    if s["slots"] is None:
        s["state"].copy_(state)
    else:
        s["state"][s["slots"].long()] = state
    return {"y": y.to(s["v_t"].dtype), "state": s["state"]}


def _plain_adapters(s):
    y = s["y"].float()
    for i, rows in s["rows_of"].items():
        x = s["x"][rows].float()
        if s["x_scale"] is not None:
            x = x * s["x_scale"][rows][:, None]
        y[rows] = y[rows] + s["scales"][i] * ((x @ s["a"][i].float().t()) @ s["b"][i].float().t())
    s["y"].copy_(y)
    return {"y": s["y"]}


# ---- the library's calls -----------------------------------------------------------------------------------------

def _own_prompt(s):
    import selective_state_space_mssm_amd as mssm
    y, state = mssm.gdr_fwd(s["q"], s["k_t"], s["v_t"], s["g"], s["beta"], s["h0"], offsets=s["offsets"], norm_qk=True)
    return {"y": y, "h_final": state}


def _own_train(s):
    import selective_state_space_mssm_amd as mssm
    q, k, v, g, beta = s["q"], s["k_t"], s["v_t"], s["g"], s["beta"]
    y, state, ctx = mssm.gdr_fwd_train(q, k, v, g, beta, s["h0"], offsets=s["offsets"], norm_qk=True)
    grads = mssm.gdr_bwd_saved(q, k, v, g, beta, s["dy"], ctx, offsets=s["offsets"], norm_qk=True, want_dh0=s["h0"] is not None)
    return {"y": y, "h_final": state, **{n: grads[n] for n in ("dq", "dk", "dv", "dg", "dbeta", "dh0")}}


def _own_token(s):
    import selective_state_space_mssm_amd as mssm
    y = mssm.gdr_step(s["q"], s["k_t"], s["v_t"], s["g"], s["beta"], s["state"], slots=s["slots"], norm_qk=True)
    return {"y": y, "state": s["state"]}


def _own_adapters(s):
    import selective_state_space_mssm_amd as mssm
    return {"y": mssm.lora(s["x"], s["a"], s["b"], s["index"], s["y"], scale=s["scales"], x_scale=s["x_scale"])}


def run(state):
    if own:
        return {"prompt": _own_prompt, "train": _own_train, "token": _own_token, "adapters": _own_adapters}[state["op"]](state)
    return {"prompt": _plain_prompt, "train": _plain_train, "token": _plain_token, "adapters": _plain_adapters}[state["op"]](state)


# ---- from the definitions, in 64 bits ----------------------------------------------------------------------------

class _Steps:
    """The recurrence token by token over sequences padded to the longest; behind its end a sequence stands still."""

    def __init__(self, s):
        lengths = s["lengths"]
        self.most = max(1, max(lengths))
        starts = [sum(lengths[:i]) for i in range(len(lengths))]
        self.where = torch.tensor([[a + t if t < n else -1 for t in range(self.most)] for a, n in zip(starts, lengths)]).cuda()
        self.live = self.where >= 0
        self.rep = s["heads"] // s["groups"]
        self.scale = 1.0 / math.sqrt(s["k"])
        self.x = {n: self.spread(s[n].double().flatten(0, 1)) for n in ("q", "k_t", "v_t", "g", "beta")}
        for n in ("q", "k_t"):
            t = self.x[n]
            self.x[n] = (t / (t.square().sum(-1, keepdim=True) + NORM_EPS).sqrt()).repeat_interleave(self.rep, 2)
        self.tokens = s["tokens"]

    def spread(self, t):
        out = t.new_zeros((*self.where.shape, *t.shape[1:]))
        out[self.live] = t[self.where[self.live]]
        return out

    def gather(self, t):
        out = t.new_zeros((self.tokens, *t.shape[2:]))
        out[self.where[self.live]] = t[self.live]
        return out

    def at(self, t):
        q, k, v = (self.x[n][:, t, :, :, None] for n in ("q", "k_t", "v_t"))
        return q, k, v, self.x["g"][:, t, :, None, None].exp(), self.x["beta"][:, t, :, None, None]

    def forward(self, state, keep):
        """state (seqs, heads, v, k); keep: a list that gets every state before its token."""
        ys = torch.empty_like(self.x["v_t"])
        for t in range(self.most):
            q, k, v, decay, beta = self.at(t)
            if keep is not None:
                keep.append(state)
            state = decay * state
            state = torch.baddbmm(state.flatten(0, 1), (beta * (v - state @ k)).flatten(0, 1), k.flatten(0, 1).transpose(1, 2)).view_as(state)
            ys[:, t] = self.scale * (state @ q)[..., 0]
        return ys, state

    def backward(self, states, final, dys):
        d = {n: torch.zeros_like(t) for n, t in self.x.items()}
        adjoint, after = torch.zeros_like(final), final
        for t in reversed(range(self.most)):
            q, k, v, decay, beta = self.at(t)
            dy, before = self.scale * dys[:, t, :, :, None], states[t]
            adjoint = adjoint + dy * q.transpose(-1, -2)
            d["q"][:, t] = (after.transpose(-1, -2) @ dy)[..., 0]
            kept = decay * before
            error = v - kept @ k
            du = adjoint @ k
            de = beta * du
            d["beta"][:, t] = (du * error).sum((-1, -2))
            d["v_t"][:, t] = de[..., 0]
            d["k_t"][:, t] = (adjoint.transpose(-1, -2) @ (beta * error) - kept.transpose(-1, -2) @ de)[..., 0]
            adjoint = adjoint - de * k.transpose(-1, -2)
            d["g"][:, t] = (adjoint * kept).sum((-1, -2))
            adjoint, after = decay * adjoint, before
        return d, adjoint


def _start(s):
    shape = (len(s["lengths"]), s["heads"], s["v"], s["k"])
    return torch.zeros(shape, dtype=torch.float64, device="cuda") if s["h0"] is None else s["h0"].double()


def _through_length(x, dn, rep):
    """The gradient of x from that of x / |x|, the heads of a group added up."""
    x = x.double()
    dn = dn.unflatten(1, (-1, rep)).sum(2)
    length = (x.square().sum(-1, keepdim=True) + NORM_EPS).sqrt()
    unit = x / length
    return (dn - unit * (unit * dn).sum(-1, keepdim=True)) / length


def exact(case, seed):
    s = prepare(case, seed)
    if s["op"] == "token":
        rep = s["heads"] // s["groups"]
        q, k = ((t / (t.square().sum(-1, keepdim=True) + NORM_EPS).sqrt()).repeat_interleave(rep, 1)[..., None]
                for t in (s["q"].double(), s["k_t"].double()))
        rows = torch.arange(s["rows"], device="cuda") if s["slots"] is None else s["slots"].long()
        full = s["state"].double()
        old = full[rows] * s["g"].double().exp()[..., None, None]
        new = old + s["beta"].double()[..., None, None] * (s["v_t"].double()[..., None] - old @ k) @ k.transpose(-1, -2)
        full[rows] = new
        return {"y": (new @ q)[..., 0] / math.sqrt(s["k"]), "state": full}
    if s["op"] == "adapters":
        out = s["y"].double()
        x = s["x"].double() if s["x_scale"] is None else s["x"].double() * s["x_scale"].double()[:, None]
        for i in range(s["adapters"]):
            rows = (s["index"] == i).nonzero()[:, 0]
            inner = torch.mm(x[rows], s["a"][i].double().t()) * s["scales"][i].double()
            out[rows] += torch.mm(inner, s["b"][i].double().t())
        return {"y": out}
    with torch.no_grad():
        steps = _Steps(s)
        states = [] if s["op"] == "train" else None
        ys, final = steps.forward(_start(s), states)
        out = {"y": steps.gather(ys).view(s["v_t"].shape), "h_final": final}
        if s["op"] == "prompt":
            return out
        d, dh0 = steps.backward(states, final, steps.spread(s["dy"].double().flatten(0, 1)))
        del states
        for name, of in (("dq", "q"), ("dk", "k_t")):
            out[name] = _through_length(s[of].flatten(0, 1), steps.gather(d[of]), steps.rep).view(s[of].shape)
        for name, of in (("dv", "v_t"), ("dg", "g"), ("dbeta", "beta")):
            out[name] = steps.gather(d[of]).view(s[of].shape)
        out["dh0"] = None if s["h0"] is None else dh0
        return out
