"""The gated delta rule and the adapters as a server uses them together: packed
prompts of requests that each have an adapter, their states into a pool, then
tokens one at a time from the pool, requests leaving and the batch changing its
order; against the whole sequences in 64 bits.

Bounds: the rows q, k, v, g and beta come from sums of D = 96 and R = 8 float32
products, off by up to 4 sqrt(D) 2^-24, 40 2^-24, of the largest; the recurrence
adds its own 128 chunks 2^-24 (gdr_ref.py) and hands those on as it does its
own: so (128 + 40 * 4) chunks 2^-24 of the largest value, 4 for the five inputs'
independent errors and the outputs that they share."""
import pytest

torch = pytest.importorskip("torch")
import gdr_ref as ref  # noqa: E402

pytestmark = pytest.mark.gpu
D, G, H, K, V, R, S = 96, 2, 4, 32, 48, 8, 3
WIDTH = 2 * G * K + H * V


@pytest.fixture(scope="module")
def mssm():
    import selective_state_space_mssm_amd as m
    return m


def weights(seed):
    r = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(s, generator=r).double()  # noqa: E731
    return dict(w=(n(WIDTH, D) * D ** -0.5).float().double(), gates=(n(2 * H, D) * D ** -0.5).float().double(),
                a=(n(S, R, D) * D ** -0.5).float().double(), b=(n(S, WIDTH, R) * R ** -0.5).float().double(),
                scale=torch.tensor([0.5, 1.0, 2.0], dtype=torch.float64))


def gates(z):
    return -torch.nn.functional.softplus(z[..., :H]), torch.sigmoid(z[..., H:])


def split(rows):
    q, k, v = rows.split([G * K, G * K, H * V], -1)
    return q.unflatten(-1, (G, K)), k.unflatten(-1, (G, K)), v.unflatten(-1, (H, V))


def whole(p, x, adapter):
    rows = x @ p["w"].T
    if 0 <= adapter < S:
        rows = rows + p["scale"][adapter] * (x @ p["a"][adapter].T) @ p["b"][adapter].T
    g, beta = gates(x @ p["gates"].T)
    return ref.sequence(*split(rows), g, beta, torch.zeros(H, V, K, dtype=torch.float64), K ** -0.5, True)


def test_prompts_and_tokens_of_many_requests(mssm):
    p, r = weights(1), torch.Generator().manual_seed(2)
    prompts, adapters, slots, tokens = [70, 1, 129, 33], [2, -1, 0, 2], [5, 0, 3, 1], [4, 6, 2, 6]
    xs = [torch.randn(n + m, D, generator=r).double() for n, m in zip(prompts, tokens)]
    u = {n: v.float().cuda() for n, v in p.items()}

    def layer(x, index):
        rows = mssm.linear(x, u["w"])
        mssm.lora(x, u["a"], u["b"], index, rows, scale=u["scale"])
        return *(t.contiguous() for t in split(rows)), *(t.contiguous() for t in gates(mssm.linear(x, u["gates"])))

    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    x = torch.cat([t[:n] for t, n in zip(xs, prompts)]).float().cuda()
    index = i32([a for a, n in zip(adapters, prompts) for _ in range(n)])
    q, k, v, g, beta = (t[None] for t in layer(x, index))
    offsets = i32([0] + list(torch.tensor(prompts).cumsum(0)))
    y, states = mssm.gdr_fwd(q, k, v, g, beta, offsets=offsets, norm_qk=True)
    pool = torch.full((7, H, V, K), 9.0, device="cuda")
    pool[slots] = states
    got = [list(t) for t in y[0].split(prompts)]
    for step in range(max(tokens)):
        live = [i for i in range(4) if step < tokens[i]]
        live = live[::-1] if step % 2 else live
        x = torch.stack([xs[i][prompts[i] + step] for i in live]).float().cuda()
        out = mssm.gdr_step(*layer(x, i32([adapters[i] for i in live])), pool, slots=i32([slots[i] for i in live]), norm_qk=True)
        for i, o in zip(live, out):
            got[i].append(o)
    for i in range(4):
        want_y, want_s = whole(p, xs[i], adapters[i])
        chunks = -(-prompts[i] // 64) + tokens[i]
        for name, a, w in (("y", torch.stack(got[i]), want_y), ("state", pool[slots[i]], want_s)):
            off = (a.double().cpu() - w).abs().max()
            assert off <= 288 * chunks * 2.0 ** -24 * w.abs().max(), (i, name, float(off), float(w.abs().max()))
    for n in set(range(7)) - set(slots):
        assert torch.all(pool[n] == 9.0)


def test_training_step_of_a_layer(mssm):
    """Rows from a projection, the recurrence, and the gradient back to the weights,
    against the same in 64 bits.  The loss's gradient of the weights sums 134 rows'
    gradients, each within 2 * 128 * 2 chunks 2^-24 of its largest (gdr_ref.py), in the
    float32 library product, and rows' own errors as above: twice (256 + 160) chunks 2^-24
    of the largest, times sqrt(134) for sums of independent ones over their largest."""
    p, r = weights(3), torch.Generator().manual_seed(4)
    x = torch.randn(134, D, generator=r).double()
    dy = torch.randn(1, 134, H, V, generator=r).double()
    ends = [0, 70, 134]

    w, wg = p["w"].clone().requires_grad_(), p["gates"].clone().requires_grad_()
    rows, (g, beta) = x @ w.T, gates(x @ wg.T)
    zero = torch.zeros(H, V, K, dtype=torch.float64)
    ys = [ref.sequence(*(t[a:b] for t in (*split(rows), g, beta)), zero, K ** -0.5, True)[0] for a, b in zip(ends, ends[1:])]
    want = torch.autograd.grad((torch.cat(ys) * dy[0]).sum(), (w, wg))

    xf, w, wg = x.float().cuda(), p["w"].float().cuda(), p["gates"].float().cuda()
    q, k, v = (t.contiguous()[None] for t in split(mssm.linear(xf, w)))
    z = mssm.linear(xf, wg).requires_grad_()
    g, beta = gates(z)
    args = (q, k, v, g.detach().contiguous()[None], beta.detach().contiguous()[None])
    offsets = torch.tensor(ends, dtype=torch.int32, device="cuda")
    _, _, ctx = mssm.gdr_fwd_train(*args, offsets=offsets, norm_qk=True, return_final_state=False)
    d = mssm.gdr_bwd_saved(*args, dy.float().cuda(), ctx, offsets=offsets, norm_qk=True, want_dh0=False)
    dz, = torch.autograd.grad((g, beta), z, (d["dg"][0], d["dbeta"][0]))
    drows = torch.cat([d[n][0].flatten(1) for n in ("dq", "dk", "dv")], 1)
    for got, w in ((drows.T.contiguous() @ xf, want[0]), (dz.T.contiguous() @ xf, want[1])):
        off = (got.double().cpu() - w).abs().max()
        assert off <= 2 * (256 + 160) * 2 * 2.0 ** -24 * 134 ** 0.5 * w.abs().max(), (float(off), float(w.abs().max()))
