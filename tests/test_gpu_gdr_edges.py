"""GPU tests of the gated delta rule over whole sequences where it can go wrong:
lengths, tokens of no sequence, offsets that are none, extreme decays and keys,
values that are no numbers, long sequences, differences, streams, graphs."""
import pytest

torch = pytest.importorskip("torch")
import gdr_ref as ref  # noqa: E402

pytestmark = pytest.mark.gpu
NAMES = ("q", "k", "v", "g", "beta")
GRADS = ("dq", "dk", "dv", "dg", "dbeta", "dh0")


@pytest.fixture(scope="module")
def mssm():
    import selective_state_space_mssm_amd as m
    return m


def args(t):
    return tuple(t[n] for n in NAMES)


def train(mssm, t, **kw):
    y, s, ctx = mssm.gdr_fwd_train(*args(t), t["h0"], offsets=t["offsets"], norm_qk=True, **kw)
    return y, s, mssm.gdr_bwd_saved(*args(t), t["dy"], ctx, t["dh_final"], offsets=t["offsets"], norm_qk=True, **kw)


def compare(mssm, x, dtype, chunks, norm=True):
    t = ref.on_gpu(x, dtype)
    want_y, want_s, want = ref.gradients(x, norm=norm)
    y, s, ctx = mssm.gdr_fwd_train(*args(t), t["h0"], offsets=t["offsets"], norm_qk=norm)
    got = mssm.gdr_bwd_saved(*args(t), t["dy"], ctx, t["dh_final"], offsets=t["offsets"], norm_qk=norm)
    ref.check(y, want_y, dtype, chunks, "y")
    ref.check(s, want_s, "f32", chunks, "h_final")
    for name, w in want.items():
        ref.check(got[name], w, dtype if name in ("dq", "dk", "dv") else "f32", chunks, name, gradient=True)


# Enough heads for each form of the forward (float32: workgroups of 64 columns, and of
# 128 from 129 pairs of a sequence and a head on; bfloat16: of 16, 64 and 128 columns).
FORMS = [("f32", 2, 128, 64), ("f32", 144, 64, 128), ("bf16", 2, 128, 64), ("bf16", 2, 64, 64), ("bf16", 100, 64, 96), ("bf16", 144, 128, 128),
         ("bf16", 300, 64, 128)]


@pytest.mark.parametrize("dtype,H,K,V", FORMS)
def test_each_form(mssm, dtype, H, K, V):
    compare(mssm, ref.inputs([3, 66], 1 if H < 100 else H // 4, H, K, V, dtype, seed=3), dtype, 2)


@pytest.mark.parametrize("dtype,H,K,V", FORMS)
def test_tokens_of_no_sequence_stay(mssm, dtype, H, K, V):
    # tokens before the first and behind the last sequence: not read, not written
    x = ref.inputs([5, 64, 70, 11], 1, H, K, V, dtype, seed=4, h0=True)
    inner = {n: (v[:, 5:139] if n in NAMES + ("dy",) else v) for n, v in x.items()}
    inner["offsets"] = torch.tensor([0, 64, 134], dtype=torch.int32)
    inner["h0"], inner["dh_final"] = x["h0"][:2], x["dh_final"][:2]
    x = {**x, "h0": inner["h0"], "dh_final": inner["dh_final"], "offsets": torch.tensor([5, 69, 139], dtype=torch.int32)}
    for n in NAMES + ("dy",):
        x[n][:, :5] = float("nan")
        x[n][:, 139:] = float("nan")
    t, u = ref.on_gpu(x, dtype), ref.on_gpu({n: v if v is None else v.contiguous() for n, v in inner.items()}, dtype)
    y = torch.full_like(t["v"], 7.0)
    y, s, ctx = mssm.gdr_fwd_train(*args(t), t["h0"], offsets=t["offsets"], norm_qk=True, y=y)
    want_y, want_s, want = train(mssm, u)
    assert torch.equal(y[:, 5:139], want_y) and torch.equal(s, want_s)
    assert torch.all(y[:, :5] == 7.0) and torch.all(y[:, 139:] == 7.0)
    got = mssm.gdr_bwd_saved(*args(t), t["dy"], ctx, t["dh_final"], offsets=t["offsets"], norm_qk=True)
    for n in GRADS:
        assert torch.equal(got[n] if n == "dh0" else got[n][:, 5:139], want[n]), n


@pytest.mark.parametrize("dtype,H,K,V", FORMS)
def test_sequences_of_no_tokens_only(mssm, dtype, H, K, V):
    x = ref.inputs([8, 0, 0], 1, H, K, V, dtype, seed=5)
    x["offsets"] = torch.tensor([3, 3, 3, 3], dtype=torch.int32)
    t = ref.on_gpu(x, dtype)
    y = torch.full_like(t["v"], 7.0)
    y, s, ctx = mssm.gdr_fwd_train(*args(t), t["h0"], offsets=t["offsets"], norm_qk=True, y=y)
    assert torch.equal(s, t["h0"]) and torch.all(y == 7.0)
    got = mssm.gdr_bwd_saved(*args(t), t["dy"], ctx, t["dh_final"], offsets=t["offsets"], norm_qk=True)
    assert torch.equal(got["dh0"], t["dh_final"])


@pytest.mark.parametrize("offsets", [[0, 200, 100, 150], [-5, 90, 1000, 2000], [150, 100, 50, 0], [2 ** 31 - 1, -2 ** 31, 7, 150],
                                     [0, 150, 150, 0]])
def test_offsets_that_are_none_stay_in_bounds(mssm, offsets):
    # results are whatever they are; what lies around every buffer stays as it was
    x = ref.inputs([50, 50, 50], 1, 2, 64, 64, "bf16", seed=6)
    t = ref.on_gpu({**x, "offsets": torch.tensor(offsets, dtype=torch.int32)}, "bf16")
    guard = 4096

    def fenced(shape, dtype):
        n = 1
        for d in shape:
            n *= d
        whole = torch.full((n + 2 * guard,), 3, dtype=dtype, device="cuda")
        return whole, whole[guard:guard + n].view(shape)

    wy, y = fenced(t["v"].shape, torch.bfloat16)
    ws, s = fenced(t["h0"].shape, torch.float32)
    need = mssm.gdr_fwd_train(*args(t), t["h0"], offsets=ref.on_gpu(x, "bf16")["offsets"], norm_qk=True)[2].numel()
    wc, ctx = fenced((need,), torch.uint8)
    mssm.gdr_fwd_train(*args(t), t["h0"], offsets=t["offsets"], norm_qk=True, y=y, h_final=s, ctx=ctx)
    mssm.gdr_bwd_saved(*args(t), t["dy"], ctx, t["dh_final"], offsets=t["offsets"], norm_qk=True)
    mssm.gdr_fwd(*args(t), t["h0"], offsets=t["offsets"], norm_qk=True, y=y, h_final=s)
    torch.cuda.synchronize()
    for w in (wy, ws, wc):
        assert torch.all(w[:guard] == 3) and torch.all(w[-guard:] == 3)


@pytest.mark.parametrize("dtype,H,K,V", FORMS[:4])
def test_extreme_decays_and_keys(mssm, dtype, H, K, V):
    x = ref.inputs([150], 1, H, K, V, dtype, seed=7)
    x["g"][0, 10], x["g"][0, 64], x["g"][0, 70], x["g"][0, 149] = -1e4, -200.0, float("-inf"), -90.0
    x["g"][0, 20:40] = 0.0
    x["beta"][0, 5:30] = 0.0
    x["beta"][0, 80:90] = 2.0
    x["k"][0, 40:60] = x["k"][0, 40].clone()     # the same key again and again
    x["k"][0, 100:110] = 0.0
    x["q"][0, 3] = 0.0
    t = ref.on_gpu(x, dtype)
    y, s, got = train(mssm, t)
    finite = {**x, "g": x["g"].clamp(min=-1e4)}  # exp is 0 either way; its derivative at -inf is no number
    want_y, want_s, want = ref.gradients(finite, norm=True)
    ref.check(y, want_y, dtype, 3, "y")
    ref.check(s, want_s, "f32", 3, "h_final")
    for n in GRADS:
        if n == "dk" or n == "dq":               # a row of no length has a gradient a thousand times the others'
            keep = x[n[1]].abs().sum(-1) > 0
            ref.check(got[n][keep.cuda()], want[n][keep], dtype, 3, n, gradient=True)
            ref.check(got[n][~keep.cuda()], want[n][~keep], dtype, 3, n, gradient=True)
        else:
            ref.check(got[n], want[n], dtype if n == "dv" else "f32", 3, n, gradient=True)


@pytest.mark.parametrize("dtype,K,V", [("f32", 64, 32), ("bf16", 128, 128), ("bf16", 64, 16)])
def test_long_sequences(mssm, dtype, K, V):
    x = ref.inputs([2500], 1, 2, K, V, dtype, seed=8, packed=False)
    t = ref.on_gpu(x, dtype)
    y, s, got = train(mssm, t)
    want_y, want_s, want = ref.gradients(x, norm=True)
    ref.check(y, want_y, dtype, 40, "y")
    ref.check(s, want_s, "f32", 40, "h_final")
    for n in GRADS:
        ref.check(got[n], want[n], dtype if n in ("dq", "dk", "dv") else "f32", 40, n, gradient=True)


@pytest.mark.parametrize("dtype,H,K,V", FORMS)
@pytest.mark.parametrize("name", NAMES)
def test_a_spoilt_token_spoils_its_sequence_only(mssm, dtype, H, K, V, name):
    x = ref.inputs([70, 200, 70], 1, H, K, V, dtype, seed=9)
    t = ref.on_gpu(x, dtype)
    bad = {**t, name: t[name].clone()}
    bad[name][0, 70 + 130, 0] = float("nan")
    y, s, got = train(mssm, t)
    y2, s2, got2 = train(mssm, bad)
    # other sequences; chunks before it (forward); other heads (of what belongs to a head)
    assert torch.equal(y2[:, :70 + 128], y[:, :70 + 128]) and torch.equal(y2[:, 270:], y[:, 270:])
    assert torch.equal(s2[0], s[0]) and torch.equal(s2[2], s[2])
    # (a query that is no number spoils its own output only)
    assert torch.isnan(y2[0, 200 if name == "q" else 269, 0]).all()
    for n in GRADS:
        if n == "dh0":
            assert torch.equal(got2[n][0], got[n][0]) and torch.equal(got2[n][2], got[n][2])
        else:
            assert torch.equal(got2[n][:, :70], got[n][:, :70]) and torch.equal(got2[n][:, 270:], got[n][:, 270:]), n
    if name in ("v", "g", "beta"):
        assert torch.equal(y2[:, :, 1:], y[:, :, 1:]) and torch.equal(s2[:, 1:], s[:, 1:])
        for n in ("dv", "dg", "dbeta"):
            assert torch.equal(got2[n][:, :, 1:], got[n][:, :, 1:]), n


def test_final_state_over_the_first(mssm):
    for dtype, H, K, V in FORMS:
        t = ref.on_gpu(ref.inputs([5, 0, 100], 1, H, K, V, dtype, seed=10), dtype)
        y, s = mssm.gdr_fwd(*args(t), t["h0"], offsets=t["offsets"], norm_qk=True)
        h = t["h0"].clone()
        y2, s2 = mssm.gdr_fwd(*args(t), h, offsets=t["offsets"], norm_qk=True, h_final=h)
        assert s2 is h and torch.equal(h, s) and torch.equal(y2, y)
        y3, s3 = mssm.gdr_fwd(*args(t), t["h0"], offsets=t["offsets"], norm_qk=True, return_final_state=False)
        assert s3 is None and torch.equal(y3, y)


def test_a_sequence_in_parts(mssm):
    # the state handed over at any token: as the whole, up to twice a value's bound
    for dtype in ("f32", "bf16"):
        x = ref.inputs([200], 2, 4, 64, 64, dtype, seed=11)
        want_y, want_s = ref.forward(x, norm=True)
        t = ref.on_gpu(x, dtype)
        state, ys = t["h0"], []
        for a, b in ((0, 1), (1, 65), (65, 90), (90, 200)):
            y, state = mssm.gdr_fwd(*(v[:, a:b].contiguous() for v in args(t)), state, norm_qk=True)
            ys.append(y)
        ref.check(torch.cat(ys, 1), want_y, dtype, 5, "y")
        ref.check(state, want_s, "f32", 5, "h_final")


@pytest.mark.parametrize("name", NAMES + ("h0",))
def test_gradients_are_differences(mssm, name):
    """Along a random direction d of an input: gradient . d against the central
    difference of the 64-bit loss with step h = 2^-10.  The difference is off by h^2 / 6
    of the third derivative along d, which for d of unit length and values of order one
    is a few times the loss's own magnitude sqrt(elements): below 2^-20 * 4 * |loss terms|.
    The gradient's elements have the forward check's bound (256 chunks 2^-24 of the
    largest); summed with d of unit length that is at most sqrt(elements) of it."""
    x = ref.inputs([70, 30], 1, 2, 32, 32, "f32", seed=12)
    t = ref.on_gpu(x, "f32")
    got = train(mssm, t)[2]["d" + name].double().cpu()
    r = torch.Generator().manual_seed(1)
    d = torch.randn(x[name].shape, generator=r, dtype=torch.float64)
    d /= d.norm()
    h = 2.0 ** -10

    def loss(at):
        y, s = ref.forward({**x, name: at}, norm=True)
        return float((y * x["dy"]).sum() + (s * x["dh_final"]).sum())

    want = (loss(x[name] + h * d) - loss(x[name] - h * d)) / (2 * h)
    terms = float(x["dy"].norm() + x["dh_final"].norm())
    room = 2 * 256 * 2.0 ** -24 * float(got.abs().max()) * d.numel() ** 0.5 + 4 * 2.0 ** -20 * terms
    assert abs(float((got * d).sum()) - want) <= room


def test_shared_heads_sum(mssm):
    # q and k of one head for four: the gradients of the four copies, summed
    for dtype in ("f32", "bf16"):
        x = ref.inputs([100], 1, 4, 64, 64, dtype, seed=13)
        t = ref.on_gpu(x, dtype)
        got = train(mssm, t)[2]
        u = {**t, "q": t["q"].repeat(1, 1, 4, 1), "k": t["k"].repeat(1, 1, 4, 1)}
        one = train(mssm, u)[2]
        for n in ("dq", "dk"):
            parts = one[n].double()
            want = parts.sum(2, keepdim=True)
            half = ref.EPS[dtype]
            # each copy is rounded once and the sum is; float32 sums of the heads besides
            bound = half * (parts.abs().sum(2, keepdim=True) + want.abs()) + 512 * 2.0 ** -24 * parts.abs().max()
            assert torch.all((got[n].double() - want).abs() <= bound), n
        for n in ("dv", "dg", "dbeta", "dh0"):
            assert torch.equal(got[n], one[n]), n


def test_calls_repeat_and_keep_their_inputs(mssm):
    for dtype, H, K, V in FORMS:
        t = ref.on_gpu(ref.inputs([64, 3, 130], 1, H, K, V, dtype, seed=14), dtype)
        kept = {n: v.clone() for n, v in t.items() if v is not None}
        first = train(mssm, t)
        for _ in range(3):
            again = train(mssm, t)
            assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
            assert all(torch.equal(first[2][n], again[2][n]) for n in GRADS)
        assert all(torch.equal(kept[n], t[n]) for n in kept)


def test_workspaces_hold_anything_before(mssm):
    t = ref.on_gpu(ref.inputs([64, 0, 131], 1, 2, 128, 64, "bf16", seed=15), "bf16")
    y, s, ctx = mssm.gdr_fwd_train(*args(t), t["h0"], offsets=t["offsets"], norm_qk=True)
    d = mssm.gdr_bwd_saved(*args(t), t["dy"], ctx, offsets=t["offsets"], norm_qk=True)
    for fill in (0, 0x7F, 0xFF):
        mem = torch.full((ctx.numel(),), fill, dtype=torch.uint8, device="cuda")
        y2, s2, _ = mssm.gdr_fwd_train(*args(t), t["h0"], offsets=t["offsets"], norm_qk=True, ctx=mem)
        ws = torch.full((64 << 20,), fill, dtype=torch.uint8, device="cuda")
        d2 = mssm.gdr_bwd_saved(*args(t), t["dy"], mem, offsets=t["offsets"], norm_qk=True, workspace=ws)
        d3 = mssm.gdr_bwd(*args(t), t["dy"], t["h0"], offsets=t["offsets"], norm_qk=True, workspace=ws.fill_(fill))
        y3, s3 = mssm.gdr_fwd(*args(t), t["h0"], offsets=t["offsets"], norm_qk=True, workspace=ws.fill_(fill))
        assert torch.equal(y2, y) and torch.equal(s2, s) and torch.equal(y3, y) and torch.equal(s3, s)
        assert all(torch.equal(d[n], d2[n]) and torch.equal(d[n], d3[n]) for n in GRADS)
    for fn in (lambda: mssm.gdr_fwd(*args(t), workspace=ws[:256], offsets=t["offsets"]),
               lambda: mssm.gdr_fwd_train(*args(t), ctx=ws[:256], offsets=t["offsets"]),
               lambda: mssm.gdr_bwd_saved(*args(t), t["dy"], ctx[:256], offsets=t["offsets"]),
               lambda: mssm.gdr_bwd_saved(*args(t), t["dy"], ctx, workspace=ws[:256], offsets=t["offsets"])):
        with pytest.raises((ValueError, RuntimeError)):
            fn()


def test_arguments_are_refused(mssm):
    t = ref.on_gpu(ref.inputs([64], 1, 2, 32, 32, "f32", seed=16, packed=False), "f32")
    z = lambda *s, **k: torch.zeros(*s, device="cuda", **k)  # noqa: E731
    i32 = torch.int32
    bad = [("q", z(1, 64, 3, 32)), ("k", z(1, 64, 1, 16)), ("g", z(1, 64, 1)), ("beta", z(64, 2)), ("h0", z(2, 2, 32, 32)),
           ("offsets", z(1, dtype=i32)), ("offsets", z(2, dtype=torch.int64)), ("k", t["k"].bfloat16()), ("g", t["g"].bfloat16()),
           ("v", z(1, 64, 2, 64)[..., ::2]), ("q", z(1, 64, 1, 32).cpu()), ("beta", z(1, 1, 2).expand(1, 64, 2))]
    for name, value in bad:
        u = {**t, name: value}
        for fn in (lambda: mssm.gdr_fwd(*args(u), u["h0"], offsets=u["offsets"]),
                   lambda: mssm.gdr_bwd(*args(u), t["dy"], u["h0"], offsets=u["offsets"])):
            with pytest.raises((ValueError, TypeError), match=name):
                fn()
    with pytest.raises(ValueError, match="packed"):
        mssm.gdr_fwd(z(2, 8, 1, 32), z(2, 8, 1, 32), z(2, 8, 2, 32), z(2, 8, 2), z(2, 8, 2), offsets=z(3, dtype=i32))
    with pytest.raises(ValueError, match="ctx"):
        mssm.gdr_bwd_saved(*args(t), t["dy"], None)
    for K, V in ((40, 32), (144, 32), (32, 8), (32, 528)):
        with pytest.raises((ValueError, RuntimeError)):
            mssm.gdr_fwd(z(1, 4, 1, K), z(1, 4, 1, K), z(1, 4, 2, V), z(1, 4, 2), z(1, 4, 2))


def test_other_streams_and_two_at_once(mssm):
    ts = [ref.on_gpu(ref.inputs([300, 64], 1, 4, 128, 128, "bf16", seed=20 + i), "bf16") for i in range(2)]
    want = [train(mssm, t) for t in ts]
    torch.cuda.synchronize()
    streams, out = [torch.cuda.Stream() for _ in ts], [None, None]
    for _ in range(3):
        for i, (s, t) in enumerate(zip(streams, ts)):
            with torch.cuda.stream(s):
                fresh = {n: v if v is None or n == "offsets" else v * 1 for n, v in t.items()}  # made on this stream just before
                out[i] = train(mssm, fresh)
        torch.cuda.synchronize()
        for w, o in zip(want, out):
            assert torch.equal(w[0], o[0]) and torch.equal(w[1], o[1]) and all(torch.equal(w[2][n], o[2][n]) for n in GRADS)


def test_captured_graphs_share_workspaces(mssm):
    """Forward, gradients and a step of two problems in two graphs that use the same
    memory, replayed in turn on new inputs, with eager calls between them."""
    fresh = lambda i: ref.on_gpu(ref.inputs([100, 30], 2, 4, 64, 64, "bf16", seed=30 + i), "bf16")  # noqa: E731
    held = [fresh(0), fresh(1)]
    mem = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")
    ctx = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")

    def work(t, m, c):
        y, s = mssm.gdr_fwd(*args(t), t["h0"], offsets=t["offsets"], norm_qk=True, workspace=m)
        y2, s2, c = mssm.gdr_fwd_train(*args(t), t["h0"], offsets=t["offsets"], norm_qk=True, ctx=c)
        d = mssm.gdr_bwd_saved(*args(t), t["dy"], c, t["dh_final"], offsets=t["offsets"], norm_qk=True, workspace=m)
        e = mssm.gdr_bwd(*args(t), t["dy"], t["h0"], t["dh_final"], offsets=t["offsets"], norm_qk=True, workspace=m)
        z = mssm.gdr_step(*(t[n][0, :2].contiguous() for n in NAMES), s2, norm_qk=True)
        return [y, s, y2, s2, z] + [d[n] for n in GRADS] + [e[n] for n in GRADS]

    graphs, outs = [], []
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for t in held:
            work(t, mem, ctx)
    torch.cuda.current_stream().wait_stream(side)
    for t in held:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(work(t, mem, ctx))
        graphs.append(g)
    for turn in range(4):
        for i in (0, 1, 1, 0):
            new = fresh(2 + 2 * turn + i)
            for n, v in held[i].items():
                v.copy_(new[n])
            graphs[i].replay()
            want = work(new, None, None)
            for a, b in zip(outs[i], want):
                assert torch.equal(a, b)
        torch.cuda.synchronize()


def test_runs_on_the_tensors_device(mssm, monkeypatch):
    from selective_state_space_mssm_amd import block
    t = ref.on_gpu(ref.inputs([40], 1, 2, 32, 32, "f32", seed=40), "f32")

    def once():
        y, s, d = train(mssm, t)
        z = mssm.gdr_step(*(t[n][0, :1].contiguous() for n in NAMES), s.clone(), norm_qk=True)
        x = torch.ones(3, 8, device="cuda")
        w = mssm.lora(x, torch.ones(2, 4, 8, device="cuda"), torch.ones(2, 8, 4, device="cuda"),
                      torch.tensor([0, 1, -1], dtype=torch.int32, device="cuda"), x.clone())
        e = mssm.gdr_bwd(*args(t), t["dy"], t["h0"], t["dh_final"], offsets=t["offsets"], norm_qk=True)
        return [y, s, z, w, *mssm.gdr_fwd(*args(t), t["h0"], offsets=t["offsets"], norm_qk=True)] + [d[n] for n in GRADS] + [e[n] for n in GRADS]

    want = once()
    entered = []

    class Device(torch.cuda.device):
        def __enter__(self):
            entered.append(self.idx)
            monkeypatch.setattr(block, "_current_device", lambda: 0)
            return super().__enter__()

        def __exit__(self, *a):
            monkeypatch.setattr(block, "_current_device", lambda: 1)
            return super().__exit__(*a)

    monkeypatch.setattr(torch.cuda, "device", Device)
    monkeypatch.setattr(block, "_current_device", lambda: 1)
    got = once()
    assert entered == [0] * 6
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    monkeypatch.undo()

    class Elsewhere(torch.Tensor):
        def get_device(self):
            return 1

    for n in ("q", "k", "g", "beta"):
        u = {**t, n: t[n].as_subclass(Elsewhere)}
        with pytest.raises(ValueError, match=f"^{n} is on"):
            mssm.gdr_fwd(*args(u))
