"""GPU tests of the gated delta rule's single tokens, against the recurrence in 64
bits.  Bounds as in gdr_ref.py: a row that is the n-th of its state has gone
through n sums of at most key_dim + 1 products, which are fewer than a chunk's,
so it is held to n times a chunk's bound."""
import pytest

torch = pytest.importorskip("torch")
import gdr_ref as ref  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mssm():
    import selective_state_space_mssm_amd as m
    return m


def make(rows, states, G, H, K, V, dtype, seed=0):
    r = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(s, generator=r, dtype=torch.float64)  # noqa: E731
    x = {"q": n(rows, G, K), "k": n(rows, G, K), "v": n(rows, H, V)}
    x = {name: t.to(ref.TYPES[dtype]).double() for name, t in x.items()}
    x["g"] = (-torch.rand((rows, H), generator=r, dtype=torch.float64)).float().double()
    x["beta"] = torch.rand((rows, H), generator=r, dtype=torch.float64).float().double()
    x["state"] = n(states, H, V, K).float().double()
    return x


def steps(x, slots, norm=True, scale=None):
    """Row after row; (y, states)."""
    K = x["q"].shape[2]
    state, y = x["state"].clone(), torch.zeros_like(x["v"])
    for b, s in enumerate(slots):
        if 0 <= s < len(state):
            one = [x[n][b:b + 1] for n in ("q", "k", "v", "g", "beta")]
            out, state[s] = ref.sequence(*one, state[s], K ** -0.5 if scale is None else scale, norm)
            y[b] = out[0]
    return y, state


def run(mssm, x, dtype, slots=None, **kw):
    t = {n: v.to(ref.TYPES[dtype] if n in ("q", "k", "v") else torch.float32).cuda() for n, v in x.items()}
    kw.setdefault("norm_qk", True)
    i = None if slots is None else torch.tensor(slots, dtype=torch.int32, device="cuda")
    y = mssm.gdr_step(t["q"], t["k"], t["v"], t["g"], t["beta"], t["state"], slots=i, **kw)
    return y, t["state"]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,G,H,K,V", [(1, 1, 1, 16, 16), (3, 2, 4, 64, 64), (5, 1, 3, 48, 80), (2, 2, 2, 128, 128), (7, 2, 6, 112, 144),
                                          (2, 1, 1, 80, 512), (70, 4, 8, 32, 48)])
def test_rows(mssm, rows, G, H, K, V, dtype):
    x = make(rows, rows + 2, G, H, K, V, dtype, seed=rows)
    for norm, scale in ((True, None), (True, 0.7)):
        y, s = run(mssm, x, dtype, norm_qk=norm, scale=scale)
        want_y, want_s = steps(x, range(rows), norm, scale)
        ref.check(y, want_y, dtype, 1, "y")
        ref.check(s, want_s, "f32", 1, "state")
        assert torch.equal(s[rows:].double().cpu(), x["state"][rows:])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_keys_as_they_are(mssm, dtype):
    x = make(4, 4, 2, 4, 64, 32, dtype)
    x["k"] = (x["k"] / 8).to(ref.TYPES[dtype]).double()
    y, s = run(mssm, x, dtype, norm_qk=False)
    want_y, want_s = steps(x, range(4), False)
    ref.check(y, want_y, dtype, 1, "y")
    ref.check(s, want_s, "f32", 1, "state")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_slots_in_any_order_and_unused_rows(mssm, dtype):
    slots = [7, -1, 0, 9, 3, 10, -2 ** 31, 2 ** 31 - 1, 5]
    x = make(len(slots), 10, 2, 4, 128, 96, dtype)
    for n in ("q", "k", "v", "g", "beta"):  # rows that are not in use are not looked at
        for b, s in enumerate(slots):
            if not 0 <= s < 10:
                x[n][b] = float("nan")
    y, s = run(mssm, x, dtype, slots)
    want_y, want_s = steps(x, slots)
    ref.check(y, want_y, dtype, 1, "y")
    ref.check(s, want_s, "f32", 1, "state")
    for b, n in enumerate(slots):
        if not 0 <= n < 10:
            assert not y[b].any()
    unused = sorted(set(range(10)) - set(slots))
    assert torch.equal(s[unused].double().cpu(), x["state"][unused])


@pytest.mark.parametrize("slots", [[2, 2], [1, 0, 1, 2, 1, 0], [0] * 5, ([3] + [1] * 63 + [0, 3]) * 2], ids=len)
def test_rows_of_one_slot_go_in_order(mssm, slots):
    x = make(len(slots), 4, 1, 2, 64, 32, "f32", seed=len(slots))
    y, s = run(mssm, x, "f32", slots)
    want_y, want_s = steps(x, slots)
    ref.check(y, want_y, "f32", max(slots.count(i) for i in set(slots)), "y")
    ref.check(s, want_s, "f32", max(slots.count(i) for i in set(slots)), "state")
    # as one row after the other, bit for bit
    state = x["state"].float().cuda()
    for b, n in enumerate(slots):
        one = [x[m][b:b + 1].float().cuda() for m in ("q", "k", "v", "g", "beta")]
        assert torch.equal(mssm.gdr_step(*one, state, slots=torch.tensor([n], dtype=torch.int32, device="cuda"), norm_qk=True)[0], y[b])
    assert torch.equal(state, s)


def test_a_spoilt_row_spoils_its_state_only(mssm):
    x = make(6, 6, 1, 2, 64, 64, "bf16")
    y, s = run(mssm, x, "bf16")
    for name in ("q", "k", "v", "g", "beta", "state"):
        bad = {n: v.clone() for n, v in x.items()}
        bad[name][2, 1 if name in ("v", "g", "beta", "state") else 0] = float("nan")
        y2, s2 = run(mssm, bad, "bf16")
        keep = [0, 1, 3, 4, 5]
        assert torch.equal(y2[keep], y[keep]) and torch.equal(s2[keep], s[keep])
        assert torch.isnan(y2[2, 1]).all()
        if name in ("v", "g", "beta", "state"):
            assert torch.equal(y2[2, 0], y[2, 0]) and torch.equal(s2[2, 0], s[2, 0])


def test_full_decay_and_no_update(mssm):
    x = make(3, 3, 1, 2, 32, 32, "f32")
    x["g"][0], x["g"][1], x["beta"][2], x["g"][2] = float("-inf"), -1e4, 0.0, 0.0
    y, s = run(mssm, x, "f32")
    want_y, want_s = steps(x, range(3))
    ref.check(y, want_y, "f32", 1, "y")
    ref.check(s, want_s, "f32", 1, "state")
    assert torch.equal(s[2].double().cpu(), x["state"][2])
    x["k"][:] = 0.0  # a key of no length, divided by its length
    y, s = run(mssm, x, "f32")
    assert torch.isfinite(y).all() and not s[0].any()


def test_given_outputs_and_refusals(mssm):
    x = make(2, 3, 1, 2, 32, 32, "f32")
    t = {n: v.float().cuda() for n, v in x.items()}
    args = [t[n] for n in ("q", "k", "v", "g", "beta")]
    y = torch.empty_like(t["v"])
    assert mssm.gdr_step(*args, t["state"].clone(), y=y) is y
    z = lambda *s, **k: torch.zeros(*s, device="cuda", **k)  # noqa: E731
    for name, err, call in [
            ("state", ValueError, lambda: mssm.gdr_step(*args, t["state"][:, :1])),
            ("states for", ValueError, lambda: mssm.gdr_step(*args, t["state"][:1].clone())),
            ("slots", ValueError, lambda: mssm.gdr_step(*args, t["state"], slots=z(3, dtype=torch.int32))),
            ("slots", TypeError, lambda: mssm.gdr_step(*args, t["state"], slots=z(2, dtype=torch.int64))),
            ("q_t", ValueError, lambda: mssm.gdr_step(z(2, 3, 32), *args[1:], t["state"])),
            ("k_t", ValueError, lambda: mssm.gdr_step(args[0], z(2, 1, 16), *args[2:], t["state"])),
            ("k_t", TypeError, lambda: mssm.gdr_step(args[0], args[1].bfloat16(), *args[2:], t["state"])),
            ("state", TypeError, lambda: mssm.gdr_step(*args, t["state"].bfloat16())),
            ("v_t", ValueError, lambda: mssm.gdr_step(args[0], args[1], z(2, 2, 64)[:, :, ::2], *args[3:], t["state"])),
            ("MSSM_ERR_SHAPE", RuntimeError, lambda: mssm.gdr_step(*args, t["state"], scale=float("nan"))),
            ("MSSM_ERR_UNSUPPORTED", RuntimeError, lambda: mssm.gdr_step(z(2, 1, 40), z(2, 1, 40), z(2, 2, 32), *args[3:], z(3, 2, 32, 40)))]:
        with pytest.raises(err, match=name):
            call()
