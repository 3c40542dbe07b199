"""GPU parity of the beam-search step (mssm_beam_select, mssm_beam_reorder) with
its definition in float64.  Tokens and parents have to be equal: the inputs keep
the deciding values further apart (2e-5, asserted on the reference) than float32
errors reach (values up to 64: log-sum within 1e-6 relative of at most 16, three
roundings of at most 4e-6), or make them exactly equal.  Scores within 2e-5."""
import numpy as np
import pytest

import block_ref as ref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
NEG = float("-inf")


@pytest.fixture(scope="module")
def mssm():
    import selective_state_space_mssm_amd as m
    return m


def check(mssm, logits, scores, finished=None, end=None, gap=2e-5):
    print(f"[beam] {tuple(logits.shape)} {logits.dtype} finished {finished is not None} end {end}", flush=True)
    s, p, t, f, least = ref.beam(logits.double().numpy(), scores.double().numpy(),
                                 None if finished is None else finished.numpy(), end)
    assert least > gap, "the inputs decide too closely"
    gs, gp, gt, gf = mssm.beam_select(logits.cuda(), scores.cuda(), None if finished is None else finished.cuda(), end)
    assert np.array_equal(gp.cpu().numpy(), p) and np.array_equal(gt.cpu().numpy(), t)
    fin = np.isfinite(s)
    gs = gs.double().cpu().numpy()
    assert np.array_equal(np.isfinite(gs), fin) and np.all(gs[~fin] == NEG)
    assert np.all(np.abs(gs[fin] - s[fin]) <= 2e-5)
    if end is None:
        assert gf is None
    else:
        assert np.array_equal(gf.cpu().numpy(), f)


def spaced(B, K, V, dtype, seed):
    """Logits whose values within a beam are apart; beams are apart by their scores (seeds chosen on the reference)."""
    g = torch.Generator().manual_seed(seed)
    x = torch.stack([torch.randperm(V, generator=g) for _ in range(B * K)]).view(B, K, V).float()
    x = x * (16.0 / V) if dtype == "f32" else (x / V * 12).bfloat16()
    return x, -torch.rand((B, K), generator=g) * 2


def good_seed(B, K, V, dtype, start=0, **kw):
    for seed in range(start, start + 200):
        x, s = spaced(B, K, V, dtype, seed)
        if ref.beam(x.double().numpy(), s.double().numpy(), **kw)[4] > 2e-5:
            return x, s
    raise AssertionError("no seed")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,K,V", [(1, 1, 1), (1, 1, 2), (2, 3, 1), (1, 4, 3), (2, 2, 63), (3, 4, 64), (2, 5, 65), (1, 16, 17), (4, 8, 100),
                                   (2, 3, 1000), (3, 16, 2049), (2, 4, 8191), (1, 7, 8193), (2, 8, 32001), (1, 16, 50277)])
def test_parity(mssm, B, K, V, dtype):
    check(mssm, *good_seed(B, K, V, dtype))


@pytest.mark.parametrize("K,V", [(1, 100), (4, 100), (8, 5000), (16, 40000)])
def test_equal_values_go_to_the_lowest_index(mssm, K, V):
    # equal beams with equal scores, every logit equal: the first K tokens of the first beam
    x, s = torch.zeros((2, K, V)), torch.zeros((2, K))
    _, p, t, _ = mssm.beam_select(x.cuda(), s.cuda())
    assert torch.all(p == 0) and torch.equal(t.cpu(), torch.arange(K).int().expand(2, K))
    # a few equal peaks far apart
    x[:, :, [V - 1, V // 2, 3]] = 5.0
    want = ref.beam(x.double().numpy(), s.double().numpy())
    _, p, t, _ = mssm.beam_select(x.cuda(), s.cuda())
    assert np.array_equal(p.cpu().numpy(), want[1]) and np.array_equal(t.cpu().numpy(), want[2])


def test_first_step_one_beam_in_use(mssm):
    x, s = good_seed(3, 4, 700, "f32", start=10)
    s[:, 1:] = NEG
    check(mssm, x, s)
    s[:, 2], s[:, 3] = float("nan"), float("inf")
    check(mssm, x, s)


def test_all_beams_out_of_use(mssm):
    x, s = spaced(2, 3, 50, "f32", 1)
    check(mssm, x, torch.full_like(s, NEG))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_banned_tokens(mssm, dtype):
    x, s = good_seed(2, 4, 3000, dtype, start=20)
    x[:, :, ::2] = NEG
    x[0, 1] = NEG                      # a beam with nothing left
    x[1, :, 1500:] = torch.finfo(x.dtype).min
    x[1, 2, :] = torch.finfo(x.dtype).min  # every logit the type's lowest: equal, not banned
    x[1, 3, 5] = float("nan")
    check(mssm, x, s)
    x[:] = NEG
    x[0, 2, 77] = 1.0                  # fewer candidates than beams
    check(mssm, x, s)


def test_infinite_logits(mssm):
    x, s = good_seed(1, 3, 200, "f32", start=30)
    x[0, 1, 50] = float("inf")
    check(mssm, x, s)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("end", [0, 7, 998])
def test_finished(mssm, end, dtype):
    x, s = good_seed(4, 4, 999, dtype, start=40)
    done = torch.zeros((4, 4), dtype=torch.bool)
    check(mssm, x, s, None, end)
    done[0, 1] = done[1, 0] = done[1, 3] = True
    done[2] = True
    s[2, 1] = NEG                      # finished and out of use
    x[0, 1] = float("nan")             # what a finished beam's logits hold does not matter
    check(mssm, x, s, done, end)
    want = ref.beam(x.double().numpy(), s.double().numpy(), done.numpy(), end)
    sc, dn = s.cuda(), done.cuda()
    out = mssm.beam_select(x.cuda(), sc, dn, end, scores_out=sc, finished_out=dn)
    assert out[0] is sc and out[3] is dn
    assert np.array_equal(out[1].cpu().numpy(), want[1]) and np.array_equal(dn.cpu().numpy(), want[3])


def test_large_logits_keep_their_differences(mssm):
    x, s = good_seed(1, 2, 300, "f32", start=50)
    big = (x * 64).round() + 4096.0    # exact in float32
    check(mssm, big, s)


def reorder_ref(t, parent):
    L, BK = t.shape[:2]
    B, K = parent.shape
    v = t.view(L, B, K, *t.shape[2:]).clone()
    out = v.clone()
    for b in range(B):
        for k in range(K):
            p = int(parent[b, k])
            if 0 <= p < K:
                out[:, b, k] = v[:, b, p]
    return out.view(t.shape)


@pytest.mark.parametrize("B,K", [(1, 1), (1, 2), (3, 4), (2, 5), (5, 8), (1, 16), (2, 13)])
def test_reorder(mssm, B, K):
    print(f"[reorder] {B} {K}", flush=True)
    g = torch.Generator().manual_seed(B * 100 + K)
    parent = torch.randint(0, K, (B, K), generator=g).int()
    states = [torch.randn((3, B * K, 70, 16), generator=g), torch.randn((3, B * K, 3, 70), generator=g).bfloat16(),
              torch.randint(0, 255, (2, B * K, 1), generator=g).to(torch.uint8),
              torch.randint(0, 255, (1, B * K, 4099), generator=g).to(torch.uint8),
              torch.randn((1, B * K, 5000), generator=g)]
    dev = [t.cuda() for t in states]
    assert mssm.beam_reorder(parent.cuda(), dev) is dev
    for t, d in zip(states, dev):
        assert torch.equal(d.cpu(), reorder_ref(t, parent)), t.shape


def test_reorder_cycles_and_strangers(mssm):
    t = torch.randn((2, 8, 1000))
    for p in ([[1, 2, 3, 0], [3, 2, 1, 0]], [[0, 1, 2, 3], [0, 0, 0, 0]], [[-1, 4, 0, 2 ** 30], [2, -2 ** 31, 1, 3]]):
        parent = torch.tensor(p, dtype=torch.int64).to(torch.int32)
        d = t.cuda()
        mssm.beam_reorder(parent.cuda(), d)
        assert torch.equal(d.cpu(), reorder_ref(t, parent))


def test_reorder_many_layers_and_rows(mssm):
    g = torch.Generator().manual_seed(3)
    parent = torch.randint(0, 4, (70, 4), generator=g).int()
    t = torch.randn((33, 280, 24), generator=g)
    d = t.cuda()
    mssm.beam_reorder(parent.cuda(), d)
    assert torch.equal(d.cpu(), reorder_ref(t, parent))


def test_select_and_reorder_in_a_graph(mssm):
    x, s = good_seed(2, 4, 5000, "f32", start=60)
    x, s = x.cuda(), s.cuda()
    state = torch.randn((2, 8, 96, 16), device="cuda")
    keep = state.clone()
    so, p, t = torch.empty_like(s), torch.empty((2, 4), dtype=torch.int32, device="cuda"), torch.empty((2, 4), dtype=torch.int32, device="cuda")
    ws = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
    g = torch.cuda.CUDAGraph()
    mssm.beam_select(x, s, scores_out=so, parent=p, token=t, workspace=ws)
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        mssm.beam_select(x, s, scores_out=so, parent=p, token=t, workspace=ws)
        mssm.beam_reorder(p, state)
    for i in range(4):
        x.copy_(x.roll(7, 2))
        s.sub_(torch.rand_like(s))
        state.copy_(keep)
        ws.fill_(255)
        es, ep, et, _ = mssm.beam_select(x, s)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(so, es) and torch.equal(p, ep) and torch.equal(t, et)
        assert torch.equal(state.cpu(), reorder_ref(keep.cpu(), ep.cpu()))


def test_more_rows_than_a_grid_dimension_holds(mssm):
    B, V = 70000, 12
    x = torch.rand((B, 1, V), device="cuda")
    s, p, t, _ = mssm.beam_select(x, torch.zeros((B, 1), device="cuda"))
    assert torch.all(p == 0) and torch.equal(t[:, 0].long(), x[:, 0].argmax(1))
    want = torch.log_softmax(x.double(), -1).amax(-1)
    assert torch.all((s.double() - want).abs() <= 2e-5)


def test_long_rows_in_several_spans_a_part(mssm):
    # 32 parts of several spans, and a part whose candidates overflow (many equal logits at the top)
    check(mssm, *good_seed(1, 3, 300001, "f32"))
    x, s = torch.zeros((1, 2, 200000)), torch.zeros((1, 2))
    x[:, :, 70000:140000] = 1.0
    s[0, 1] = -1.0
    _, p, t, _ = mssm.beam_select(x.cuda(), s.cuda())
    assert p.cpu().tolist() == [[0, 0]] and t.cpu().tolist() == [[70000, 70001]]
    x, s = torch.zeros((64, 8, 20000)), torch.zeros((64, 8))
    x[:, :, 11111:] = 2.0
    _, p, t, _ = mssm.beam_select(x.bfloat16().cuda(), s.cuda())
    assert torch.all(p == 0) and torch.equal(t.cpu(), (11111 + torch.arange(8)).int().expand(64, 8))


@pytest.mark.parametrize("K", [3, 8, 16])
def test_reorder_states_beyond_the_caches(mssm, K):
    g = torch.Generator().manual_seed(K)
    parent = torch.randint(0, K, (2, K), generator=g).int().cuda()
    rows = (torch.arange(2, device="cuda")[:, None] * K + parent).view(-1)
    t = torch.randint(0, 2 ** 31, (8, 2 * K, (300 << 20) // (64 * K) // 4 * 4), dtype=torch.int32, device="cuda")
    odd = torch.randn((2, 2 * K, 77), device="cuda").bfloat16()
    want, want_odd = t[:, rows], odd[:, rows]
    mssm.beam_reorder(parent, [t, odd])
    assert torch.equal(t, want) and torch.equal(odd, want_odd)
