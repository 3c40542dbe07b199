"""GPU tests of the gated delta rule where long sequences of few heads are gone
through in pieces side by side, against the recurrence in 64 bits (gdr_ref.py has
it, and the bounds)."""
import pytest

torch = pytest.importorskip("torch")
import gdr_ref as ref  # noqa: E402
from test_gpu_gdr_edges import GRADS, args, train  # noqa: E402

pytestmark = pytest.mark.gpu

CASES = [  # lengths (their mean makes 8 pieces of 512 tokens, float32 4), G, H, K, V, dtype, h0, packed
    ([4096], 1, 1, 128, 128, "bf16", True, False),
    ([4200], 1, 2, 64, 64, "bf16", False, False),
    ([9000, 0, 513, 3200, 1], 1, 1, 32, 16, "bf16", True, True),    # 5 sequences, some without a second piece
    ([1600, 1600], 1, 2, 64, 128, "f32", True, False),
    ([2049], 1, 1, 128, 48, "f32", True, False),
    ([4300, 0, 1024, 1025], 1, 2, 48, 80, "f32", True, True),
]


@pytest.fixture(scope="module")
def mssm():
    import selective_state_space_mssm_amd as m
    return m


def memory(mssm, t, **kw):
    return mssm.gdr_fwd_train(*args(t), t["h0"], offsets=t["offsets"], norm_qk=True, **kw)[2].numel()


@pytest.mark.parametrize("lengths,G,H,K,V,dtype,h0,packed", CASES)
def test_outputs_and_gradients(mssm, lengths, G, H, K, V, dtype, h0, packed):
    x = ref.inputs(lengths, G, H, K, V, dtype, seed=1, h0=h0, packed=packed)
    t = ref.on_gpu(x, dtype)
    chunks = -(-max(lengths) // 64)
    want_y, want_s, want = ref.gradients(x, norm=True)
    y, s, got = train(mssm, t)
    ref.check(y, want_y, dtype, chunks, "y")
    ref.check(s, want_s, "f32", chunks, "h_final")
    for n, w in want.items():
        ref.check(got[n], w, dtype if n in ("dq", "dk", "dv") else "f32", chunks, n, gradient=True)
    y2, s2 = mssm.gdr_fwd(*args(t), t["h0"], offsets=t["offsets"], norm_qk=True)
    again = mssm.gdr_bwd(*args(t), t["dy"], t["h0"], t["dh_final"], offsets=t["offsets"], norm_qk=True)
    assert torch.equal(y, y2) and torch.equal(s, s2) and all(torch.equal(got[n], again[n]) for n in GRADS if got[n] is not None)
    h = s.clone() if t["h0"] is None else t["h0"].clone()
    if t["h0"] is not None:  # the final state over the first
        mssm.gdr_fwd(*args(t), h, offsets=t["offsets"], norm_qk=True, h_final=h)
        assert torch.equal(h, s)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_strong_keys_and_full_decays_between_pieces(mssm, dtype):
    x = ref.inputs([4700], 1, 1, 64, 32, dtype, seed=2)
    x["g"][0, 511], x["g"][0, 512], x["g"][0, 1600] = float("-inf"), -200.0, -1e4
    x["g"][0, 2000:4000] = 0.0          # nothing decays over several pieces
    x["beta"][0, 2500:3300] = 0.0       # more than a piece that changes nothing
    x["k"][0, 1024:1536] = x["k"][0, 1024].clone()
    y, s = mssm.gdr_fwd(*args(ref.on_gpu(x, dtype)), x["h0"].float().cuda(), offsets=x["offsets"].cuda(), norm_qk=True)
    want_y, want_s = ref.forward(x, norm=True)
    ref.check(y, want_y, dtype, 74, "y")
    ref.check(s, want_s, "f32", 74, "h_final")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_tokens_of_no_sequence_and_offsets_that_are_none(mssm, dtype):
    x = ref.inputs([9000, 100], 1, 1, 64, 64, dtype, seed=3)
    x["offsets"] = torch.tensor([70, 8900, 8990], dtype=torch.int32)
    t = ref.on_gpu(x, dtype)
    inner = {n: v[:, 70:8990].contiguous() if n in ("q", "k", "v", "g", "beta", "dy") else v for n, v in t.items()}
    inner["offsets"] = t["offsets"] - 70
    for n in ("q", "k", "v", "g", "beta"):
        t[n][:, :70] = float("nan")
        t[n][:, 8990:] = float("nan")
    y = torch.full_like(t["v"], 7.0)
    y, s = mssm.gdr_fwd(*args(t), t["h0"], offsets=t["offsets"], norm_qk=True, y=y)
    want_y, want_s = ref.forward({n: v if v is None else v.cpu() if n == "offsets" else v.double().cpu() for n, v in inner.items()}, norm=True)
    ref.check(y[:, 70:8990], want_y, dtype, 140, "y")
    ref.check(s, want_s, "f32", 140, "h_final")
    assert torch.all(y[:, :70] == 7.0) and torch.all(y[:, 8990:] == 7.0)
    need, guard = memory(mssm, t), 65536
    for offsets in ([0, 2 ** 31 - 1, -9], [9100, 0, 9100], [-5, 9000, 3]):
        whole = torch.full((need + 2 * guard,), 3, dtype=torch.uint8, device="cuda")
        t["offsets"].copy_(torch.tensor(offsets, dtype=torch.int32))
        mssm.gdr_fwd_train(*args(t), t["h0"], offsets=t["offsets"], norm_qk=True, ctx=whole[guard:guard + need])
        torch.cuda.synchronize()
        assert torch.all(whole[:guard] == 3) and torch.all(whole[-guard:] == 3)


def test_a_spoilt_token_spoils_what_follows_it_only(mssm):
    t = ref.on_gpu(ref.inputs([5000, 4000], 1, 2, 64, 32, "bf16", seed=4), "bf16")
    y, s = mssm.gdr_fwd(*args(t), t["h0"], offsets=t["offsets"], norm_qk=True)
    t["v"][0, 1300, 0] = float("nan")
    y2, s2 = mssm.gdr_fwd(*args(t), t["h0"], offsets=t["offsets"], norm_qk=True)
    assert torch.equal(y2[:, :, 1], y[:, :, 1]) and torch.equal(s2[:, 1], s[:, 1])
    assert torch.equal(y2[:, :1280, 0], y[:, :1280, 0]) and torch.equal(y2[:, 5000:], y[:, 5000:]) and torch.equal(s2[1], s[1])
    assert torch.isnan(y2[0, 1536:5000, 0]).all() and torch.isnan(s2[0, 0]).all()


def test_replayed_and_on_two_streams(mssm):
    fresh = lambda i: ref.on_gpu(ref.inputs([4096], 1, 2, 64, 64, "bf16", seed=10 + i, packed=False), "bf16")  # noqa: E731
    held, out = fresh(0), {}
    ws = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")

    def work(t, m):
        return mssm.gdr_fwd(*args(t), t["h0"], norm_qk=True, workspace=m)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        work(held, ws)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = work(held, ws)
    for turn in range(3):
        new = fresh(1 + turn)
        for n, v in held.items():
            if v is not None:
                v.copy_(new[n])
        graph.replay()
        want = work(new, None)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for i, s in enumerate(streams):
        with torch.cuda.stream(s):
            out[i] = work(held, None)
    torch.cuda.synchronize()
    assert all(torch.equal(out[i][0], want[0]) and torch.equal(out[i][1], want[1]) for i in out)
