"""GPU tests of the gated delta rule with h_final over h0 where sequences are gone through in pieces: a last piece of
one token, sequences of one piece among longer ones, heads that lie on different XCDs, and another stream's work on the
card.  Outputs equal those with a buffer of its own, bit for bit."""
import pytest

torch = pytest.importorskip("torch")
import gdr_ref as ref  # noqa: E402
from test_gpu_gdr_edges import args  # noqa: E402

pytestmark = pytest.mark.gpu

CASES = [  # lengths (in pieces of 512 tokens or more), G, H, K, V, dtype
    ([4097], 1, 3, 64, 64, "bf16"),                # eight pieces and one token
    ([2049], 1, 3, 64, 32, "f32"),
    ([9000, 1, 0, 512, 513], 1, 1, 64, 80, "bf16"),
    ([6000, 64, 511, 2561], 1, 2, 128, 64, "f32"),
]


@pytest.fixture(scope="module")
def mssm():
    import selective_state_space_mssm_amd as m
    return m


@pytest.mark.parametrize("lengths,G,H,K,V,dtype", CASES)
@pytest.mark.parametrize("kind", ["gdr_fwd", "gdr_fwd_train"])
def test_final_over_initial_states(mssm, lengths, G, H, K, V, dtype, kind):
    x = ref.inputs(lengths, G, H, K, V, dtype, seed=5)
    t = ref.on_gpu(x, dtype)
    run = lambda h0, **kw: getattr(mssm, kind)(*args(t), h0, offsets=t["offsets"], norm_qk=True, **kw)[:2]  # noqa: E731
    chunks = -(-max(lengths) // 64)
    want_y, want_s = ref.forward(x, norm=True)
    y, s = run(t["h0"])
    ref.check(y, want_y, dtype, chunks, "y")
    ref.check(s, want_s, "f32", chunks, "h_final")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    busy = torch.randn((4096, 4096), device="cuda")
    for _ in range(3):
        h = t["h0"].clone()
        with torch.cuda.stream(side):  # compute units taken by other work, now here, now there
            for _ in range(2):
                busy = busy * 0.5 + 1.0
        y2, s2 = run(h, h_final=h)
        assert s2 is h and torch.equal(h, s) and torch.equal(y2, y)
    torch.cuda.synchronize()


def test_no_initial_states(mssm):
    t = ref.on_gpu(ref.inputs([4097, 300], 1, 2, 64, 64, "bf16", seed=6), "bf16")
    run = lambda h0: mssm.gdr_fwd(*args(t), h0, offsets=t["offsets"], norm_qk=True,  # noqa: E731
                                  workspace=torch.full((64 << 20,), 0xFF, dtype=torch.uint8, device="cuda"))
    none, zeros = run(None), run(torch.zeros_like(t["h0"]))
    assert torch.equal(none[0], zeros[0]) and torch.equal(none[1], zeros[1])
