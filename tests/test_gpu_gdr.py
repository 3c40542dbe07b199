"""GPU tests of the gated delta rule over whole sequences and of its gradients,
against the recurrence in 64 bits (gdr_ref.py has it, and the bounds)."""
import pytest

torch = pytest.importorskip("torch")
import gdr_ref as ref  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mssm():
    import selective_state_space_mssm_amd as m
    return m


def chunks_of(lengths):
    return max(1, max(-(-n // 64) for n in lengths))


CASES = [
    # lengths, G, H, K, V, dtype, h0, packed
    ([64], 1, 1, 64, 64, "f32", False, False),
    ([64], 1, 1, 128, 128, "bf16", False, False),
    ([1], 1, 1, 16, 16, "f32", True, False),
    ([1, 1, 1], 2, 4, 128, 128, "bf16", True, False),
    ([63, 63], 1, 2, 64, 64, "f32", True, False),
    ([65], 2, 2, 128, 128, "f32", True, False),
    ([130, 130], 1, 3, 48, 80, "f32", True, False),
    ([200], 2, 4, 112, 144, "bf16", True, False),
    ([5, 0, 64, 1, 129, 0], 2, 4, 64, 64, "f32", True, True),
    ([7, 64, 100], 1, 4, 128, 128, "bf16", False, True),
    ([33, 0, 1, 191], 3, 3, 96, 32, "bf16", True, True),
    ([128] * 3, 1, 48, 32, 96, "bf16", True, False),   # enough sequences and heads for the wide tiles
    ([70, 3] * 3, 1, 32, 80, 112, "bf16", True, True),
    ([70, 3] * 3, 1, 32, 64, 112, "f32", True, True),
    ([20, 90], 1, 1, 16, 512, "bf16", True, True),
]


@pytest.mark.parametrize("lengths,G,H,K,V,dtype,h0,packed", CASES)
@pytest.mark.parametrize("norm", [True, False])
def test_forward(mssm, lengths, G, H, K, V, dtype, h0, packed, norm):
    x = ref.inputs(lengths, G, H, K, V, dtype, seed=1, h0=h0, unit=not norm, packed=packed)
    t = ref.on_gpu(x, dtype)
    want_y, want_s = ref.forward(x, norm=norm)
    y, s = mssm.gdr_fwd(t["q"], t["k"], t["v"], t["g"], t["beta"], t["h0"], offsets=t["offsets"], norm_qk=norm)
    ref.check(y, want_y, dtype, chunks_of(lengths), "y")
    ref.check(s, want_s, "f32", chunks_of(lengths), "h_final")


@pytest.mark.parametrize("lengths,G,H,K,V,dtype,h0,packed", CASES)
@pytest.mark.parametrize("norm", [True, False])
def test_gradients(mssm, lengths, G, H, K, V, dtype, h0, packed, norm):
    x = ref.inputs(lengths, G, H, K, V, dtype, seed=2, h0=h0, unit=not norm, packed=packed)
    t = ref.on_gpu(x, dtype)
    want_y, want_s, want = ref.gradients(x, norm=norm)
    args = (t["q"], t["k"], t["v"], t["g"], t["beta"])
    y, s, ctx = mssm.gdr_fwd_train(*args, t["h0"], offsets=t["offsets"], norm_qk=norm)
    plain = mssm.gdr_fwd(*args, t["h0"], offsets=t["offsets"], norm_qk=norm)
    assert torch.equal(y, plain[0]) and torch.equal(s, plain[1])
    got = mssm.gdr_bwd_saved(*args, t["dy"], ctx, t["dh_final"], offsets=t["offsets"], norm_qk=norm)
    again = mssm.gdr_bwd(*args, t["dy"], t["h0"], t["dh_final"], offsets=t["offsets"], norm_qk=norm)
    for name, w in want.items():
        kind = dtype if name in ("dq", "dk", "dv") else "f32"
        ref.check(got[name], w, kind, chunks_of(lengths), name, gradient=True)
        assert torch.equal(got[name], again[name]), name
