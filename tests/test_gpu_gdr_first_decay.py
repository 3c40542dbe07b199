"""GPU tests of the gradient of log decays where it is exactly zero: nothing passes the first token of a sequence without
an initial state, so its decay changes nothing, whatever the tokens behind it do.  Of sequences of one token that is all
of dg."""
import pytest

torch = pytest.importorskip("torch")
import gdr_ref as ref  # noqa: E402
from test_gpu_gdr_edges import args  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mssm():
    import selective_state_space_mssm_amd as m
    return m


@pytest.mark.parametrize("lengths,G,H,K,V,packed", [
    ([1, 1], 1, 1, 64, 96, False), ([1] * 40, 2, 4, 128, 128, False), ([1, 0, 1, 1], 1, 3, 16, 16, True), ([1, 2, 1], 1, 2, 48, 80, True),
    ([33, 64, 65, 1, 200], 2, 4, 64, 64, True), ([130, 130], 1, 2, 128, 64, False)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("norm", [True, False])
def test_nothing_passes_the_first_token(mssm, lengths, G, H, K, V, packed, dtype, norm):
    x = ref.inputs(lengths, G, H, K, V, dtype, seed=7, h0=False, unit=not norm, packed=packed)
    t = ref.on_gpu(x, dtype)
    kw = dict(offsets=t["offsets"], norm_qk=norm)
    _, _, want = ref.gradients(x, norm=norm)
    got = mssm.gdr_bwd(*args(t), t["dy"], None, t["dh_final"], **kw)
    starts = [sum(lengths[:i]) for i, n in enumerate(lengths) if n]
    assert float(want["dg"].reshape(-1, H)[starts].abs().max()) == 0.0
    assert float(got["dg"].reshape(-1, H)[starts].abs().max()) == 0.0
    ref.check(got["dg"], want["dg"], "f32", -(-max(lengths) // 64), "dg", gradient=True)
    # a gradient of zero goes in: of the state behind (and of y) nothing comes back
    zero = mssm.gdr_bwd(*args(t), torch.zeros_like(t["dy"]), None, None, **kw)
    if packed is False:
        assert all(float(zero[n].abs().max()) == 0.0 for n in ("dq", "dk", "dv", "dg", "dbeta", "dh0"))
