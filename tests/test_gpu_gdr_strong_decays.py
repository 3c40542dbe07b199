"""GPU tests of the gradient of log decays where all decays are strong: what passes a token is small then, and so is dg;
what does not (a token with itself, the last write) is of ordinary size and must not leave its roundings there.  The
bound is that of any gradient, a multiple of 2^-24 of the largest value of the output, which is 10^-3 to 10^-6 here."""
import pytest

torch = pytest.importorskip("torch")
import gdr_ref as ref  # noqa: E402
from test_gpu_gdr_edges import args  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lengths,G,H,K,V,h0,dh_final,packed", [
    ([2, 2], 1, 1, 64, 64, False, False, False), ([5], 1, 2, 16, 16, False, True, False), ([70, 70], 1, 2, 64, 64, False, True, False),
    ([40], 2, 4, 128, 128, True, True, False), ([200, 3, 64], 1, 2, 128, 48, True, False, True), ([33, 0, 130], 2, 2, 48, 80, False, True, True)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("least,most", [(-9.0, -7.0), (-14.0, -12.0)])
def test_dg_is_as_exact_as_it_is_small(lengths, G, H, K, V, h0, dh_final, packed, dtype, least, most):
    import selective_state_space_mssm_amd as mssm
    x = ref.inputs(lengths, G, H, K, V, dtype, seed=8, h0=h0, packed=packed)
    x["g"] = (most + (least - most) * torch.rand(x["g"].shape, generator=torch.Generator().manual_seed(9))).double()
    t = ref.on_gpu(x, dtype)
    _, _, want = ref.gradients(x, norm=True, dh_final=dh_final)
    got = mssm.gdr_bwd(*args(t), t["dy"], t["h0"], t["dh_final"] if dh_final else None, offsets=t["offsets"], norm_qk=True)
    chunks = -(-max(lengths) // 64)
    ref.check(got["dg"], want["dg"], "f32", chunks, "dg", gradient=True)
    for n in ("dq", "dk", "dv", "dbeta"):
        ref.check(got[n], want[n], "f32" if n == "dbeta" else dtype, chunks, n, gradient=True)
