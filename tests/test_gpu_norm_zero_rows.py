"""Rows of zeros through the 8-bit norm: q = 0 and the scale 1e-30 / 448 for
every eps that is accepted, 0 too, where the row's 1 / sqrt(mean + eps) is
infinite.  The other rows of the call are as without it."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def mssm():
    import selective_state_space_mssm_amd as m
    return m


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,dim", [(3, 1), (3, 100), (3, 2560), (3, 1537), (3, 20001), (4099, 100), (4099, 2049)])
@pytest.mark.parametrize("eps", [0.0, 1e-5])
def test_zero_rows(mssm, eps, rows, dim, dtype):
    print(f"[norm zeros] {rows} x {dim} {dtype} eps {eps}", flush=True)
    g = torch.Generator().manual_seed(dim)
    x = torch.randn((rows, dim), generator=g).to(DT[dtype])
    x[x == 0] = 1.0
    res = torch.randn((rows, dim), generator=g)
    zero = torch.zeros(rows, dtype=torch.bool)
    zero[0], zero[rows - 1] = True, True
    x[0], res[0] = 0, 0
    res[rows - 1] = -x[rows - 1].float()  # the sum is zero
    w = 1 + 0.2 * torch.randn(dim, generator=g)
    q, scale, h = mssm.add_rmsnorm_q8(x.cuda(), w.cuda(), res.cuda(), eps=eps)
    assert torch.all(h.cpu()[zero] == 0) and torch.all(q.float().cpu()[zero] == 0)
    assert torch.all(scale.cpu()[zero] == float(np.float32(1e-30) / np.float32(448)))
    # the other rows, at their places (a sum's order goes by the place), are those of a call without zero rows
    x[zero] = 1.0
    q2, scale2, _ = mssm.add_rmsnorm_q8(x.cuda(), w.cuda(), res.cuda(), eps=eps)
    keep = ~zero
    assert torch.isfinite(q2.float()).all()
    assert torch.equal(q.cpu()[keep].view(torch.uint8), q2.cpu()[keep].view(torch.uint8)) and torch.equal(scale.cpu()[keep], scale2.cpu()[keep])


def test_a_weight_of_zeros(mssm):
    q, scale, _ = mssm.add_rmsnorm_q8(torch.randn((5, 300), device="cuda"), torch.zeros(300, device="cuda"), eps=0.0)
    assert torch.all(q.float() == 0) and torch.all(scale == float(np.float32(1e-30) / np.float32(448)))
