"""Beam selection takes -0.0 and +0.0 for the equal values that they are: ties
between them go to the lowest k * vocab + v, in a beam's logits, among beams and
among finished beams' scores.  Tokens and parents are compared exactly with the
float64 definition (a stable sort, to which the zeros are equal)."""
import numpy as np
import pytest

import block_ref as ref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def mssm():
    import selective_state_space_mssm_amd as m
    return m


def select(mssm, x, s, finished=None, end=None):
    print(f"[beam zeros] {tuple(x.shape)} {x.dtype}", flush=True)
    want = ref.beam(x.double().numpy(), s.double().numpy(), None if finished is None else finished.numpy(), end)
    out = mssm.beam_select(x.cuda(), s.cuda(), None if finished is None else finished.cuda(), end)
    assert np.array_equal(out[1].cpu().numpy(), want[1]) and np.array_equal(out[2].cpu().numpy(), want[2])
    assert np.all(np.abs(out[0].double().cpu().numpy() - want[0]) <= 2e-5)
    return out


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_two_tokens(mssm, dtype):
    _, _, t, _ = select(mssm, torch.tensor([[[-0.0, 0.0]]]).to(DT[dtype]), torch.zeros((1, 1)))
    assert t.item() == 0
    _, _, t, _ = select(mssm, torch.tensor([[[0.0, -0.0]]]).to(DT[dtype]), torch.zeros((1, 1)))
    assert t.item() == 0


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,K,V", [(2, 4, 100), (1, 16, 5001), (64, 8, 8200), (64, 8, 8201)])
def test_logits_under_a_mask(mssm, B, K, V, dtype):
    # what a 0/1 mask leaves of negative logits are -0.0, of others +0.0; they are the largest here
    g = torch.Generator().manual_seed(V)
    x = torch.where(torch.rand((B, K, V), generator=g) < 0.5, -0.0, 0.0)
    x[torch.rand((B, K, V), generator=g) < 0.9] = -3.0
    _, p, t, _ = select(mssm, x.to(DT[dtype]), torch.zeros((B, K)))
    x[:] = -0.0  # all equal, the first token of the other sign and the last
    x[:, :, 0] = x[:, :, V - 1] = 0.0
    select(mssm, x.to(DT[dtype]), torch.zeros((B, K)))


def test_finished_beams_with_scores_of_either_sign(mssm):
    x = torch.zeros((2, 4, 50))
    s = torch.tensor([[-0.0, 0.0, -0.0, 0.0], [0.0, -0.0, 0.0, -0.0]])
    _, p, t, f = select(mssm, x, s, torch.ones((2, 4), dtype=torch.bool), 7)
    assert p.cpu().tolist() == [[0, 1, 2, 3]] * 2 and torch.all(t == 7) and torch.all(f)
