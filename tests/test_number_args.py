"""Numbers that a call takes (a scale, an eps, an end token) count by their value at the call, also where they come as a
tensor of one number that is changed in place between calls: what the bindings remember by them must not outlast it."""
import pytest

torch = pytest.importorskip("torch")
mssm = pytest.importorskip("selective_state_space_mssm_amd")


def test_a_scale_that_changes():
    scale = torch.tensor(0.5)
    sizes = (64, 1, 1, 1, 16, 16, 0, 0)
    assert mssm.gdr._problem(*sizes, scale, None)[2].scale == 0.5
    scale.mul_(4)
    assert mssm.gdr._problem(*sizes, scale, None)[2].scale == 2.0
    assert mssm.gdr._problem(*sizes, None, None)[2].scale == 0.25


@pytest.mark.gpu
def test_calls_with_numbers_that_change():
    g = torch.Generator().manual_seed(0)
    n = lambda *s: torch.randn(s, generator=g).cuda()  # noqa: E731
    q, v, gate = n(1, 70, 2, 32), n(1, 70, 2, 16), -torch.rand((1, 70, 2), generator=g).cuda()
    x, w, logits, scores = n(3, 40), n(40), n(2, 3, 50), n(2, 3)
    number, done = torch.tensor(0.25), torch.ones((2, 3), dtype=torch.bool).cuda()
    end = torch.tensor(7)
    for _ in range(2):
        s, e = float(number), int(end)
        for a, b in ((mssm.gdr_fwd(q, q, v, gate, gate.abs(), scale=number, norm_qk=True), mssm.gdr_fwd(q, q, v, gate, gate.abs(), scale=s, norm_qk=True)),
                     (mssm.add_rmsnorm(x, w, x, eps=number), mssm.add_rmsnorm(x, w, x, eps=s)),
                     (mssm.beam_select(logits, scores, done, end_token=end), mssm.beam_select(logits, scores, done, end_token=e))):
            assert all(torch.equal(i, j) for i, j in zip(a, b))
        assert bool((mssm.beam_select(logits, scores, done, end_token=end)[2] == e).all())  # finished beams take it
        number.mul_(16)
        end.add_(5)
