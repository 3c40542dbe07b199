"""The operators around the scan and the devices of their tensors: all have to be
on the first one's, and the call runs there whatever device is current.  One GPU
stands in for two: a tensor that says it is on the next one, and a binding that is
told that the next one is current."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mssm():
    import selective_state_space_mssm_amd as m
    return m


class Elsewhere(torch.Tensor):
    def get_device(self):
        return 1


def elsewhere(*args, **kw):
    return torch.ones(*args, device="cuda", **kw).as_subclass(Elsewhere)


def here(*args, **kw):
    return torch.ones(*args, device="cuda", **kw)


def test_tensors_of_two_devices_are_refused(mssm):
    f8 = lambda t: t.to(torch.float8_e4m3fn)  # noqa: E731
    x, w = here(2, 8), here(8)
    calls = [
        ("weight", lambda: mssm.add_rmsnorm(x, elsewhere(8))),
        ("residual", lambda: mssm.add_rmsnorm(x, w, elsewhere(2, 8))),
        ("residual_out", lambda: mssm.add_rmsnorm(x, w, x, residual_out=elsewhere(2, 8))),
        ("y", lambda: mssm.add_rmsnorm(x, w, y=elsewhere(2, 8))),
        ("scale", lambda: mssm.add_rmsnorm_q8(x, w, scale=elsewhere(2))),
        ("w", lambda: mssm.linear(x, elsewhere(4, 8))),
        ("bias", lambda: mssm.linear(x, here(4, 8), elsewhere(4))),
        ("residual", lambda: mssm.linear(x, here(4, 8), None, elsewhere(2, 4))),
        ("w_scale", lambda: mssm.linear(f8(x), f8(here(4, 8)), x_scale=here(2), w_scale=elsewhere(4))),
        ("scores", lambda: mssm.beam_select(here(1, 2, 5), elsewhere(1, 2))),
        ("parent", lambda: mssm.beam_select(here(1, 2, 5), here(1, 2), parent=elsewhere(1, 2, dtype=torch.int32))),
        (r"states\[0\]", lambda: mssm.beam_reorder(here(1, 2, dtype=torch.int32), elsewhere(1, 2, 4))),
    ]
    for name, call in calls:
        with pytest.raises(ValueError, match=f"^{name} is on"):
            call()


def test_runs_on_the_tensors_device(mssm, monkeypatch):
    from selective_state_space_mssm_amd import block
    x, w = torch.randn(300, 64, device="cuda"), torch.randn(50, 64, device="cuda")
    logits, scores = torch.randn(2, 3, 40, device="cuda"), torch.zeros(2, 3, device="cuda")

    def once():
        state = torch.arange(6.0, device="cuda").view(1, 6, 1).clone()
        s, p, t, _ = mssm.beam_select(logits, scores)
        mssm.beam_reorder(p, state)
        return [mssm.add_rmsnorm(x, here(64))[0], *mssm.add_rmsnorm_q8(x, here(64))[:2], mssm.linear(x, w), s, p, t, state]

    want = once()
    entered = []

    class Device(torch.cuda.device):
        def __enter__(self):
            entered.append(self.idx)
            monkeypatch.setattr(block, "_current_device", lambda: 0)
            return super().__enter__()

        def __exit__(self, *a):
            monkeypatch.setattr(block, "_current_device", lambda: 1)
            return super().__exit__(*a)

    monkeypatch.setattr(torch.cuda, "device", Device)
    monkeypatch.setattr(block, "_current_device", lambda: 1)
    got = once()
    assert entered == [0] * 5
    for a, b in zip(want, got):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
