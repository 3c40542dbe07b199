"""CPU test: the forward calls of the gated delta rule record no gradient, and their docstrings say so and name the call
that computes it."""
import pytest

mssm = pytest.importorskip("selective_state_space_mssm_amd")


@pytest.mark.parametrize("name,by", [("gdr_fwd", "gdr_bwd"), ("gdr_fwd_train", "gdr_bwd_saved")])
def test_that_no_gradient_is_recorded_is_said(name, by):
    text = " ".join(getattr(mssm, name).__doc__.split())
    assert f"No gradient is recorded, also of tensors that require one: {by} computes them." in text
