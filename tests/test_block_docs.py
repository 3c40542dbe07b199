"""CPU test: the operators around the scan have no backward, and their
docstrings say so."""
import pytest

mssm = pytest.importorskip("selective_state_space_mssm_amd")


@pytest.mark.parametrize("name", ["add_rmsnorm", "add_rmsnorm_q8", "linear", "beam_select", "beam_reorder"])
def test_forward_only_is_said(name):
    assert "Forward only: no gradient is recorded." in " ".join(getattr(mssm, name).__doc__.split())
