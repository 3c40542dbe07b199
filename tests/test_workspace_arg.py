"""CPU tests of the binding's check of a caller's workspace: it has to be memory
of the device that the kernels run on, and as long as its elements say."""
import pytest

torch = pytest.importorskip("torch")
binding = pytest.importorskip("selective_state_space_mssm_amd").binding


def test_workspace_of_another_device_is_refused():
    host = torch.empty(64, dtype=torch.uint8)
    with pytest.raises(ValueError, match="workspace is on cpu"):
        binding._workspace(64, torch.device("cuda", 0), host)
    with pytest.raises(ValueError, match="workspace is on cpu"):  # nothing may be written beyond, wherever it lies
        binding._workspace(64, torch.device("meta"), host)


def test_workspace_with_fewer_bytes_than_elements_is_refused():
    # 64 elements, one byte of memory
    with pytest.raises(ValueError, match="contiguous"):
        binding._workspace(64, torch.device("cpu"), torch.empty(1, dtype=torch.uint8).expand(64))


def test_workspace_that_fits_is_taken():
    ws = torch.empty(64, dtype=torch.uint8)
    assert binding._workspace(64, torch.device("cpu"), ws) is ws
    assert binding._workspace(0, torch.device("cpu"), ws) is None
    with pytest.raises(ValueError, match="needs 65"):
        binding._workspace(65, torch.device("cpu"), ws)
    assert binding._workspace(32, torch.device("cpu")).numel() == 32
