"""The norm's kernels that small row counts do not reach: one wave a row (4,096
rows or more) at every number of vectors a lane, widths on and off a vector
boundary; four waves a row at every number of vectors.  Tolerances are those of
test_gpu_norm.py."""
import pytest

from test_gpu_norm import check, inputs, test_eight_bit_values_are_the_nearest as nearest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mssm():
    import selective_state_space_mssm_amd as m
    return m


@pytest.mark.parametrize("dtype,residual", [("bf16", "f32"), ("f32", "bf16"), ("f32", None), ("bf16", "bf16")])
@pytest.mark.parametrize("dim", [24, 505, 777, 1024, 1025, 1535, 1536, 1537, 2040, 2049, 2553, 2554, 2560])
def test_one_wave_a_row(mssm, dim, dtype, residual):
    check(mssm, *inputs(4099, dim, dtype, residual))


@pytest.mark.parametrize("dtype,residual", [("bf16", "f32"), ("f32", "bf16"), ("f32", None)])
@pytest.mark.parametrize("dim", [2561, 4089, 6137, 6144, 6145, 7000, 8177, 8184, 8192, 8193, 16377, 16378, 16383])
def test_four_waves_a_row(mssm, dim, dtype, residual):
    check(mssm, *inputs(5, dim, dtype, residual))


@pytest.mark.parametrize("rows", [4099])
@pytest.mark.parametrize("dim", [777, 1537, 2040, 2049, 2560])
@pytest.mark.parametrize("dtype,residual", [("bf16", "f32"), ("f32", "bf16"), ("bf16", None)])
def test_eight_bit_values_of_many_rows(mssm, rows, dim, dtype, residual, monkeypatch):
    import test_gpu_norm as base
    monkeypatch.setattr(base, "inputs", lambda _, d, *a, **k: inputs(rows, d, *a, **k))
    nearest(mssm, dim, dtype, residual)
