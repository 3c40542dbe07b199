"""Products at the largest row and column counts that the problem accepts: more
tiles than one row of a launch's workgroups holds."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mssm():
    import selective_state_space_mssm_amd as m
    return m


@pytest.mark.parametrize("rows,columns", [(2 ** 31 - 1, 1), (1, 2 ** 31 - 1)])
def test_the_most_rows_and_columns(mssm, rows, columns):
    print(f"[linear] {rows} x 1 x {columns}", flush=True)
    many = torch.empty((max(rows, columns), 1), dtype=torch.bfloat16, device="cuda")
    many.random_(-8, 9)
    one = torch.full((1, 1), 2.0, dtype=torch.bfloat16, device="cuda")
    y = mssm.linear(many if rows > 1 else one, one if rows > 1 else many)
    assert y.shape == (rows, columns)
    y, many = y.view(-1), many.view(-1)
    step = 1 << 28
    for i in range(0, many.numel(), step):
        assert torch.equal(y[i:i + step], many[i:i + step] * 2)
