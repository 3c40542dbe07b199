"""GPU test: a row's norm does not depend on its place in the batch.  Rows whose length is no whole number of vectors
start at eight different offsets from a vector boundary, and their elements then lie in other lanes; the sum of the
squares, in float64, rounds to the same float32 whatever its order (sums of at most 20,001 exact squares differ by
2^-38 at most, relative, so that one in 2^14 rows could differ at the worst, one in 2^29 at 9 elements)."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mssm():
    import selective_state_space_mssm_amd as m
    return m


@pytest.mark.parametrize("rows,dim", [(4000, 9), (600, 333), (300, 1537), (5000, 1537), (20, 20001)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_a_row_is_the_same_at_every_place(mssm, rows, dim, dtype):
    g = torch.Generator(device="cuda").manual_seed(dim)
    x = torch.randn((rows, dim), generator=g, device="cuda").to(dtype)
    w = torch.rand(dim, generator=g, device="cuda") + 0.5
    y, h = mssm.add_rmsnorm(x, w, x)
    q, s, _ = mssm.add_rmsnorm_q8(x, w, x)
    for shift in (1, 2, 3, 5, 7):  # 3 and the odd ones together reach all eight offsets
        moved = x.roll(shift, 0).contiguous()
        y2, h2 = mssm.add_rmsnorm(moved, w, moved)
        q2, s2, _ = mssm.add_rmsnorm_q8(moved, w, moved)
        assert torch.equal(y2.roll(-shift, 0), y) and torch.equal(h2.roll(-shift, 0), h) and torch.equal(s2.roll(-shift, 0), s)
        assert torch.equal(q2.view(torch.uint8).roll(-shift, 0), q.view(torch.uint8))
