"""GPU test of bfloat16 outputs of the low-rank adapters where what an adapter adds cancels: the inner sums stay
float32.  Rows, weights and all sums are whole numbers below 2^24, so float32 has every one of them exactly, in any
order, and y is their value rounded to bfloat16 once.  Inner sums have 17 to 22 bits, and those of a pair of the rank
differ by their last product only."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float8_e4m3fn])
@pytest.mark.parametrize("M,N,R,S", [(3, 40, 8, 2), (64, 300, 16, 64), (65, 64, 8, 3), (300, 333, 16, 7), (1000, 256, 33, 5), (2048, 70, 128, 2),
                                     (2049, 64, 8, 4), (2100, 100, 48, 3), (2500, 257, 100, 3)])
def test_sums_that_cancel(M, N, R, S, dtype):
    import selective_state_space_mssm_amd as mssm
    r = torch.Generator().manual_seed(M + R)
    n = lambda top, *s: torch.randint(-top, top + 1, s, generator=r).float()  # noqa: E731
    K, pairs = 256, min(2, R // 2)
    sign = torch.where(torch.rand(K, generator=r) < 0.5, -1.0, 1.0)  # of the rows and of the weights: no inner sum is small
    x = n(127 if dtype == torch.bfloat16 else 15, M, K).abs() * sign  # exact in the type
    a, b = torch.zeros((S, R, K)), torch.zeros((S, N, R))
    for i in range(S):
        for p, q in torch.randperm(R, generator=r)[:2 * pairs].view(pairs, 2).tolist():
            a[i, p] = n(127, K).abs() * sign
            a[i, q] = a[i, p]
            a[i, q, -1] = n(127, 1)
            w = n(1, N)
            b[i, :, p], b[i, :, q] = w, -w
    index = torch.randint(-1, S, (M,), generator=r).int()
    y0 = n(1, M, N)
    want = y0.double()
    for i in range(S):
        rows = (index == i).nonzero()[:, 0]
        want[rows] += (x[rows].double() @ a[i].double().T) @ b[i].double().T
    y = y0.bfloat16().cuda()
    scale = {"x_scale": torch.ones(M, device="cuda")} if dtype == torch.float8_e4m3fn else {}
    mssm.lora(x.to(dtype).cuda(), a.bfloat16().cuda(), b.bfloat16().cuda(), index.cuda(), y, **scale)
    assert torch.equal(y.cpu(), want.bfloat16())
