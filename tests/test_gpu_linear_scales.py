"""The scales of 8-bit operands are applied one after the other, as the formula
has them: their product alone may leave float32's range where the result does
not.  Within (K + 16) EPS32 of the float64 result, for all variants."""
import pytest

import block_ref as ref
import linear_plan

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
F8 = torch.float8_e4m3fn
SIZES = [(20, 1024, 300, "rows"), (9000, 512, 100, "columns"), (1000, 1024, 3000, "tile128"), (1000, 1024, 2999, "tile128"),
         (5054, 1232, 1585, "tile128"), (5054, 1232, 1584, "tile128")]


@pytest.fixture(scope="module")
def mssm():
    import selective_state_space_mssm_amd as m
    return m


@pytest.mark.parametrize("M,K,N,variant", SIZES)
@pytest.mark.parametrize("xs,ws", [(3e-33, 1.1e-12), (1.1e-12, 3e-33), (1e-30, 1e38), (3e-38, 2e36)])
def test_products_of_scales_out_of_range(mssm, M, K, N, variant, xs, ws):
    print(f"[linear scales] {M} x {K} x {N} {xs} {ws}", flush=True)
    if torch.cuda.get_device_properties(0).multi_processor_count == 256:
        assert linear_plan.plan(M, K, N, "f8", "f32")[0] == variant
    g = torch.Generator(device="cuda").manual_seed(M + N)
    x, w = ((torch.rand(s, generator=g, device="cuda") * 448).to(F8) for s in ((M, K), (N, K)))
    x[0] = 0
    xs, ws = torch.full((M,), xs, device="cuda"), torch.full((N,), ws, device="cuda")
    y = mssm.linear(x, w, x_scale=xs, w_scale=ws, out_dtype=torch.float32).double()
    want = (x.double() @ w.double().t().contiguous()) * xs.double()[:, None] * ws.double()
    assert want[1:].abs().min() > 2.0 ** -126 and want.abs().max() < 3e38
    assert torch.all((y - want).abs() <= (K + 16) * ref.EPS32 * want.abs())


def test_zero_sums_stay_zero(mssm):
    for M, N in ((3, 40), (9000, 100), (1000, 3000)):
        big = torch.full((max(M, N),), 1e25, device="cuda")
        y = mssm.linear(torch.zeros((M, 512), device="cuda").to(F8), torch.ones((N, 512), device="cuda").to(F8), x_scale=big[:M],
                        w_scale=big[:N], out_dtype=torch.float32)
        assert torch.all(y == 0)
