"""SiLU of the projections' epilogue in float32 outputs, value by value: within
8 units of 2^-23 relative of v / (1 + exp(-v)) wherever that is a normal float32
(exp2 and the reciprocal 1 unit each, the exponent's remainder carried, the
sum and two products half a unit each: below 5), on every variant's epilogue."""
import numpy as np
import pytest

import linear_plan

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f8": torch.float8_e4m3fn}


@pytest.fixture(scope="module")
def mssm():
    import selective_state_space_mssm_amd as m
    return m


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f8"])
@pytest.mark.parametrize("M,row_bytes,N,path,splits", [(20000, 64, 100, "columns", 1), (30, 68, 40, "rows", 1),
                                                       (2500, 256, 4000, "tile", 1), (2500, 1028, 4001, "tile", 1),
                                                       (700, 4096, 1300, "tile", 4)])
def test_relative_error(mssm, M, row_bytes, N, path, splits, dtype):
    K = row_bytes // {"f32": 4, "bf16": 2, "f8": 1}[dtype]
    print(f"[linear silu] {M} x {K} x {N} {dtype}", flush=True)
    if torch.cuda.get_device_properties(0).multi_processor_count == 256:
        plan = linear_plan.plan(M, K, N, dtype, "f32")
        assert plan[0].startswith(path) and (splits == 1 or plan[3] > 1)
    # one term a sum, so that the activation's argument is exact: x[m, 0] * w[n, 0] + bias[n]
    x, w = torch.zeros((M, K)), torch.zeros((N, K))
    x[:, 0], w[:, 0] = 0.0, 1.0
    v = torch.linspace(-85.0, 85.0, N) + torch.rand(N, generator=torch.Generator().manual_seed(N)) * 0.01
    kw = {"x_scale": torch.ones(M, device="cuda"), "w_scale": torch.ones(N, device="cuda")} if dtype == "f8" else {}
    y = mssm.linear(x.to(DT[dtype]).cuda(), w.to(DT[dtype]).cuda(), v.cuda(), activation="silu", out_dtype=torch.float32, **kw)
    e = np.exp(-v.double().numpy())
    want = v.double().numpy() / (1 + e)
    err = (np.abs(y.double().cpu().numpy() - want) / np.abs(want)).max()
    assert err <= 8 * 2.0 ** -23, err


def test_infinities(mssm):
    b = torch.tensor([float("inf"), -float("inf"), float("nan"), 200.0, -200.0, 0.0])
    y = mssm.linear(torch.zeros((1, 4), device="cuda"), torch.zeros((6, 4), device="cuda"), b.cuda(), activation="silu")[0].cpu()
    assert y[0] == float("inf") and torch.isnan(y[1:3]).all() and y[3] == 200 and y[4] == 0 and y[5] == 0
