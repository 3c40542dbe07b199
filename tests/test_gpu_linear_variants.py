"""Every variant of the projections (csrc/linear_plan.h) with its whole epilogue,
against float64: whole and cut tiles of both sizes, ragged in rows and columns,
outputs that start on 16-byte boundaries and off them, all column counts of the
few-columns kernel.  Each size is checked to take the variant that it is here
for (on the 256 compute units that the rule is tested with).

Tolerances.  A float32 sum of K terms in any order is within K EPS32 of the sum
of magnitudes; scales, bias, activation (slopes below 1.13) and residual add 16
EPS32 of it; an 8-bit sum for a bfloat16 output may lose 2^-10 of it as well; a
bfloat16 output adds its half ulp."""
import pytest

import block_ref as ref
import linear_plan

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f8": torch.float8_e4m3fn}
ACTIVATIONS = ["none", "relu", "silu", "gelu"]
# dtype, output, rows, in_dim, out_dim, variant, whole tiles?, cut tiles?
TILES = [
    ("f32", "f32", 390, 28, 5981, "tile128", 1, 0), ("f32", "f32", 1147, 6768, 49, "tile128", 0, 1),
    ("f32", "f32", 1298, 228, 5947, "tile128", 1, 1), ("f32", "f32", 325, 25, 8031, "tile128", 1, 0),
    ("f32", "f32", 4655, 229, 1836, "tile128", 1, 1), ("f32", "f32", 130, 1416, 7136, "tile256", 0, 1),
    ("f32", "f32", 3779, 996, 5503, "tile256", 1, 1),
    ("bf16", "bf16", 73, 64, 7955, "tile128", 1, 0), ("bf16", "bf16", 4258, 2584, 33, "tile128", 0, 1),
    ("bf16", "bf16", 3045, 600, 5493, "tile128", 1, 1), ("bf16", "bf16", 7492, 46, 178, "tile128", 1, 0),
    ("bf16", "bf16", 1795, 449, 4605, "tile128", 1, 1), ("bf16", "bf16", 5553, 32, 1427, "tile256", 1, 0),
    ("bf16", "bf16", 130, 8464, 2291, "tile256", 0, 1), ("bf16", "bf16", 2554, 792, 6635, "tile256", 1, 1),
    ("bf16", "f32", 5325, 56, 132, "tile128", 1, 0), ("bf16", "f32", 3004, 3544, 33, "tile128", 0, 1),
    ("bf16", "f32", 143, 53, 8079, "tile128", 1, 0), ("bf16", "f32", 3338, 453, 2486, "tile128", 1, 1),
    ("bf16", "f32", 6536, 32, 1163, "tile256", 1, 0), ("bf16", "f32", 129, 3936, 6297, "tile256", 0, 1),
    ("bf16", "f32", 4770, 808, 3474, "tile256", 1, 1),
    ("f8", "bf16", 88, 128, 7014, "tile128", 1, 0), ("f8", "bf16", 1306, 15840, 33, "tile128", 0, 1),
    ("f8", "bf16", 4612, 2608, 1748, "tile128", 1, 1), ("f8", "bf16", 8090, 117, 130, "tile128", 1, 0),
    ("f8", "bf16", 5943, 906, 1384, "tile128", 1, 1), ("f8", "bf16", 5481, 64, 1424, "tile256", 1, 0),
    ("f8", "bf16", 129, 20240, 2273, "tile256", 0, 1), ("f8", "bf16", 6621, 1424, 2433, "tile256", 1, 1),
    ("f8", "f32", 74, 128, 7915, "tile128", 1, 0), ("f8", "f32", 65, 20448, 593, "tile128", 0, 1),
    ("f8", "f32", 150, 117, 7049, "tile128", 1, 0), ("f8", "f32", 1167, 989, 6596, "tile128", 1, 1),
]
PAIRS = [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32"), ("f8", "bf16"), ("f8", "f32")]


@pytest.fixture(scope="module")
def mssm():
    import selective_state_space_mssm_amd as m
    return m


def plan(M, K, N, dtype, out):
    if torch.cuda.get_device_properties(0).multi_processor_count != 256:
        pytest.skip("the sizes are chosen for 256 compute units")
    return linear_plan.plan(M, K, N, dtype, out)


def activated(v, name):
    if name == "relu":
        return v.clamp(min=0.0)
    if name == "silu":
        return v * torch.sigmoid(v)
    if name == "gelu":
        return 0.5 * v * torch.special.erfc(-v / 2.0 ** 0.5)
    return v


def check(mssm, M, K, N, dtype, out, activation, bias=True, residual=True):
    print(f"[linear] {M} x {K} x {N} {dtype} -> {out} {activation} bias {bias} residual {residual}", flush=True)
    g = torch.Generator(device="cuda").manual_seed(M * 7 + K * 3 + N)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    x, w = rnd(M, K).to(DT[dtype]), (rnd(N, K) * (4 if dtype == "f8" else K ** -0.5)).to(DT[dtype])
    b = rnd(N) if bias else None
    r = rnd(M, N).to(DT[out]) if residual else None
    xs = ws = None
    if dtype == "f8":
        xs, ws = (0.5 + rnd(M).abs()) * K ** -0.5, 0.1 + 0.1 * rnd(N).abs()
    y = mssm.linear(x, w, b, r, activation, xs, ws, DT[out])
    assert y.dtype == DT[out] and y.shape == (M, N)
    want, mag = x.double() @ w.double().t().contiguous(), x.double().abs() @ w.double().abs().t().contiguous()
    if xs is not None:
        scale = xs.double()[:, None] * ws.double()
        want, mag = want * scale, mag * scale
    lost = 2.0 ** -10 * mag if (dtype, out) == ("f8", "bf16") else 0.0
    if b is not None:
        want, mag = want + b.double(), mag + b.double().abs()
    want = activated(want, activation)
    tol = 1.13 * ((K + 16) * ref.EPS32 * mag + lost) + 2 * ref.EPS32 * want.abs() + 1e-38
    if r is not None:
        want, tol = want + r.double(), tol + ref.EPS32 * r.double().abs()
    if out == "bf16":
        tol = tol * (1 + ref.EPSB) + ref.EPSB * want.abs()
    else:
        tol = tol + ref.EPS32 * want.abs()
    err = (y.double() - want).abs()
    bad = (~(err <= tol)).nonzero()
    assert bad.numel() == 0, f"{bad.shape[0]} of {M * N} off, first at {bad[0].tolist()}"


@pytest.mark.parametrize("dtype,out,M,K,N,variant,whole,cut", TILES)
@pytest.mark.parametrize("columns", ["as they are", "whole vectors"])
def test_tiles(mssm, dtype, out, M, K, N, variant, whole, cut, columns):
    if columns == "whole vectors":
        N = (N + 7) // 8 * 8
    p = plan(M, K, N, dtype, out)
    assert (p[0], p[1] > 0, p[2] > 0 and p[3] > 1) == (variant, bool(whole), bool(cut))
    for activation in ACTIVATIONS:
        check(mssm, M, K, N, dtype, out, activation)
    check(mssm, M, K, N, dtype, out, "none", bias=False, residual=False)


@pytest.mark.parametrize("dtype,out", PAIRS)
@pytest.mark.parametrize("N", [5, 16, 23, 40, 57, 72, 88, 96, 97, 128])
def test_columns(mssm, N, dtype, out):
    for M, row_bytes in ((9001, 448), (16100, 1040)):
        K = row_bytes // {"f32": 4, "bf16": 2, "f8": 1}[dtype]
        assert plan(M, K, N, dtype, out)[0] == "columns"
        for activation in ACTIVATIONS:
            check(mssm, M, K, N, dtype, out, activation)
        check(mssm, M, K, N, dtype, out, "none", bias=False, residual=False)


@pytest.mark.parametrize("dtype,out", PAIRS)
def test_residual_in_place_behind_cut_tiles(mssm, dtype, out):
    M, K, N = {"f32": (1298, 228, 5947), "bf16": (3045, 600, 5493), "f8": (4612, 2608, 1748)}[dtype]
    if (dtype, out) == ("f8", "f32"):
        M, K, N = 5054, 1232, 1585
    p = plan(M, K, N, dtype, out)
    assert p[1] > 0 and p[2] > 0
    g = torch.Generator(device="cuda").manual_seed(5)
    x, w = (torch.randn(s, generator=g, device="cuda").to(DT[dtype]) for s in ((M, K), (N, K)))
    r = torch.randn((M, N), generator=g, device="cuda").to(DT[out])
    kw = {"x_scale": torch.ones(M, device="cuda"), "w_scale": torch.ones(N, device="cuda")} if dtype == "f8" else {}
    y = mssm.linear(x, w, None, r, out_dtype=DT[out], **kw)
    r2 = r.clone()
    mssm.linear(x, w, None, r2, out_dtype=DT[out], y=r2, **kw)
    assert torch.equal(r2, y)
