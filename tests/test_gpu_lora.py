"""GPU tests of the low-rank adapters against the same sums in 64 bits.

Bound of an output: the inner sum of K products is float32 (K <= 1537 here:
random rounding errors of 2^-24 of up to sqrt(K) sums, four standard deviations,
of the root mean square magnitude of its terms; 2 sqrt(K) 2^-24 of the sum of
magnitudes covers it), and so is the outer one of R; with bfloat16 outputs the
inner values are two bfloat16 planes cut off, 2^-15 of themselves.  The sum with
y is rounded once to y's type."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "fp8": torch.float8_e4m3fn}
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}


@pytest.fixture(scope="module")
def mssm():
    import selective_state_space_mssm_amd as m
    return m


def make(M, K, N, R, S, dtype, out, order, seed=0):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    x, xs = n(M, K), None
    if dtype == "fp8":
        xs = x.abs().amax(1) / 448.0
        x = x / xs[:, None]
    w = torch.float32 if dtype == "f32" else torch.bfloat16
    if order == "any":
        index = torch.randint(-2, S + 1, (M,), generator=g)
    elif order == "none":
        index = torch.full((M,), -1)
    else:
        index = (torch.arange(M) * S // M + 1) % S
    t = dict(x=x.to(TYPES[dtype]), a=(n(S, R, K) * K ** -0.5).to(w), b=(n(S, N, R) * R ** -0.5).to(w), index=index.int(),
             y=n(M, N).to(TYPES[out]), scale=torch.rand(S, generator=g) + 0.5, x_scale=xs)
    return {k: v if v is None else v.cuda() for k, v in t.items()}


def run(mssm, t, **kw):
    y = t["y"].clone()
    out = mssm.lora(t["x"], t["a"], t["b"], t["index"], y, scale=t["scale"], x_scale=t["x_scale"], **kw)
    assert out is y
    return y


def check(t, got, out):
    S, R, K = t["a"].shape
    x = t["x"].double() if t["x_scale"] is None else t["x"].double() * t["x_scale"].double()[:, None]
    want, room = t["y"].double(), torch.zeros_like(t["y"], dtype=torch.float64)
    for i in range(S):
        rows = (t["index"] == i).nonzero()[:, 0]
        a, b, s = t["a"][i].double(), t["b"][i].double(), t["scale"][i].double()
        inner, size = (x[rows] @ a.T.contiguous()) * s, (x[rows].abs() @ a.abs().T.contiguous()) * s
        want[rows] += inner @ b.T.contiguous()
        off = size * 2 * K ** 0.5 * 2.0 ** -24 + inner.abs() * (2.0 ** -15 if out == "bf16" else 2 * R ** 0.5 * 2.0 ** -24 + 2.0 ** -23)
        room[rows] += off @ b.abs().T.contiguous()
    bound = want.abs() * HALF[out] + room * (1 + HALF[out]) + t["y"].double().abs() * 2.0 ** -23
    off = (got.double() - want).abs()
    assert torch.all(off <= bound), (float(off.max()), float((off / (bound + 1e-300)).max()))
    none = (t["index"] < 0) | (t["index"] >= S)
    assert torch.equal(got[none], t["y"][none])


@pytest.mark.parametrize("dtype,out", [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32"), ("fp8", "bf16"), ("fp8", "f32")])
@pytest.mark.parametrize("M,K,N,R,S,order", [
    (1, 16, 16, 1, 1, "runs"), (3, 1537, 333, 12, 7, "any"), (64, 256, 700, 16, 64, "any"), (65, 129, 65, 17, 3, "any"),
    (300, 1537, 333, 12, 7, "any"), (130, 520, 256, 33, 5, "runs"), (2048, 64, 96, 64, 9, "runs"), (2049, 96, 70, 100, 4, "runs"),
    (2500, 70, 257, 128, 3, "any"), (2100, 40, 64, 5, 50, "any"), (100, 1, 1, 3, 2, "any"), (70, 33, 40, 7, 3, "none")])
def test_sums(mssm, M, K, N, R, S, order, dtype, out):
    t = make(M, K, N, R, S, dtype, out, order, seed=M + K)
    check(t, run(mssm, t), out)
