"""GPU parity of the residual addition + root-mean-square norm (mssm_add_rmsnorm,
mssm_add_rmsnorm_q8) with its definition in float64.

Tolerances.  h = x + residual is rounded once (half an ulp, EPS32 relative).
The sum of squares of D terms, each with two roundings, is formed by at least
64 partial sums: at most (D / 64 + 10) roundings deep, halved by the square
root; then mean, eps, root, reciprocal and two products: (D / 128 + 16) EPS32
relative to y covers all.  A bfloat16 output adds its own half ulp, EPSB; an
e4m3 output half a step of its value."""
import numpy as np
import pytest

import block_ref as ref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def mssm():
    import selective_state_space_mssm_amd as m
    return m


def np64(t):
    return t.detach().double().cpu().numpy()


def inputs(rows, dim, dtype, residual, seed=0, spread=True):
    g = torch.Generator().manual_seed(seed + 1000 * rows + dim)
    x = torch.randn((rows, dim), generator=g)
    if spread:
        x[:, ::7] *= 8.0
    res = None if residual is None else (3 * torch.randn((rows, dim), generator=g)).to(DT[residual]).cuda()
    return x.to(DT[dtype]).cuda(), res, (1 + 0.2 * torch.randn(dim, generator=g)).cuda()


def check(mssm, x, res, w, eps=1e-5):
    print(f"[norm] {tuple(x.shape)} {x.dtype} residual {None if res is None else res.dtype}", flush=True)
    D = x.shape[-1]
    tol = (D / 128 + 16) * ref.EPS32
    yr, hr = ref.norm(np64(x), np64(w), None if res is None else np64(res), eps)
    y, h = mssm.add_rmsnorm(x, w, res, eps)
    q, scale, h8 = mssm.add_rmsnorm_q8(x, w, res, eps)
    torch.cuda.synchronize()
    assert y.dtype == x.dtype and q.dtype == torch.float8_e4m3fn
    half = ref.EPSB if x.dtype == torch.bfloat16 else ref.EPS32
    assert np.all(np.abs(np64(y) - yr) <= np.abs(yr) * (tol + half) + 1e-38)
    if res is None:
        assert h is None and h8 is None
    else:
        half = ref.EPSB if res.dtype == torch.bfloat16 else 0.0
        assert np.all(np.abs(np64(h) - hr) <= np.abs(hr) * (half + ref.EPS32) + 1e-38)
        assert torch.equal(h, h8)
    sr = np.maximum(np.abs(yr).max(-1), 1e-30) / 448
    assert np.all(np.abs(np64(scale) - sr) <= sr * (tol + 2 * ref.EPS32))
    v = yr / sr[..., None]
    assert np.all(np.abs(np64(q.float()) - v) <= 0.5 * ref.f8_step(v) + np.abs(v) * (2 * tol + 4 * ref.EPS32))


@pytest.mark.parametrize("residual", [None, "f32", "bf16"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,dim", [(1, 1), (3, 7), (5, 64), (1, 2560), (4, 768), (2, 511), (3, 513), (7, 1537), (2, 4095),
                                      (2, 4104), (9, 5120), (2, 8191), (1, 16384), (2, 16392), (1, 33001)])
def test_parity(mssm, rows, dim, dtype, residual):
    check(mssm, *inputs(rows, dim, dtype, residual))


@pytest.mark.parametrize("dim", list(range(2, 34)) + [127, 129, 255, 257, 1023, 1025, 1033, 2047, 2049, 3583, 3585])
def test_every_small_width_and_around_the_vector_steps(mssm, dim):
    check(mssm, *inputs(3, dim, "bf16", "f32"))
    check(mssm, *inputs(3, dim, "f32", "bf16"))


def test_many_rows(mssm):
    check(mssm, *inputs(4099, 640, "bf16", "f32"))


def test_leading_dimensions(mssm):
    x, res, w = inputs(24, 96, "f32", "f32")
    y, h = mssm.add_rmsnorm(x, w, res)
    y3, h3 = mssm.add_rmsnorm(x.view(2, 3, 4, 96), w, res.view(2, 3, 4, 96))
    assert torch.equal(y3.view(24, 96), y) and torch.equal(h3.view(24, 96), h)
    q, s, _ = mssm.add_rmsnorm_q8(x.view(2, 12, 96), w)
    assert q.shape == (2, 12, 96) and s.shape == (2, 12)


@pytest.mark.parametrize("dim", [768, 1537, 5120, 20001])
def test_in_place(mssm, dim):
    x, res, w = inputs(6, dim, "bf16", "bf16")
    y, h = mssm.add_rmsnorm(x, w, res)
    x2, r2 = x.clone(), res.clone()
    y2, h2 = mssm.add_rmsnorm(x2, w, r2, y=x2, residual_out=r2)
    assert y2 is x2 and h2 is r2
    assert torch.equal(y2, y) and torch.equal(h2, h)


def test_residual_out_without_residual(mssm):
    x, _, w = inputs(3, 100, "bf16", None)
    out = torch.empty((3, 100), device="cuda")
    y, h = mssm.add_rmsnorm(x, w, residual_out=out)
    assert h is out and torch.equal(h, x.float())


@pytest.mark.parametrize("dim", [100, 768, 1537, 20001])
def test_zeros_and_values_that_are_no_numbers(mssm, dim):
    x, res, w = inputs(6, dim, "f32", "f32")
    x[0], res[0] = 0, 0
    x[1], res[1] = 1e-37, 0
    x[2, dim // 2] = float("nan")
    x[3, dim // 3] = float("inf")
    q, scale, _ = mssm.add_rmsnorm_q8(x, w, res, eps=1e-5)
    y, _ = mssm.add_rmsnorm(x, w, res, eps=1e-5)
    s, v, n = np64(scale), np64(q.float()), np64(y)
    assert np.all(v[0] == 0) and s[0] == np.float32(1e-30) / np.float32(448) and np.all(n[0] == 0)
    assert np.all(np.isfinite(v[1])) and s[1] > 0
    assert np.isnan(s[2]) and np.all(np.isnan(v[2])) and np.all(np.isnan(n[2]))
    assert np.isnan(s[3]) and np.all(np.isnan(v[3])) and np.isnan(n[3, dim // 3])
    check(mssm, x[4:].clone(), res[4:].clone(), w)


def test_large_and_small_magnitudes(mssm):
    for m in (1e-15, 1e15):
        x, res, w = inputs(4, 320, "f32", "f32")
        check(mssm, x * m, res * m, w, eps=0.0)


def test_other_stream_and_repeats(mssm):
    x, res, w = inputs(64, 1537, "bf16", "f32")
    q, s, h = mssm.add_rmsnorm_q8(x, w, res)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        for _ in range(3):
            q2, s2, h2 = mssm.add_rmsnorm_q8(x, w, res)
    st.synchronize()
    assert torch.equal(q.view(torch.uint8), q2.view(torch.uint8)) and torch.equal(s, s2) and torch.equal(h, h2)


def test_more_rows_than_a_launch_holds(mssm):
    rows, dim = (1 << 22) + 5, 9
    x = torch.randn((rows, dim), device="cuda").bfloat16()
    w = torch.rand(dim, device="cuda") + 0.5
    y, h = mssm.add_rmsnorm(x, w, x)
    q, s, _ = mssm.add_rmsnorm_q8(x, w, x)
    tail = slice(rows - 9, rows)
    y2, h2 = mssm.add_rmsnorm(x[tail].clone(), w, x[tail].clone())
    q2, s2, _ = mssm.add_rmsnorm_q8(x[tail].clone(), w, x[tail].clone())
    assert torch.equal(y[tail], y2) and torch.equal(h[tail], h2) and torch.equal(s[tail], s2)
    assert torch.equal(q[tail].view(torch.uint8), q2.view(torch.uint8))
    full = (2 * x.float()).double()
    want = full / torch.sqrt((full * full).mean(1, keepdim=True) + 1e-5) * w.double()
    assert torch.all((y.double() - want).abs() <= want.abs() * (ref.EPSB + 20 * ref.EPS32) + 1e-38)


@pytest.mark.parametrize("dim", [2560, 1537, 20001])
@pytest.mark.parametrize("dtype,residual", [("bf16", "f32"), ("f32", "bf16"), ("bf16", None)])
def test_eight_bit_values_are_the_nearest(mssm, dim, dtype, residual):
    # h w (448 / max |h w|) is rounded once: every value is the e4m3 nearest to the exact one (r cancels), but
    # for those within the carried product's error, 2^-40 relative, of a rounding boundary
    x, res, w = inputs(4000 if dim < 10000 else 100, dim, dtype, residual, seed=3)
    q, _, _ = mssm.add_rmsnorm_q8(x, w, res)
    t = (np64(x) + (0 if res is None else np64(res))) * np64(w)
    v = t * (448.0 / np.abs(t).max(1, keepdims=True))
    step = ref.f8_step(v)
    q = np64(q.float())
    assert np.all(np.abs(q - v) <= 0.5 * step + np.abs(v) * 2.0 ** -40)
    sure = np.abs(np.abs(np.fmod(v / step, 1.0)) - 0.5) * step > np.abs(v) * 2.0 ** -40
    assert np.array_equal(q[sure], (np.round(v / step) * step)[sure])
