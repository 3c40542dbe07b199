"""GPU parity of the projections (mssm_linear) with their definition in float64.

Two kinds of inputs.  Small whole numbers: every partial sum is a whole number
below 2^24 (below 2^8 times the output's precision for a bfloat16 output), so
the result is exact in any order and has to be equal.  Normal ones: a sum of K
terms in float32 in any order is within K EPS32 of the sum of magnitudes; the
epilogue's few operations add 16 EPS32 of the same magnitude (the activations
have slopes below 1.13), a bfloat16 output its half ulp."""
import numpy as np
import pytest

import block_ref as ref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f8": torch.float8_e4m3fn}
PAIRS = [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32"), ("f8", "bf16"), ("f8", "f32")]


@pytest.fixture(scope="module")
def mssm():
    import selective_state_space_mssm_amd as m
    return m


def np64(t):
    return t.detach().float().double().cpu().numpy()


def whole(g, shape, top):
    return torch.randint(-top, top + 1, shape, generator=g).float()


def run_exact(mssm, M, K, N, dtype, out, residual=True, bias=True):
    print(f"[linear] exact {M} x {K} x {N} {dtype} -> {out}", flush=True)
    g = torch.Generator().manual_seed(M * 7 + K * 3 + N)
    # zeros in most places keep a bfloat16 result's magnitude below 256
    x = whole(g, (M, K), 2) * (torch.rand((M, K), generator=g) < min(1.0, 16 / K))
    w = whole(g, (N, K), 2)
    if out == "f32":
        x = whole(g, (M, K), 3)
    b = whole(g, (N,), 8) if bias else None
    r = whole(g, (M, N), 8) if residual else None
    kw = {}
    if dtype == "f8":  # scales that are powers of two keep it exact
        kw = {"x_scale": torch.ldexp(torch.ones(M), torch.arange(M) % 2).cuda(),
              "w_scale": torch.ldexp(torch.ones(N), -(torch.arange(N) % 2)).cuda()}
    y = mssm.linear(x.to(DT[dtype]).cuda(), w.to(DT[dtype]).cuda(), None if b is None else b.cuda(),
                    None if r is None else r.to(DT[out]).cuda(), out_dtype=DT[out], **kw)
    want, _ = ref.linear(x.double().numpy(), w.double().numpy(), None if b is None else b.double().numpy(),
                         None if r is None else r.double().numpy(), None,
                         *(np64(kw[k]) for k in ("x_scale", "w_scale") if k in kw))
    want = torch.from_numpy(want).to(DT[out])
    assert y.dtype == DT[out] and y.shape == (M, N)
    bad = (y.cpu() != want).nonzero()
    assert bad.numel() == 0, f"{bad.shape[0]} of {M * N} differ, first at {bad[0].tolist()}"


def run_normal(mssm, M, K, N, dtype, out, activation=None, bias=True, residual=True, seed=0):
    print(f"[linear] {M} x {K} x {N} {dtype} -> {out} {activation}", flush=True)
    g = torch.Generator().manual_seed(seed + M * 7 + K * 3 + N)
    x = torch.randn((M, K), generator=g).to(DT[dtype])
    w = (torch.randn((N, K), generator=g) * (4 if dtype == "f8" else K ** -0.5)).to(DT[dtype])
    b = torch.randn(N, generator=g) if bias else None
    r = torch.randn((M, N), generator=g).to(DT[out]) if residual else None
    xs = ws = None
    if dtype == "f8":
        xs = (0.5 + torch.rand(M, generator=g)) * K ** -0.5
        ws = 0.1 + 0.1 * torch.rand(N, generator=g)
    dev = lambda t: None if t is None else t.cuda()  # noqa: E731
    n = lambda t: None if t is None else np64(t)  # noqa: E731
    y = mssm.linear(dev(x), dev(w), dev(b), dev(r), activation, dev(xs), dev(ws), DT[out])
    want, mag = ref.linear(n(x), n(w), n(b), n(r), activation, n(xs), n(ws))
    tol = (K + 16) * ref.EPS32 * mag * 1.13 + ref.EPS32 * np.abs(want) * 2 + 1e-38
    if r is not None:
        tol = tol + ref.EPS32 * np.abs(n(r))
    if out == "bf16":
        tol = tol * (1 + ref.EPSB) + ref.EPSB * np.abs(want)
    err = np.abs(np64(y) - want)
    assert np.all(err <= tol), f"off by up to {np.max(err / tol):.3g} of the bound"


@pytest.mark.parametrize("dtype,out", PAIRS)
@pytest.mark.parametrize("M,K,N", [(1, 1, 1), (1, 16, 16), (2, 17, 3), (16, 64, 16), (17, 160, 33), (64, 256, 80), (65, 96, 64),
                                   (33, 1537, 129), (100, 512, 257), (128, 128, 128), (129, 144, 130), (256, 320, 256),
                                   (300, 1537, 333), (257, 2560, 511), (1000, 192, 48), (513, 63, 260)])
def test_exact(mssm, M, K, N, dtype, out):
    run_exact(mssm, M, K, N, dtype, out)


@pytest.mark.parametrize("dtype,out", PAIRS)
@pytest.mark.parametrize("M", [1, 2, 5, 8, 16, 31, 48, 64])
def test_few_rows(mssm, M, dtype, out):
    run_exact(mssm, M, 2560, 1024, dtype, out)
    run_exact(mssm, M, 515, 331, dtype, out)
    run_normal(mssm, M, 2560, 192, dtype, out, "silu")


@pytest.mark.parametrize("dtype,out", PAIRS)
@pytest.mark.parametrize("K", [1, 2, 3, 5, 8, 15, 31, 33, 64, 65, 127, 129, 250, 255, 257])
def test_every_kind_of_depth(mssm, K, dtype, out):
    run_exact(mssm, 7, K, 70, dtype, out)
    run_exact(mssm, 150, K, 70, dtype, out)


@pytest.mark.parametrize("dtype,out", PAIRS)
@pytest.mark.parametrize("activation", [None, "relu", "silu", "gelu"])
def test_epilogue(mssm, activation, dtype, out):
    for bias in (False, True):
        for residual in (False, True):
            run_normal(mssm, 70, 200, 90, dtype, out, activation, bias, residual)
    run_normal(mssm, 3, 5120, 72, dtype, out, activation)
    run_normal(mssm, 515, 1536, 80, dtype, out, activation)
    run_normal(mssm, 300, 321, 333, dtype, out, activation)


@pytest.mark.parametrize("dtype,out", PAIRS)
def test_many_tiles(mssm, dtype, out):
    run_exact(mssm, 2055, 136, 1544, dtype, out)
    run_exact(mssm, 1024, 256, 2048, dtype, out)


@pytest.mark.parametrize("dtype,out", PAIRS)
def test_long_sum_of_few_tiles(mssm, dtype, out):
    run_exact(mssm, 96, 20000, 40, dtype, out)
    run_exact(mssm, 200, 9001, 130, dtype, out)


@pytest.mark.parametrize("dtype,out", PAIRS)
def test_residual_in_place_and_leading_dimensions(mssm, dtype, out):
    g = torch.Generator().manual_seed(5)
    for M, K, N in ((6, 320, 100), (288, 320, 100), (96, 20000, 40)):
        x, w = whole(g, (M, K), 1).to(DT[dtype]).cuda(), whole(g, (N, K), 1).to(DT[dtype]).cuda()
        r = whole(g, (M, N), 8).to(DT[out]).cuda()
        kw = {"x_scale": torch.ones(M, device="cuda"), "w_scale": torch.ones(N, device="cuda")} if dtype == "f8" else {}
        y = mssm.linear(x, w, None, r, out_dtype=DT[out], **kw)
        r2 = r.clone()
        if kw:
            kw["x_scale"] = kw["x_scale"].view(2, M // 2)
        y2 = mssm.linear(x.view(2, M // 2, K), w, None, r2.view(2, M // 2, N), out_dtype=DT[out], y=r2.view(2, M // 2, N), **kw)
        assert torch.equal(y2.view(M, N), y) and torch.equal(r2, y)


@pytest.mark.parametrize("M", [3, 200])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f8"])
def test_values_that_are_no_numbers_stay_in_their_row(mssm, dtype, M):
    K, N = 72, 50
    x, w = torch.ones((M, K)), torch.ones((N, K))
    x[1, 5], w[7, 9] = float("nan"), float("nan")
    if dtype != "f8":
        x[2, K - 1] = float("inf")
    kw = {"x_scale": torch.ones(M, device="cuda"), "w_scale": torch.ones(N, device="cuda")} if dtype == "f8" else {}
    y = mssm.linear(x.to(DT[dtype]).cuda(), w.to(DT[dtype]).cuda(), out_dtype=torch.float32, **kw).cpu()
    nan = torch.zeros((M, N), dtype=torch.bool)
    nan[1], nan[:, 7] = True, True
    assert torch.equal(torch.isnan(y), nan)
    rest = y[~nan]
    assert torch.all((rest == K) | (rest == float("inf")))


def test_bitwise_repeats_on_another_stream(mssm):
    g = torch.Generator().manual_seed(1)
    for M, K, N in ((4, 2560, 1000), (96, 20000, 40), (300, 1537, 333)):
        x, w = torch.randn((M, K), generator=g).bfloat16().cuda(), torch.randn((N, K), generator=g).bfloat16().cuda()
        y = mssm.linear(x, w, activation="gelu")
        torch.cuda.synchronize()
        st = torch.cuda.Stream()
        with torch.cuda.stream(st):
            ys = [mssm.linear(x, w, activation="gelu") for _ in range(3)]
        st.synchronize()
        assert all(torch.equal(y, t) for t in ys)


@pytest.mark.parametrize("dtype,out", PAIRS)
@pytest.mark.parametrize("M,K,N", [(8200, 96, 17), (8300, 200, 128), (16400, 64, 33), (16385, 48, 80), (9000, 416, 100), (16384, 16, 16)])
def test_few_columns(mssm, M, K, N, dtype, out):
    run_exact(mssm, M, K, N, dtype, out)


@pytest.mark.parametrize("dtype,out", PAIRS)
@pytest.mark.parametrize("K", [1921, 2049, 2111, 2113, 3071, 4090])
def test_uneven_rows_end_anywhere_in_a_wave_s_steps(mssm, K, dtype, out):
    run_exact(mssm, 5, K, 37, dtype, out)      # few outputs
    run_exact(mssm, 70, K, 50, dtype, out)
    run_exact(mssm, 600, K, 1300, dtype, out)  # tiles


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f8"])
def test_large_tiles_with_a_split_tail(mssm, dtype):
    # 17 x 16 tiles of 256: one round of 256 and a tail that is cut along in_dim
    run_exact(mssm, 4352, 4096 // {"f32": 4, "bf16": 2, "f8": 1}[dtype], 4096, dtype, "f32" if dtype == "f32" else "bf16")


def test_eight_bit_sums_keep_float32_accuracy(mssm):
    # a float32 output shows what the 8-bit matrix instructions drop (1.5e-5): below 1e-6 here
    g = torch.Generator().manual_seed(9)
    for M, K, N in ((4, 2560, 512), (300, 2560, 512), (1100, 512, 1100), (8300, 512, 64)):
        x, w = (30 * torch.randn((M, K), generator=g)).to(DT["f8"]), (30 * torch.randn((N, K), generator=g)).to(DT["f8"])
        one = lambda n: torch.ones(n, device="cuda")  # noqa: E731
        y = mssm.linear(x.cuda(), w.cuda(), x_scale=one(M), w_scale=one(N), out_dtype=torch.float32)
        want = np64(x) @ np64(w).T
        assert np.linalg.norm(np64(y) - want) <= 1e-6 * np.linalg.norm(want)


@pytest.mark.parametrize("dtype,out", PAIRS)
@pytest.mark.parametrize("steps", [1, 2, 3, 4, 5, 6, 7, 11])
def test_few_rows_any_number_of_steps_a_wave(mssm, steps, dtype, out):
    size = {"f32": 4, "bf16": 2, "f8": 1}[dtype]
    for k in (1024 * steps, 1024 * steps - 112):  # bytes: all 8 waves' steps full, and the last cut short
        run_exact(mssm, 3, k // size, 40, dtype, out)
