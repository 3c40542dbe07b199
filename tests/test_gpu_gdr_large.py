"""GPU tests of the gated delta rule and the adapters where counts and offsets are
large: more sequences than a wave looks through at once, tensors of more than 2^31
elements (their last part is checked)."""
import pytest

torch = pytest.importorskip("torch")
import gdr_ref as ref  # noqa: E402
from test_gpu_gdr_edges import GRADS, train  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mssm():
    import selective_state_space_mssm_amd as m
    return m


@pytest.mark.parametrize("lengths", [[i % 4 for i in range(200)], [0] * 65 + [70] + [0] * 70 + [1]], ids=["200", "137"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_many_sequences(mssm, lengths, dtype):
    x = ref.inputs(lengths, 1, 2, 32, 32, dtype, seed=1)
    t = ref.on_gpu(x, dtype)
    want_y, want_s, want = ref.gradients(x, norm=True)
    y, s, got = train(mssm, t)
    chunks = -(-max(lengths) // 64)
    ref.check(y, want_y, dtype, chunks, "y")
    ref.check(s, want_s, "f32", chunks, "h_final")
    for n in GRADS:
        ref.check(got[n], want[n], dtype if n in ("dq", "dk", "dv") else "f32", chunks, n, gradient=True)


@pytest.mark.parametrize("lengths", [[int(i % 50 == 7) for i in range(5000)], [130] + [0] * 4200 + [65]], ids=["5000", "4202"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_thousands_of_sequences(mssm, lengths, dtype):
    # as the ones that have tokens by themselves, bit for bit; the others hand their states on
    x = ref.inputs(lengths, 1, 2, 32, 32, dtype, seed=2)
    t = ref.on_gpu(x, dtype)
    some = torch.tensor(lengths) > 0
    ends = torch.tensor([0] + [n for n in lengths if n]).cumsum(0).int()
    u = {**t, "offsets": ends.cuda(), "h0": t["h0"][some.cuda()], "dh_final": t["dh_final"][some.cuda()]}
    y, s, got = train(mssm, t)
    want_y, want_s, want = train(mssm, u)
    if dtype == "f32":  # one form for any number of sequences
        assert torch.equal(y, want_y) and torch.equal(s[some.cuda()], want_s)
        for n in GRADS:
            assert torch.equal(got[n][some.cuda()] if n == "dh0" else got[n], want[n]), n
    else:
        ref.check(s[some.cuda()], want_s.cpu(), "f32", 3, "h_final")
    ref.check(y, ref.forward({n: v if n == "offsets" else v.double().cpu() for n, v in u.items()} | {"offsets": ends}, norm=True)[0],
              dtype, 3, "y")
    none = ~some.cuda()
    assert torch.equal(s[none], t["h0"][none]) and torch.equal(got["dh0"][none], t["dh_final"][none])


def test_more_elements_than_31_bits(mssm):
    T, last, H, K, V = 140_000, 1000, 128, 16, 128
    assert T * H * V > 2 ** 31
    g = torch.Generator(device="cuda").manual_seed(1)
    n = lambda *s, **k: torch.randn(*s, generator=g, device="cuda", **k)  # noqa: E731
    bf = dict(dtype=torch.bfloat16)
    x = (n(1, T, 1, K, **bf), n(1, T, 1, K, **bf), n(1, T, H, V, **bf), -0.1 * torch.rand(1, T, H, generator=g, device="cuda"),
         torch.rand(1, T, H, generator=g, device="cuda"))
    offsets = torch.tensor([0, T - last, T], dtype=torch.int32, device="cuda")
    y, s = mssm.gdr_fwd(*x, offsets=offsets, norm_qk=True)
    part = {k: v[:, T - last:].double().cpu() for k, v in zip(("q", "k", "v", "g", "beta"), x)}
    want_y, want_s = ref.forward({**part, "h0": None, "offsets": None}, norm=True)
    ref.check(y[:, T - last:], want_y, "bf16", 16, "y")
    ref.check(s[1:], want_s, "f32", 16, "h_final")


def test_a_pool_of_more_than_31_bits(mssm):
    S, H, K, V = 4200, 32, 128, 128
    assert S * H * K * V > 2 ** 31
    pool = torch.zeros(S, H, V, K, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(1)
    x = [torch.randn(2, h, d, generator=g, device="cuda") for h, d in ((H, K), (H, K), (H, V))]
    gates = [-torch.rand(2, H, generator=g, device="cuda"), torch.rand(2, H, generator=g, device="cuda")]
    start = torch.randn(2, H, V, K, generator=g, device="cuda")
    pool[S - 1], pool[0] = start[0], start[1]
    y = mssm.gdr_step(*x, *gates, pool, slots=torch.tensor([S - 1, 0], dtype=torch.int32, device="cuda"), norm_qk=True)
    want = mssm.gdr_step(*x, *gates, start, norm_qk=True)
    assert torch.equal(y, want) and torch.equal(pool[S - 1], start[0]) and torch.equal(pool[0], start[1])
    assert not pool[1:S - 1].any()


def test_adapters_of_more_elements_than_31_bits(mssm):
    M, K, N, R = 215_000, 16, 10_240, 4
    assert M * N > 2 ** 31
    g = torch.Generator(device="cuda").manual_seed(1)
    bf = dict(generator=g, device="cuda", dtype=torch.bfloat16)
    x, a, b = torch.randn(M, K, **bf), torch.randn(3, R, K, **bf), torch.randn(3, N, R, **bf)
    y = torch.zeros(M, N, device="cuda", dtype=torch.bfloat16)
    index = torch.full((M,), -1, dtype=torch.int32, device="cuda")
    index[-100:] = torch.arange(100, device="cuda") % 4 - 1
    mssm.lora(x, a, b, index, y)
    want = torch.zeros(100, N, device="cuda", dtype=torch.bfloat16)
    mssm.lora(x[-100:].contiguous(), a, b, index[-100:].contiguous(), want)
    # two sums of the same float32 products in another order: a step of bfloat16 apart at most
    off = (y[-100:].double() - want.double()).abs()
    assert torch.all(off <= want.double().abs() * 2.0 ** -7 + 2.0 ** -15 * want.double().abs().max())
    assert want[index[-100:] >= 0].any() and not y[:-100].any() and not y[-100:][index[-100:] < 0].any()


def test_a_single_row_without_leading_sizes(mssm):
    x, a, b = torch.ones(8, device="cuda"), torch.ones(1, 2, 8, device="cuda"), torch.ones(1, 5, 2, device="cuda")
    y = mssm.lora(x, a, b, torch.tensor(0, dtype=torch.int32, device="cuda"), torch.zeros(5, device="cuda"))
    assert torch.equal(y.cpu(), torch.full((5,), 16.0))
