"""Beam selection at the sizes that take the many-rows form (4,096 logits a row
or more, rows enough for 512 spans of 8,192): distinct and repeated logits,
vocabularies on and off 16-byte boundaries, scores compared, beams finished and
out of use.  Every beam holds the same multiset of logits on a grid and the
scores lie a fraction of its step apart, so that the deciding values differ by
more than 2e-5 (asserted on the reference) or are equal within a beam."""
import numpy as np
import pytest

from test_gpu_beam import check

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mssm():
    import selective_state_space_mssm_amd as m
    return m


def inputs(B, K, V, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    if dtype == "f32":  # all distinct
        step, level = max(16.0 / V, 64e-6 * K), torch.arange(V)
    else:  # multiples of 1 / 16 up to 12: the upper ones once or twice, the lower ones many times
        top = torch.tensor([i for i in range(191, 150, -1) for _ in range(1 + i % 2)])
        step, level = 1.0 / 16, torch.cat([top, torch.arange(V - len(top)) * 150 // (V - len(top))])
    x = torch.stack([level[torch.randperm(V, generator=g)] for _ in range(B * K)]).view(B, K, V).float() * step
    scores = step * (torch.randint(0, 9, (B, K), generator=g) - torch.arange(K) / K)
    return x.bfloat16() if dtype == "bf16" else x, scores.float()


def many(B, K, V):
    return V >= 4096 and B * K * -(-V // 8192) >= 512


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,K,V", [(64, 8, 8200), (64, 8, 20001), (33, 16, 9000), (171, 3, 4097), (520, 1, 5000), (2, 8, 262001)])
def test_parity(mssm, B, K, V, dtype):
    assert many(B, K, V)
    x, s = inputs(B, K, V, dtype, V)
    check(mssm, x, s)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [8200, 20001])
def test_finished_banned_and_unused(mssm, V, dtype):
    B, K, end = 64, 8, 5
    x, s = inputs(B, K, V, dtype, V + 1)
    # bans go by the value, so that every beam of a row keeps the same multiset and the same softmax sum
    step = 16.0 / V if dtype == "f32" else 1.0 / 16
    level = (x.float() / step).round()
    x[(level % 97 == 1) & (x < 9)] = float("-inf")
    x[4][x[4] < 9] = torch.finfo(x.dtype).min
    low = torch.where(torch.isfinite(x[5, 1].float()), x[5, 1].float(), 99.0).argmin()
    x[5, 1, low] = float("nan")
    total = x[:, 0].double().logsumexp(-1)
    x[3, 2] = float("-inf")
    g = torch.Generator().manual_seed(V)
    done = torch.rand((B, K), generator=g) < 0.3
    done[7] = True
    # a finished beam's value is its score: half a beam's share of a step off the others' values
    most = V if dtype == "f32" else 192
    top = torch.randint(most - 4, most + 9, (B, K), generator=g) * step
    s = torch.where(done, (top - total[:, None] + step * (torch.arange(K) + 0.5) / K).float(), s)
    s[1, 1:] = float("-inf")
    s[2, 4] = float("nan")
    check(mssm, x, s, done, end)
    check(mssm, x, s)


def test_long_rows_of_few_distinct_values(mssm):
    # ties by the thousand in every span, the best in the last one
    B, K, V = 32, 16, 30000
    x = (torch.arange(V) % 7).float().expand(B, K, V).clone()
    x[:, :, V - 100:] += 1.0
    s = -torch.arange(K).float().expand(B, K) / 64
    check(mssm, x, s)
    check(mssm, x.bfloat16(), s)
