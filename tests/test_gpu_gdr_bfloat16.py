"""GPU tests of y of whole bfloat16 sequences where what the state holds cancels against what is written: the sums are
float32 and rounded once.

Keys and queries are unit vectors, a chunk's all different, beta = 1, nothing decays: a token replaces a column of the
state, S e_j + (v - S e_j) = v.  A state's column and every product are exact then; v - S e_j, its sum with S e_j for y
and the same sum for the state round once each, by 2^-24 of what was the column, and a later token reads a column that
two such roundings have gone into: 5 of them in all at most, of M = max|v|, |S|.  y is then rounded to bfloat16 once,
2^-8 of itself.  The values of every second chunk are 4096 times those between: 16 bits of a column leave 2^-16 M, and
the small values then have no digit left."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

CASES = [  # sequences, tokens, heads, K, V
    (1, 200, 2, 64, 32), (2, 200, 1, 128, 48), (3, 130, 8, 128, 128),     # few columns
    (1, 200, 80, 64, 64), (2, 200, 72, 128, 64),                          # 64 columns a workgroup
    (3, 200, 48, 64, 112), (2, 200, 80, 128, 128),                        # 128
    (1, 5000, 2, 64, 64), (1, 4160, 1, 128, 128),                         # in pieces
]


@pytest.mark.parametrize("B,L,H,K,V", CASES)
@pytest.mark.parametrize("kind", ["gdr_fwd", "gdr_fwd_train"])
def test_values_come_back_from_under_large_ones(B, L, H, K, V, kind):
    import selective_state_space_mssm_amd as mssm
    r = torch.Generator().manual_seed(L + H)
    keys = torch.stack([torch.cat([torch.randperm(K, generator=r)[:64] for _ in range(-(-L // 64))])[:L] for _ in range(B)])
    big = 4096.0
    size = torch.where(torch.arange(L) // 64 % 2 == 1, big, 1.0)[:, None, None]
    v = (torch.randn((B, L, H, V), generator=r) * size).bfloat16()
    h0 = torch.randn((B, H, V, K), generator=r) * big
    k = torch.nn.functional.one_hot(keys, K).bfloat16()[:, :, None].cuda()
    g, beta = torch.zeros((B, L, H), device="cuda"), torch.ones((B, L, H), device="cuda")
    y, s = getattr(mssm, kind)(k, k, v.cuda(), g, beta, h0.cuda(), scale=1.0)[:2]
    m = float(max(v.float().abs().max(), h0.abs().max()))
    off = (y.cpu().double() - v.double()).abs()
    assert torch.all(off <= 2.0 ** -8 * v.double().abs() + 5 * 2.0 ** -24 * m), float((off / m).max())
    want = h0.clone()
    for t in range(L):
        for b in range(B):
            want[b, :, :, keys[b, t]] = v[b, t].float()
    assert float((s.cpu() - want).abs().max()) <= 5 * 2.0 ** -24 * m
