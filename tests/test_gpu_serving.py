"""The operators around the scan run together, as examples/serve_beam.py uses
them: a beam search whose scores have to be those of its sequences, scored
again from the start by one prefill of prompt + sequence (no beams, no steps,
no reordering).  Both ways round the same rows the same, but for the scan's and
the step's own float32 differences, which a bfloat16 or 8-bit rounding can
carry over: 2e-2 a token at most, by the forward tolerance of bfloat16 paths."""
import os
import sys

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def serve():
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import serve_beam
    return serve_beam


@pytest.mark.parametrize("batch,beams,prompt,tokens,dim", [(1, 4, 17, 9, 128), (3, 3, 5, 12, 64), (2, 1, 40, 6, 256)])
def test_scores_are_those_of_the_sequences(serve, batch, beams, prompt, tokens, dim):
    model = serve.Model(layers=3, dim=dim, vocab=501)
    p = torch.randint(0, 501, (batch, prompt), device="cuda", generator=torch.Generator("cuda").manual_seed(prompt))
    seq, scores, _ = serve.beam_search(model, p, beams, tokens)
    assert torch.all(scores[:, :-1] >= scores[:, 1:])
    whole = torch.cat([p[:, None].expand(batch, beams, prompt), seq.long()], 2).view(batch * beams, -1)
    logits, _, _ = model.prefill(whole[:, :-1].contiguous(), every=True)
    logp = torch.log_softmax(logits.double(), -1)[:, prompt - 1:]
    again = logp.gather(2, whole[:, prompt:, None])[..., 0].sum(1).view(batch, beams)
    assert torch.all((again - scores.double()).abs() <= 2e-2 * tokens), (again, scores)
    # the beams of a batch row are different sequences
    for b in range(batch):
        assert len({tuple(s) for s in seq[b].tolist()}) == beams


def test_finished_beams_stay_as_they_are(serve):
    model = serve.Model(layers=2, dim=64, vocab=50)
    p = torch.randint(0, 50, (2, 8), device="cuda", generator=torch.Generator("cuda").manual_seed(0))
    seq, scores, finished = serve.beam_search(model, p, 4, 40, end_token=7)
    for b in range(2):
        for k in range(4):
            s = seq[b, k].tolist()
            assert bool(finished[b, k]) == (7 in s)
            if 7 in s:
                assert all(t == 7 for t in s[s.index(7):])
