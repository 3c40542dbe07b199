"""Serving a small Mamba language model with beam search, on this library's operators alone.

    python examples/serve_beam.py [--layers 4 --dim 512 --beams 4 --prompt 64 --tokens 32]

Random weights (a demonstration of the calls, not of a trained model).  A block
is residual + norm (8-bit rows), projections on the 8-bit rows, causal conv1d +
SiLU + selective scan, output projection; the residual stream is float32 and its
addition is fused into the next block's norm.  Step size, B and C are projected
from the block's input next to x and z, so that the conv runs fused in front of
the scan.  A prompt goes through conv_scan_fwd in one call a layer, then every
token of every beam through conv_step; after each selection the stacked states
of all layers follow their beams in one beam_reorder call.
"""
from __future__ import annotations

import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import selective_state_space_mssm_amd as mssm  # noqa: E402


def rows8(w):
    """Weight rows in 8 bits with a scale each."""
    scale = w.abs().amax(1).clamp(min=1e-30) / 448.0
    return (w / scale[:, None]).to(torch.float8_e4m3fn), scale


class Model:
    """dim: width of the residual stream; every layer has 2 * dim channels."""

    def __init__(self, layers=4, dim=512, vocab=4096, dstate=16, dconv=4, seed=0, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)
        rnd = lambda *s, k=1.0: torch.randn(s, generator=g, device=device) * k  # noqa: E731
        self.dim, self.inner, self.vocab, self.dstate, self.dconv = dim, 2 * dim, vocab, dstate, dconv
        self.rank = max(16, dim // 16)
        D, R = self.inner, self.rank
        self.embedding = rnd(vocab, dim).bfloat16()
        self.head = (rnd(vocab, dim, k=3 * dim ** -0.5)).bfloat16()
        self.norm = torch.ones(dim, device=device)
        self.layers = []
        for _ in range(layers):
            dt = torch.exp(torch.empty(D, device=device).uniform_(-6.9, -2.3, generator=g))
            self.layers.append({
                "norm": 1 + rnd(dim, k=0.1),
                "x": rows8(rnd(D, dim, k=dim ** -0.5)), "z": rows8(rnd(D, dim, k=dim ** -0.5)),
                "dt": rows8(rnd(R, dim, k=dim ** -0.5)),
                "B": rows8(rnd(dstate, dim, k=dim ** -0.5)), "C": rows8(rnd(dstate, dim, k=dim ** -0.5)),
                "dt_up": rnd(D, R, k=0.5 * R ** -0.5).bfloat16(), "dt_bias": dt + torch.log(-torch.expm1(-dt)),
                "conv_w": rnd(D, dconv, k=dconv ** -0.5), "conv_b": rnd(D, k=0.1),
                "A": -torch.arange(1, dstate + 1, device=device).float().repeat(D, 1), "D": torch.ones(D, device=device),
                "out": rnd(dim, D, k=D ** -0.5).bfloat16()})

    def states(self, rows):
        dev, L = self.embedding.device, len(self.layers)
        return (torch.zeros((L, rows, self.inner, self.dstate), device=dev),
                torch.zeros((L, rows, self.dconv - 1, self.inner), dtype=torch.bfloat16, device=dev))

    def _projections(self, p, h, residual):
        q, scale, residual = mssm.add_rmsnorm_q8(h, p["norm"], residual)
        x, z, dt, B, C = (mssm.linear(q, p[k][0], x_scale=scale, w_scale=p[k][1]) for k in ("x", "z", "dt", "B", "C"))
        return x, z, mssm.linear(dt, p["dt_up"]), B, C, residual

    def _logits(self, h, residual):
        h, _ = mssm.add_rmsnorm(h, self.norm, residual)
        return mssm.linear(h, self.head, out_dtype=torch.float32)

    def prefill(self, tokens, every=False):
        """(rows, L) tokens: logits after the last one (or after each), and the states they leave."""
        rows, L = tokens.shape
        ssm, conv = self.states(rows)
        h = self.embedding[tokens]
        residual = torch.zeros((rows, L, self.dim), device=h.device)
        for i, p in enumerate(self.layers):
            x, z, dt, B, C, residual = self._projections(p, h, residual)
            y, _, _ = mssm.conv_scan_fwd(x, p["conv_w"], dt, p["A"], B, C, p["D"], z, p["dt_bias"], conv_b=p["conv_b"],
                                         h_final=ssm[i])
            n = min(L, self.dconv - 1)
            conv[i, :, self.dconv - 1 - n:] = x[:, L - n:]
            h = mssm.linear(y, p["out"])
        if not every:
            h, residual = h[:, -1].contiguous(), residual[:, -1].contiguous()
        return self._logits(h, residual), ssm, conv

    def step(self, tokens, ssm, conv):
        """(rows) tokens, one each: logits; the states move on in place."""
        h = self.embedding[tokens]
        residual = torch.zeros((tokens.shape[0], self.dim), device=h.device)
        for i, p in enumerate(self.layers):
            x, z, dt, B, C, residual = self._projections(p, h, residual)
            y = mssm.conv_step(x, p["conv_w"], conv[i], dt, p["A"], B, C, ssm[i], p["D"], z, p["dt_bias"], conv_b=p["conv_b"])
            h = mssm.linear(y, p["out"])
        return self._logits(h, residual)


@torch.no_grad()
def beam_search(model, prompt, beams, tokens, end_token=None):
    """prompt (batch, L): (sequences (batch, beams, tokens), scores, finished), best beam first."""
    batch = prompt.shape[0]
    logits, ssm, conv = model.prefill(prompt)
    # every beam starts from the prompt's state; only the first is in use, so that the first choice is among its tokens
    ssm, conv = (t.repeat_interleave(beams, 1) for t in (ssm, conv))
    logits = logits.repeat_interleave(beams, 0).view(batch, beams, -1)
    scores = torch.full((batch, beams), float("-inf"), device=prompt.device)
    scores[:, 0] = 0.0
    finished = None if end_token is None else torch.zeros((batch, beams), dtype=torch.bool, device=prompt.device)
    sequences = torch.zeros((batch, beams, 0), dtype=torch.int32, device=prompt.device)
    for t in range(tokens):
        scores, parent, token, finished = mssm.beam_select(logits, scores, finished, end_token)
        mssm.beam_reorder(parent, [ssm, conv])
        sequences = torch.cat([sequences.gather(1, parent.long()[:, :, None].expand_as(sequences)), token[:, :, None]], 2)
        if t + 1 < tokens:
            logits = model.step(token.view(-1).long(), ssm, conv).view(batch, beams, -1)
    return sequences, scores, finished


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    for name, value in (("layers", 4), ("dim", 512), ("vocab", 4096), ("batch", 2), ("beams", 4), ("prompt", 64), ("tokens", 32)):
        ap.add_argument("--" + name, type=int, default=value)
    a = ap.parse_args()
    model = Model(a.layers, a.dim, a.vocab)
    prompt = torch.randint(0, a.vocab, (a.batch, a.prompt), device="cuda", generator=torch.Generator("cuda").manual_seed(1))
    beam_search(model, prompt, a.beams, 2)
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    sequences, scores, _ = beam_search(model, prompt, a.beams, a.tokens)
    torch.cuda.synchronize()
    ms = (time.perf_counter() - t0) * 1e3
    for b in range(a.batch):
        print(f"prompt {b}: score {scores[b, 0].item():.3f}, tokens {sequences[b, 0].tolist()}")
    print(f"{a.batch} x {a.beams} beams, {a.prompt} + {a.tokens} tokens, {a.layers} layers of {2 * a.dim} channels: {ms:.1f} ms, "
          f"{ms / a.tokens:.2f} ms a token step")


if __name__ == "__main__":
    main()
