"""Scores a prompt and continues it greedily with one projection and the head of a language model.

The operators as an engine chains them, on random weights:

  prompt  add_rmsnorm_e4m3_blk -> e4m3_blk_gemm -> add_rmsnorm -> mxfp4_quantize -> mxfp4_gemm (head) -> logprobs
  decode  add_rmsnorm_q8_1 -> q8_0_gemv -> add_rmsnorm -> mxfp4_gemv (head) -> logprobs, one token at a time

    python examples/score_prompt.py [--tokens 512] [--new 8] [--width 4096] [--vocab 64448]
"""
import argparse
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import block_quantized_matmul_02_amd as bqm  # noqa: E402
import workloads  # noqa: E402

EPS = 1e-6


class Model:
    """An embedding, one square projection (block-128 FP8 for prompts, Q8_0 for decode) and an MXFP4 head."""

    def __init__(self, width, vocab, device="cuda:0", seed=0):
        rng = np.random.default_rng(seed)
        g = torch.Generator(device=device).manual_seed(seed)
        self.embedding = torch.randn((vocab, width), generator=g, device=device)
        self.gains = [1.0 + 0.1 * torch.randn(width, generator=g, device=device) for _ in range(2)]
        codes, grid = workloads.e4m3_blk_weights(width, width, rng)
        self.w8, self.w8_grid = torch.from_numpy(codes).to(device), torch.from_numpy(grid).to(device)
        self.wq = torch.from_numpy(workloads.q8_0_weights(width, width, rng)).to(device)
        head = 0.02 * torch.randn((vocab, width), generator=g, device=device)
        self.head, self.head_scales = bqm.bqm_mxfp4_quantize(head)

    def prompt_logits(self, tokens):
        """Logits [m, vocab] after each of the prompt's tokens."""
        x = self.embedding.index_select(0, tokens)
        xq, xs, _ = bqm.bqm_add_rmsnorm_e4m3_blk(x, None, self.gains[0], EPS)
        out = bqm.bqm_e4m3_blk_gemm(self.w8, self.w8_grid, xq, xs)
        y, _ = bqm.bqm_add_rmsnorm(out, x, self.gains[1], EPS)
        yq, ys = bqm.bqm_mxfp4_quantize(y)
        return bqm.bqm_mxfp4_gemm(self.head, self.head_scales, yq, ys)

    def token_logits(self, token):
        """Logits [1, vocab] after one token."""
        x = self.embedding.index_select(0, token.view(1))
        xq, xds, _ = bqm.bqm_add_rmsnorm_q8_1(x, None, self.gains[0], EPS)
        out = bqm.bqm_q8_0_gemv(self.wq, xq, xds)
        y, _ = bqm.bqm_add_rmsnorm(out, x, self.gains[1], EPS, h=out)
        return bqm.bqm_mxfp4_gemv(self.head, self.head_scales, y)


def score(model, tokens, top=5):
    """Log probability of every prompt token but the first, the entropies, and the alternatives at each place."""
    logits = model.prompt_logits(tokens[:-1])
    logp, _, entropy, ids, top_logp = bqm.bqm_logprobs(logits, tokens[1:].int().view(-1, 1), top)
    return logp[:, 0], entropy, ids, top_logp


def continue_greedily(model, token, count, top=5):
    """The `count` likeliest next tokens, one after another, with their log probabilities."""
    chosen = []
    for _ in range(count):
        _, _, _, ids, top_logp = bqm.bqm_logprobs(model.token_logits(token), None, top)
        token = ids[0, 0].long()
        chosen.append((int(token), float(top_logp[0, 0])))
    return chosen


def main():
    p = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    p.add_argument("--tokens", type=int, default=512)
    p.add_argument("--new", type=int, default=8)
    p.add_argument("--width", type=int, default=4096)
    p.add_argument("--vocab", type=int, default=64448)
    a = p.parse_args()
    model = Model(a.width, a.vocab)
    tokens = torch.randint(0, a.vocab, (a.tokens,), device="cuda:0")
    logp, entropy, ids, _ = score(model, tokens)
    print(f"{a.tokens - 1} tokens scored: mean log probability {float(logp.mean()):.4f}, "
          f"mean entropy {float(entropy.mean()):.4f}, "
          f"in the top 5 {float((ids == tokens[1:, None]).any(1).float().mean()):.3f}")
    for token, lp in continue_greedily(model, tokens[-1], a.new):
        print(f"  next token {token}, log probability {lp:.4f}")


if __name__ == "__main__":
    main()
