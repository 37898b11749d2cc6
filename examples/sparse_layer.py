"""One layer of a sparse language model that serves several fine-tunes: a projection with low-rank adapters beside it,
and a layer of gated experts, on random weights.

  prompt  add_rmsnorm -> f16_gemm + lora_add -> add_rmsnorm -> f16_gemm (router) -> route -> group_rows ->
          mxfp4_quantize -> mxfp4_grouped_gemm (gated) -> mxfp4_quantize -> mxfp4_grouped_gemm -> combine
  decode  add_rmsnorm -> q8_0_gemv + lora_add -> add_rmsnorm -> f16_gemm (router) -> route ->
          mxfp4_expert_gemv (gated) -> mxfp4_expert_gemv -> combine, up to 15 tokens at a time

    python examples/sparse_layer.py [--tokens 512] [--width 4096] [--inner 1408] [--experts 64] [--top 6] [--adapters 8]
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


class Layer:
    """A square projection (Q8_0, with its fp16 mirror for prompts), adapters, a router and MXFP4 experts."""

    def __init__(self, width, inner, experts, top, adapters, rank=16, device="cuda:0", seed=0):
        g = torch.Generator(device=device).manual_seed(seed)

        def normal(*shape, std=1.0):
            return std * torch.randn(shape, generator=g, device=device)

        self.top, self.experts, self.adapters = top, experts, adapters
        self.gains = [1.0 + normal(width, std=0.1) for _ in range(2)]
        self.w = torch.from_numpy(workloads.q8_0_weights(width, width, np.random.default_rng(seed))).to(device)
        self.w16 = bqm.bqm_q8_0_dequant_f16(self.w, width)
        self.a = normal(adapters, rank, width, std=width ** -0.5).bfloat16()
        self.b = normal(adapters, width, rank, std=0.1).bfloat16()
        self.scale = 0.5 + torch.rand(adapters, generator=g, device=device)
        self.router = normal(experts, width, std=2 * width ** -0.5).half()
        self.up, self.up_scales = self._experts(normal, 2 * inner, width)
        self.down, self.down_scales = self._experts(normal, width, inner)

    def _experts(self, normal, n, k):
        codes, scales = zip(*(bqm.bqm_mxfp4_quantize(normal(n, k, std=k ** -0.5)) for _ in range(self.experts)))
        return torch.stack(codes), torch.stack(scales)

    def plan(self, adapter_ids):
        """The rows' adapters (int32, -1 for none) as lora_add takes them: one plan serves every layer of a step."""
        return bqm.bqm_group_rows(adapter_ids, self.adapters)

    def route(self, y):
        """Each token's experts and their weights."""
        return bqm.bqm_route(bqm.bqm_f16_gemm(self.router, bqm.bqm_f16_cvt(y)), self.top)

    def prompt(self, x, plan):
        """A prompt's rows ``x [m, width]`` (f32) -> the layer's output."""
        y, _ = bqm.bqm_add_rmsnorm(x, None, self.gains[0], EPS)
        out = bqm.bqm_f16_gemm(self.w16, bqm.bqm_f16_cvt(y))
        bqm.bqm_lora_add(y, self.a, self.b, *plan, scale=self.scale, res=out, y=out)
        y, h = bqm.bqm_add_rmsnorm(out, x, self.gains[1], EPS)
        ids, weights = self.route(y)
        slots = bqm.bqm_group_rows(ids, self.experts)
        inner = bqm.bqm_mxfp4_grouped_gemm(self.up, self.up_scales, *bqm.bqm_mxfp4_quantize(y), *slots, glu=True,
                                           out_dtype=torch.bfloat16)
        outer = bqm.bqm_mxfp4_grouped_gemm(self.down, self.down_scales, *bqm.bqm_mxfp4_quantize(inner), *slots,
                                           out_dtype=torch.bfloat16)
        return bqm.bqm_combine(outer, weights, res=h)

    def decode(self, x, plan):
        """One token of each of up to 15 requests."""
        y, _ = bqm.bqm_add_rmsnorm(x, None, self.gains[0], EPS)
        out = bqm.bqm_q8_0_gemv(self.w, *bqm.bqm_q8_1_quantize(y))
        bqm.bqm_lora_add(y, self.a, self.b, *plan, scale=self.scale, res=out, y=out)
        y, h = bqm.bqm_add_rmsnorm(out, x, self.gains[1], EPS)
        ids, weights = self.route(y)
        inner = bqm.bqm_mxfp4_expert_gemv(self.up, self.up_scales, y, ids, glu=True)
        outer = bqm.bqm_mxfp4_expert_gemv(self.down, self.down_scales, inner, ids)
        return bqm.bqm_combine(outer, weights, res=h)


def main():
    p = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    for name, value in (("tokens", 512), ("width", 4096), ("inner", 1408), ("experts", 64), ("top", 6), ("adapters", 8)):
        p.add_argument(f"--{name}", type=int, default=value)
    a = p.parse_args()
    layer = Layer(a.width, a.inner, a.experts, a.top, a.adapters)
    g = torch.Generator(device="cuda:0").manual_seed(1)
    x = torch.randn((a.tokens, a.width), generator=g, device="cuda:0")
    ids = torch.randint(-1, a.adapters, (a.tokens,), generator=g, device="cuda:0", dtype=torch.int32)
    out = layer.prompt(x, layer.plan(ids))
    few = min(a.tokens, 8)
    steps = layer.decode(x[:few].contiguous(), layer.plan(ids[:few].contiguous()))
    gap = (out[:few] - steps).norm() / steps.norm()
    print(f"{a.tokens} rows through the prompt's path, {few} of them through the decode path: "
          f"relative difference {float(gap):.3f} (the prompt's activations have 4 bits)")


if __name__ == "__main__":
    main()
