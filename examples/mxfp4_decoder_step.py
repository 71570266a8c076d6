"""One decoding step of a small mixture-of-experts block with 4-bit weights.

    python examples/mxfp4_decoder_step.py [--tokens 4] [--steps 20]

Quantises the weights once (a projection, the experts), then runs steps of

    h = x + projection(x)           # matmul_mxfp4: activations quantised on the way
    y = h + experts(norm(h))        # moe_mxfp4: routing and the chosen experts in one kernel

and compares the last one with the same block computed by the library's fp32
product on the values that the 4-bit weights stand for.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import memory_hierarchy_reuse_gb300 as mhr  # noqa: E402


def norm(x):
    x = x.float()
    return (x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)).bfloat16()


class Block:
    """Weights in 4 bits, and the values that they stand for (for the comparison)."""

    def __init__(self, hidden, inner, experts, top):
        def normal(rows, cols):
            return torch.randn(rows, cols, device="cuda") * cols ** -0.5

        self.top, self.inner = top, inner
        # a K x N projection, blocks along K; experts' rows as the layer takes them
        self.proj, self.proj_v = mhr.quantize_mxfp4(normal(hidden, hidden), axis=0, values=True)
        self.up, self.up_v = mhr.quantize_mxfp4(normal(2 * experts * inner, hidden), values=True)
        self.down, self.down_v = mhr.quantize_mxfp4(normal(experts * hidden, inner), values=True)
        self.router = normal(experts, hidden).bfloat16()

    def step(self, x):
        h = x + mhr.matmul_mxfp4(x, self.proj, out_dtype=torch.bfloat16)
        y, experts, weights = mhr.moe_mxfp4(norm(h), self.router, self.up, self.down, self.top)
        return h + y, h, experts, weights

    def plain_step(self, x, experts, weights):
        _, xv = mhr.quantize_mxfp4(x, values=True)
        h = x + mhr.matmul(xv.float(), self.proj_v).bfloat16()
        n, hidden, inner = norm(h).float(), x.shape[1], self.inner
        y = torch.zeros(h.shape, device="cuda")
        for t in range(x.shape[0]):
            for e, w in zip(experts[t].tolist(), weights[t].tolist()):
                up = self.up_v[2 * e * inner:2 * (e + 1) * inner].t().contiguous()
                gate, value = mhr.matmul(n[t:t + 1], up).split(inner, 1)
                down = self.down_v[e * hidden:(e + 1) * hidden].t().contiguous()
                y[t] += w * mhr.matmul(torch.nn.functional.silu(gate) * value, down)[0]
        return h + y.bfloat16()


def main(tokens=4, steps=20, hidden=1024, inner=512, experts=32, top=4):
    torch.manual_seed(0)
    block = Block(hidden, inner, experts, top)
    x = torch.randn(tokens, hidden, device="cuda").bfloat16()
    block.step(x)
    start, stop = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    start.record()
    for _ in range(steps):
        out, _, experts_of, weights = block.step(x)
    stop.record()
    torch.cuda.synchronize()
    status = mhr.gemm_check(torch.cuda.current_stream().cuda_stream)
    assert status == mhr.MHR_OK, mhr.gemm_status_string(status)
    want = block.plain_step(x, experts_of, weights)
    err = float((out.float() - want.float()).norm() / want.float().norm())
    print(f"{tokens} tokens: {start.elapsed_time(stop) * 1e3 / steps:.1f} us a step, "
          f"relative difference from the plain block {err:.2e}")
    return err


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--tokens", type=int, default=4)
    ap.add_argument("--steps", type=int, default=20)
    a = ap.parse_args()
    sys.exit(0 if main(a.tokens, a.steps) < 1e-2 else 1)
