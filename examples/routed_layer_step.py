"""One training step of a small mixture-of-experts layer, written out by hand.

    python examples/routed_layer_step.py [--tokens 512]

    p_t, e_t = the router's weights and experts of token t   # choose_experts, sort_by_expert
    y_t      = sum over j of p_tj  relu(x_t up_e) down_e      # matmul_experts
    out_t    = y_t + (x_t a_t^T) b_t                          # add_adapters

and the way back from the gradient of out to those of x, the router and the experts
(the adapters are held fixed). Returns the results, for a comparison.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import memory_hierarchy_reuse_gb300 as mhr  # noqa: E402


class Layer:
    def __init__(self, hidden, inner, experts, top, adapters, rank):
        def normal(*shape):
            return (torch.randn(*shape, device="cuda") * shape[-2] ** -0.5).bfloat16()

        self.top, self.experts = top, experts
        self.router = torch.randn(hidden, experts, device="cuda") * hidden ** -0.5
        self.bias = torch.zeros(experts, device="cuda")
        self.up, self.down = normal(experts, hidden, inner), normal(experts, inner, hidden)
        self.a, self.b = normal(adapters, rank, hidden), normal(adapters, rank, hidden)

    def forward(self, x, which):
        s = {"x": x, "which": which}
        s["logits"] = mhr.matmul(x.float(), self.router, path="3xtf32")
        s["chosen"], s["p"] = mhr.choose_experts(s["logits"], self.top, "sigmoid", self.bias)
        s["offsets"], s["order"] = mhr.sort_by_expert(s["chosen"], self.experts)
        at, order = s["offsets"], s["order"]
        # rows in the experts' order between the products, in (token, slot) order after them
        s["h"] = mhr.matmul_experts(x, self.up, at, gather=order, top=self.top).relu_()
        s["each"] = mhr.matmul_experts(s["h"], self.down, at, scatter=order)
        y = (s["each"].view(len(x), self.top, -1) * s["p"][:, :, None]).sum(1)
        return mhr.add_adapters(y, x, self.a, self.b, which), s

    def backward(self, d_out, s):
        """The gradients of x, the router, up and down."""
        x, top, at, order = s["x"], self.top, s["offsets"], s["order"]
        T, hidden = x.shape
        dp = (s["each"].view(T, top, -1) * d_out[:, None]).sum(2)
        d_each = (d_out[:, None] * s["p"][:, :, None]).to(x.dtype).view(T * top, hidden)
        d_down = mhr.matmul_experts_grad(s["h"], d_each, at, scatter=order, out_dtype=torch.float32)
        dh = mhr.matmul_experts(d_each, self.down, at, gather=order, transposed=True)
        dh *= s["h"] > 0
        d_up = mhr.matmul_experts_grad(x, dh, at, gather=order, top=top, out_dtype=torch.float32)
        dx = mhr.matmul_experts(dh, self.up, at, scatter=order, transposed=True,
                                out_dtype=torch.float32).view(T, top, hidden).sum(1)
        d_logits = mhr.choose_experts_grad(s["logits"], s["chosen"], dp, "sigmoid")
        dx += mhr.matmul(d_logits, self.router.t().contiguous(), path="3xtf32")
        # the adapters' part, with the two matrices' places changed
        dx = mhr.add_adapters(dx, d_out.to(x.dtype), self.b, self.a, s["which"])
        d_router = mhr.matmul(x.float().t().contiguous(), d_logits, path="3xtf32")
        return dx, d_router, d_up, d_down


def main(tokens=512, hidden=256, inner=384, experts=16, top=4, adapters=3, rank=8):
    torch.manual_seed(0)
    layer = Layer(hidden, inner, experts, top, adapters, rank)
    x = torch.randn(tokens, hidden, device="cuda").bfloat16()
    which = torch.randint(-1, adapters, (tokens,), device="cuda", dtype=torch.int32)
    out, saved = layer.forward(x, which)
    d_out = torch.randn_like(out)
    grads = layer.backward(d_out, saved)
    status = mhr.gemm_check(torch.cuda.current_stream().cuda_stream)
    assert status == mhr.MHR_OK, mhr.gemm_status_string(status)
    load = saved["offsets"].diff()
    print(f"{tokens} tokens, {top} of {experts} experts: {int(load.min())} to {int(load.max())} "
          f"rows an expert, gradient norms " + " ".join(f"{float(g.norm()):.3g}" for g in grads))
    return layer, x, which, d_out, out, saved, grads


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--tokens", type=int, default=512)
    main(ap.parse_args().tokens)
