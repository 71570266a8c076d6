"""The operators that go by an index per row together, as the example runs them."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("tokens", [1, 37, 700])
def test_layer_step(mhr, tokens):
    """Against automatic differentiation in 64 bits with the same choice. Between x and a result
    lie at most five roundings to bf16 (h, the experts' outputs, their gradients, dh, the output's
    gradient), each within 2^-8 of a value; maps that mix many such values leave the ratio of the
    norms where it is, twice it is allowed for those that do not."""
    import torch

    spec = importlib.util.spec_from_file_location(
        "routed_layer_step", os.path.join(ROOT, "examples", "routed_layer_step.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    layer, x, which, d_out, out, saved, grads = example.main(tokens=tokens)
    leaves = [t.double().cpu().requires_grad_() for t in (x, layer.router, layer.up, layer.down)]
    xd, router, up, down = leaves
    chosen, w = saved["chosen"].long().cpu(), which.long().cpu()
    s = torch.sigmoid(xd @ router).gather(1, chosen)
    p = s / s.sum(1, keepdim=True)
    # (relu's side as the 16-bit values have it: its gradient jumps there)
    h = torch.empty(chosen.numel(), up.shape[2], dtype=torch.float64)
    h[saved["order"].long().cpu()] = (saved["h"] > 0).double().cpu()
    h = h.view(*chosen.shape, -1) * torch.einsum("tk,tjkn->tjn", xd, up[chosen])
    y = (torch.einsum("tjn,tjnk->tjk", h, down[chosen]) * p[:, :, None]).sum(1)
    a, b = layer.a.double().cpu()[w.clamp(min=0)], layer.b.double().cpu()[w.clamp(min=0)]
    v = torch.einsum("tk,trk->tr", xd, a) * (w >= 0)[:, None]
    want = y + torch.einsum("tr,trk->tk", v, b)
    want.backward(d_out.double().cpu())
    for got, ref in zip((out, *grads), (want.detach(), *(t.grad for t in leaves))):
        err = float((got.double().cpu() - ref).norm() / ref.norm())
        assert err < 2 * 5 * 2.0 ** -8, err
