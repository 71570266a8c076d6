"""Calls by an index per row at the edges of what include/mhr_routed.h states, against 64-bit numpy."""
import numpy as np
import pytest

import routed_ref as ref

pytestmark = pytest.mark.gpu


def types():
    import torch

    return {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def f64(t):
    return t.double().cpu().numpy()


def same(got, want):
    """got is want (float64) rounded to got's type, infinities and NaN in their places."""
    import torch

    want = torch.from_numpy(want).to(got.dtype)
    assert torch.equal(got.cpu().nan_to_num(nan=0.0, posinf=1e38, neginf=-1e38),
                       want.nan_to_num(nan=0.0, posinf=1e38, neginf=-1e38))
    assert torch.equal(got.cpu().isnan(), want.isnan())


@pytest.mark.parametrize("T", [6, 300, 700])
@pytest.mark.parametrize("rank", [3, 100])
@pytest.mark.parametrize("dtype,out", [("bf16", "bf16"), ("bf16", "f16"), ("bf16", "f32"),
                                       ("f16", "f16"), ("f16", "bf16"), ("f16", "f32")])
def test_the_sum_between_an_adapters_products_is_held_to_22_bits(mhr, T, rank, dtype, out):
    """v = (2^15 + 2^5 + 2^-5, 2^15, 2^5) against up = (1, -1, -1): what is left is 2^-5, the last
    of v's 21 bits. All sums are exact in fp32."""
    import torch

    K, N = 64, 72
    x = torch.zeros(T, K)
    x[:, 3], x[:, 40], x[:, 63] = 2.0 ** 15, 2.0 ** 5, 2.0 ** -5
    x *= 2.0 ** -(torch.arange(T) % 8)[:, None]
    down, up = torch.zeros(2, rank, K), torch.zeros(2, rank, N)
    a, b, c = 0, rank // 2, rank - 1
    down[:, a, 3] = down[:, a, 40] = down[:, a, 63] = down[:, b, 3] = down[:, c, 40] = 1
    up[:, a], up[:, b], up[:, c] = 1, -1, -1
    x, down, up = (t.to(types()[dtype]).cuda() for t in (x, down, up))
    y = torch.zeros(T, N, dtype=types()[out], device="cuda")
    which = (torch.arange(T, dtype=torch.int32, device="cuda") // 5) % 2
    got = mhr.add_adapters(y, x, down, up, which)
    want = ref.adapters(f64(y), f64(x), f64(down), f64(up), which.cpu().numpy())
    assert want.min() == 2.0 ** (-5 - min(T - 1, 7)) and want.max() == 2.0 ** -5
    same(got, want)
