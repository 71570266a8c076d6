"""A result's type that is given twice has to be the same, without a GPU."""
import pytest


@pytest.fixture(scope="module")
def mhr():
    from memory_hierarchy_reuse_gb300 import build as b

    b.build()
    import memory_hierarchy_reuse_gb300 as m

    m.load()
    return m


def test_out_and_out_dtype_that_differ(mhr):
    import torch

    x, w = torch.zeros(4, 16, dtype=torch.bfloat16), torch.zeros(2, 16, 8, dtype=torch.bfloat16)
    offsets, out = torch.zeros(3, dtype=torch.int32), torch.zeros(4, 8)
    grad = torch.zeros(2, 16, 16)
    with pytest.raises(TypeError, match="out must be of out_dtype"):
        mhr.matmul_experts(x, w, offsets, out=out, out_dtype=torch.bfloat16)
    with pytest.raises(TypeError, match="out must be of out_dtype"):
        mhr.matmul_experts_grad(x, x, offsets, out=grad, out_dtype=torch.float16)
    with pytest.raises(TypeError, match="out_dtype must be"):
        mhr.matmul_experts(x, w, offsets, out=out, out_dtype=torch.int32)
    # as given, or the same: the next check is the device's
    for dtype in (None, torch.float32):
        with pytest.raises(ValueError, match="CUDA"):
            mhr.matmul_experts(x, w, offsets, out=out, out_dtype=dtype)
        with pytest.raises(ValueError, match="CUDA"):
            mhr.matmul_experts_grad(x, x, offsets, out=grad, out_dtype=dtype)
