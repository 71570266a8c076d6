"""The compiled tensor-level calls of the 4-bit operators, without a GPU."""
import pytest


def test_values_without_a_truth_value(mhr_cpu):
    """The error of an argument that has no truth value is the caller's to see."""
    import torch

    class Neither:
        def __bool__(self):
            raise ArithmeticError("neither")

    with pytest.raises(ArithmeticError, match="neither"):
        mhr_cpu.quantize_mxfp4(torch.zeros(4, 64), values=Neither())


@pytest.fixture(scope="module")
def mhr_cpu():
    from memory_hierarchy_reuse_gb300 import build as b

    b.build()
    import memory_hierarchy_reuse_gb300 as m

    return m
