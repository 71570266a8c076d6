"""Edges of the 4-bit products: calls that start early."""
import pytest

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows,size", [(1, 256), (4, 512), (1, 4096)])
def test_products_that_read_what_the_call_before_wrote(mhr, rows, size):
    """A chain over two buffers, whose kernels start before the ones in front of them have ended:
    the same, bit for bit, as with a wait after every call."""
    import torch

    B = mhr.quantize_mxfp4(torch.randn(size, size, device="cuda") * 1.5 * size ** -0.5)
    start = torch.randn(rows, size, device="cuda").bfloat16()

    def chain(wait):
        buf = [start.clone(), torch.zeros_like(start)]
        kept = []
        for i in range(40):
            mhr.matmul_mxfp4(buf[i % 2], B, out=buf[(i + 1) % 2])
            if wait:
                torch.cuda.synchronize()
            if i % 8 == 7:
                kept.append(buf[(i + 1) % 2].clone())
        torch.cuda.synchronize()
        return torch.stack(kept)

    want = chain(True)
    assert bool(torch.isfinite(want).all()) and bool((want[-1] != 0).any())
    for _ in range(20):
        assert torch.equal(chain(False), want)


@pytest.mark.parametrize("size", [96, 256])
def test_dense_products_of_what_the_call_before_wrote(mhr, size):
    """The same with the one-launch fp32 product, which splits its operands as it loads them, behind
    a quantisation whose values it multiplies."""
    import torch

    w = torch.randn(size, size, device="cuda") * size ** -0.5
    start = torch.randn(size, size, device="cuda")

    def chain(wait):
        buf = [start.clone(), torch.zeros_like(start)]
        kept = []
        for i in range(40):
            v = mhr.quantize_mxfp4(buf[i % 2], values=True)[1]
            if wait:
                torch.cuda.synchronize()
            a, b = (w, v) if i % 4 < 2 else (v, w)
            mhr.matmul(a, b, "3xtf32", out=buf[(i + 1) % 2])
            if wait:
                torch.cuda.synchronize()
            if i % 8 == 7:
                kept.append(buf[(i + 1) % 2].clone())
        torch.cuda.synchronize()
        return torch.stack(kept)

    want = chain(True)
    assert bool(torch.isfinite(want).all()) and bool((want[-1] != 0).any())
    for _ in range(20):
        assert torch.equal(chain(False), want)
