"""Edges of the 4-bit products: what can be captured, calls that start early, pitches past 2^31 bytes."""
import pytest

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("N", [1, 130, 40000])
@pytest.mark.parametrize("M,K", [(1, 4096), (3, 4096), (8, 1536), (12, 1024), (16, 768), (25, 512), (32, 256)])
def test_small_quantized_products_can_be_captured(mhr, M, K, N):
    """The rule that the header gives: K <= 4096, at most 32 rows, rows x ceil(K / 256) <= 50."""
    import torch

    assert K <= 4096 and M <= 32 and M * -(-K // 256) <= 50
    x = torch.randn(M, K, device="cuda").bfloat16()
    B = mhr.quantize_mxfp4(torch.randn(N, K, device="cuda"))
    mhr.matmul_mxfp4(x, B)
    mhr.gemm_release()  # no workspace is left that a captured call could take
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = mhr.matmul_mxfp4(x, B)
    x.copy_(torch.randn_like(x))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got, mhr.matmul_mxfp4(x, B))


def test_calls_with_a_workspace_are_refused_in_a_capture(mhr):
    """A graph would keep the address of a workspace that later calls may free. The capture goes on."""
    import torch

    E, H, I = 4, 256, 64
    big, x = torch.randn(300, 1024, device="cuda"), torch.randn(2, H, device="cuda").bfloat16()
    B = mhr.quantize_mxfp4(torch.randn(130, 1024, device="cuda"))
    up = mhr.quantize_mxfp4(torch.randn(2 * E * I, H, device="cuda"))
    down = mhr.quantize_mxfp4(torch.randn(E * H, I, device="cuda"))
    router = torch.randn(E, H, device="cuda").bfloat16()
    want = mhr.moe_mxfp4(x, router, up, down, 2)[0], mhr.matmul_mxfp4(big, B)
    torch.cuda.synchronize()
    for mode in ("global", "relaxed"):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, capture_error_mode=mode):
            with pytest.raises(mhr.GemmError):
                mhr.moe_mxfp4(x, router, up, down, 2)
            with pytest.raises(mhr.GemmError):
                mhr.matmul_mxfp4(big, B)
            got = mhr.matmul_mxfp4(mhr.quantize_mxfp4(big), B)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, want[1])
    assert torch.equal(mhr.moe_mxfp4(x, router, up, down, 2)[0], want[0])
    assert torch.equal(mhr.matmul_mxfp4(big, B), want[1])
    assert mhr.gemm_check(None) == mhr.MHR_OK


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


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_zero_k_with_rows_far_apart(mhr, dtype):
    import torch

    far = 2_300_000_000
    buf = torch.empty(far + 4096, dtype=getattr(torch, dtype), device="cuda")
    out = buf.as_strided((2, 300), (far, 1))
    out.fill_(3)
    buf[300:600] = 5
    e = torch.empty((0,), dtype=torch.uint8, device="cuda")
    A, B = (mhr.MxFp4Matrix(e.new_empty((n, 0)), e, n, 0) for n in (2, 300))
    mhr.matmul_mxfp4(A, B, out=out)
    assert bool((out == 0).all()) and bool((buf[300:600] == 5).all())
    out.fill_(3)
    mhr.matmul_mxfp4(torch.empty((2, 0), device="cuda"), B, out=out)
    assert bool((out == 0).all()) and bool((buf[300:600] == 5).all())
