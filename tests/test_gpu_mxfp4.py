"""Quantisation to MXFP4 and its products on the GPU, against 64-bit numpy (mxfp4_ref)."""
import numpy as np
import pytest

import mxfp4_ref as ref

pytestmark = pytest.mark.gpu


def torch_dtype(name):
    import torch

    return {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}[name]


def wild(rows, cols, dtype, seed):
    """Values over the type's whole range, by random bits: normal, subnormal and zero ones,
    blocks of one size and of many, ties between codes; no infinities or NaNs."""
    import torch

    rng = np.random.default_rng(seed)
    x = rng.standard_normal((rows, cols))
    kind = rng.integers(0, 6, (rows, -(-cols // 32))).repeat(32, 1)[:, :cols]
    x = np.where(kind == 0, rng.integers(-28, 29, (rows, cols)) / 4, x)  # multiples of 1/4: ties
    x = np.where(kind == 1, 0.0, x)
    spread = {"f32": 148, "bf16": 132, "f16": 23}[dtype]
    top = {"f32": 120, "bf16": 120, "f16": 12}[dtype]
    x = np.where(kind == 2, x * np.exp2(rng.integers(-spread, top, (rows, cols))), x)
    x = np.where(kind == 3, x * np.exp2(-float(spread)), x)
    return torch.from_numpy(x).to(torch_dtype(dtype))


def check_quantized(mhr, x, axis, **kw):
    """Codes, scales and values of x, all equal to the definition's."""
    q, v = mhr.quantize_mxfp4(x, axis=axis, values=True, **kw)
    assert mhr.gemm_check(None) == mhr.MHR_OK
    x64 = x.double().cpu().numpy()
    x64 = x64 if axis == 1 else x64.T
    codes, scales = ref.quantize(x64)
    data, tiled = ref.pack(codes, scales)
    assert (q.rows, q.cols) == x64.shape
    assert np.array_equal(q.scales.cpu().numpy(), tiled)  # its zero padding too
    got = q.data.cpu().numpy()
    # the sign of a zero code is free
    bare = lambda d: np.where((d & 7) == 0, d & 0xF0, d) & np.where((d & 0x70) == 0, 0x0F, 0xFF)  # noqa: E731
    assert np.array_equal(bare(got), bare(data))
    want = ref.values(codes, scales, x64.shape[1])
    v = v.double().cpu().numpy()
    assert np.array_equal(v if axis == 1 else v.T, want, equal_nan=True)


SHAPES = [(1, 1), (1, 32), (3, 31), (1, 4096), (5, 33), (129, 160), (64, 1056), (200, 257), (31, 2000),
          (130, 1023)]


@pytest.mark.parametrize("axis", [1, 0])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_quantize(mhr, rows, cols, dtype, axis):
    check_quantized(mhr, wild(rows, cols, dtype, rows * 7 + cols).cuda(), axis)


@pytest.mark.parametrize("axis", [1, 0])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_quantize_strided_and_unaligned(mhr, dtype, axis):
    import torch

    big = wild(70, 1100, dtype, 5).cuda()
    check_quantized(mhr, big[:, :1000], axis)      # a pitch of 1100
    check_quantized(mhr, big[3:50, 1:700], axis)   # rows off 16 (and 4) bytes
    check_quantized(mhr, big[::2, 8:1032], axis)   # every second row
    flat = torch.zeros(64 * 999 + 1, dtype=big.dtype, device="cuda")
    x = flat[1:].view(64, 999)
    x.copy_(big[:64, :999])
    check_quantized(mhr, x, axis)


@pytest.mark.parametrize("axis", [1, 0])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_quantize_infinities_and_nans(mhr, dtype, axis):
    """A block that holds one is NaN whole; its neighbours are untouched."""
    x = wild(96, 160, dtype, 9)
    x[3, 40], x[33, 7], x[50, 159], x[51, 0] = float("inf"), float("nan"), float("-inf"), float("nan")
    check_quantized(mhr, x.cuda(), axis)


def test_quantize_extremes(mhr):
    import torch

    tiny, huge = np.float32(1e-45), np.finfo(np.float32).max
    rows = [[0.0] * 32, [-0.0] * 32, [tiny] * 32, [huge] * 31 + [tiny], [2.0 ** -126] * 32,
            [2.0 ** -125, 2.0 ** -126, 2.0 ** -127, 2.0 ** -128, 2.0 ** -129] + [0.0] * 27,
            [7.9999995, 5.0, 4.9999995, 3.5, 2.5, 1.75, 1.25, 0.75, 0.25, 0.24999999] + [0.25000003] * 22]
    check_quantized(mhr, torch.tensor(rows, dtype=torch.float32).cuda(), 1)


def product_case(mhr, M, N, K, dtype, seed=0, ldc=None, offset=0, lda=None, **kw):
    """gemm_mxfp4 on uniform codes against 64 bits; C's padding must stay untouched."""
    import torch

    a, sa, av = ref.random_packed(M, K, seed + 1)
    b, sb, bv = ref.random_packed(N, K, seed + 2)
    S = np.abs(av) @ np.abs(bv).T
    want = av @ bv.T
    if lda:
        wide = np.full((M, lda), 0x77, np.uint8)
        wide[:, :a.shape[1]] = a
        a = wide
    A = mhr.MxFp4Matrix(torch.from_numpy(a).cuda(), torch.from_numpy(sa).cuda(), M, K)
    B = mhr.MxFp4Matrix(torch.from_numpy(b).cuda(), torch.from_numpy(sb).cuda(), N, K)
    ldc = ldc or N
    buf = torch.full((M * ldc + offset,), 7.0, dtype=torch_dtype(dtype), device="cuda")
    out = torch.as_strided(buf, (M, N), (ldc, 1), offset)
    mhr.matmul_mxfp4(A, B, out=out, **kw)
    assert mhr.gemm_check(None) == mhr.MHR_OK
    err = np.abs(out.double().cpu().numpy() - want)
    bound = ref.product_bound(K, S, want, dtype)
    assert np.all(err <= bound), float((err / bound).max())
    full = buf.float().cpu().numpy()
    written = np.zeros(full.shape, bool)
    idx = offset + np.arange(M)[:, None] * ldc + np.arange(N)
    written[idx] = True
    assert np.all(full[~written] == 7.0)
    return out


PRODUCTS = [(1, 1, 1), (1, 128, 64), (1, 4096, 4096), (2, 130, 32), (7, 257, 96), (8, 64, 8192),
            (16, 1000, 300), (33, 128, 2048), (64, 384, 511), (127, 129, 1000), (128, 128, 128),
            (129, 200, 260), (200, 333, 777), (256, 256, 256), (300, 520, 2000), (257, 513, 64),
            (512, 768, 1056), (1000, 1111, 640)]


@pytest.fixture(params=[0, 1, 2], ids=["auto", "narrow", "pair"])
def kernel(mhr, request):
    """The product's kernel: the library's choice, and each of them for every shape."""
    old = mhr.gemm_testing_set_cta_pair_mode(request.param)
    yield request.param
    mhr.gemm_testing_set_cta_pair_mode(old)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("M,N,K", PRODUCTS)
def test_product(mhr, kernel, M, N, K, dtype):
    product_case(mhr, M, N, K, dtype, seed=M + N + K)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_product_of_many_tiles(mhr, kernel, dtype):
    """More tiles than run at once: accumulators alternate, ragged last ones."""
    product_case(mhr, 2600, 3300, 300, dtype)


@pytest.mark.parametrize("width", [128, 192, 256])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_product_tile_widths(mhr, width, dtype):
    """The pair kernel at every tile width, aligned and unaligned C, several tiles a pair."""
    old_mode = mhr.gemm_testing_set_cta_pair_mode(2)
    old = mhr.gemm_testing_set_pair_tile_n(width)
    try:
        product_case(mhr, 300, 1000, 776, dtype)
        product_case(mhr, 300, 1001, 776, dtype, ldc=1003, offset=1)
        product_case(mhr, 2100, 2560, 640, dtype)
        assert f"<n{width}>" in mhr.gemm_testing_last_main_kernel()
    finally:
        mhr.gemm_testing_set_pair_tile_n(old)
        mhr.gemm_testing_set_cta_pair_mode(old_mode)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("M,N,K", [(2300, 2300, 300), (4000, 2500, 300), (4000, 2428, 1100)])
def test_product_last_round_in_halves(mhr, M, N, K, dtype):
    """Tiles of 256 columns over one and two rounds (81 and 160 of them on 76 pairs), and the
    halves of what is left: on either accumulator, one of them past the last column."""
    old_mode = mhr.gemm_testing_set_cta_pair_mode(2)
    old = mhr.gemm_testing_set_pair_tile_n(256)
    try:
        product_case(mhr, M, N, K, dtype)
    finally:
        mhr.gemm_testing_set_pair_tile_n(old)
        mhr.gemm_testing_set_cta_pair_mode(old_mode)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("M,N,K", [(5, 200, 300), (140, 200, 300), (300, 260, 520)])
def test_product_strides_and_offsets(mhr, kernel, M, N, K, dtype):
    product_case(mhr, M, N, K, dtype, ldc=N + 3, offset=1)
    product_case(mhr, M, N, K, dtype, ldc=N + 8, offset=8, lda=-(-K // 32) * 16 + 48)


@pytest.mark.parametrize("M", [3, 200, 520])
def test_product_repeats_bit_for_bit(mhr, kernel, M):
    import torch

    first = product_case(mhr, M, 384, 4096, "f32").clone()
    for _ in range(3):
        assert torch.equal(product_case(mhr, M, 384, 4096, "f32"), first)


def test_product_integers_are_exact(mhr, kernel):
    """Codes of whole values and scales of 1: every sum is a whole number below 2^24."""
    import torch

    rng = np.random.default_rng(3)
    for M, N, K in [(9, 300, 4096), (300, 300, 4096), (520, 600, 1024)]:
        pick = np.array([0, 2, 4, 5, 6, 7, 10, 12, 13, 14, 15], np.uint8)
        qa, qb = (pick[rng.integers(0, 11, (r, K))] for r in (M, N))
        ones = lambda r: np.full((r, K // 32), 127, np.uint8)  # noqa: E731
        A, B = (mhr.MxFp4Matrix(*(torch.from_numpy(t).cuda() for t in ref.pack(q, ones(r))), r, K)
                for q, r in ((qa, M), (qb, N)))
        want = ref.values(qa, ones(M), K) @ ref.values(qb, ones(N), K).T
        assert np.array_equal(mhr.matmul_mxfp4(A, B).double().cpu().numpy(), want)


def test_product_scales_reach_every_block(mhr, kernel):
    """One nonzero block per row, each with a scale of its own."""
    import torch

    for M, N in [(40, 160), (300, 400)]:
        K = 2080
        blocks = K // 32
        av, bv = np.zeros((M, K), np.uint8), np.zeros((N, K), np.uint8)
        sa, sb = np.full((M, blocks), 127, np.uint8), np.full((N, blocks), 127, np.uint8)
        for i in range(M):
            av[i, (i % blocks) * 32:(i % blocks) * 32 + 32] = 2
            sa[i, i % blocks] = 100 + i % 50
        bv[:] = 2
        sb[:] = 110 + (np.arange(N)[:, None] * 7 + np.arange(blocks) * 3) % 30
        A = mhr.MxFp4Matrix(*(torch.from_numpy(t).cuda() for t in ref.pack(av, sa)), M, K)
        B = mhr.MxFp4Matrix(*(torch.from_numpy(t).cuda() for t in ref.pack(bv, sb)), N, K)
        want = ref.values(av, sa, K) @ ref.values(bv, sb, K).T
        assert np.array_equal(mhr.matmul_mxfp4(A, B).double().cpu().numpy(), want)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("M,N,K", [(1, 512, 1000), (5, 77, 4096), (17, 130, 33), (32, 300, 9000),
                                   (33, 200, 512), (9, 40, 33000), (48, 300, 600), (333, 500, 1032)])
def test_product_quantized_on_the_way(mhr, M, N, K, dtype):
    """The same C, bit for bit, as quantising first; a strided, unaligned A."""
    import torch

    x = wild(M, K + 5, dtype, M).clamp(-100, 100).cuda()[:, 3:K + 3]
    b, sb, _ = ref.random_packed(N, K, 4)
    B = mhr.MxFp4Matrix(torch.from_numpy(b).cuda(), torch.from_numpy(sb).cuda(), N, K)
    want = mhr.matmul_mxfp4(mhr.quantize_mxfp4(x), B)
    got = mhr.matmul_mxfp4(x, B)
    assert mhr.gemm_check(None) == mhr.MHR_OK
    assert torch.equal(got, want) and bool(torch.isfinite(got).all())


def test_product_nan_scale_reaches_its_rows_only(mhr, kernel):
    import torch

    for M in (40, 300):
        x = torch.randn(M, 256, device="cuda")
        x[17, 40] = float("inf")
        B = mhr.quantize_mxfp4(torch.randn(256, 300, device="cuda"), axis=0)
        c = mhr.matmul_mxfp4(x, B)
        nan = torch.isnan(c)
        assert bool(nan[17].all()) and int(nan.sum()) == 300


def test_product_zero_k_and_empty(mhr):
    import torch

    e = torch.empty((0,), dtype=torch.uint8, device="cuda")
    A = mhr.MxFp4Matrix(e.view(0, 0).new_empty((4, 0)), e, 4, 0)
    B = mhr.MxFp4Matrix(e.new_empty((6, 0)), e, 6, 0)
    out = torch.full((4, 6), 3.0, device="cuda", dtype=torch.bfloat16)
    mhr.matmul_mxfp4(A, B, out=out)
    assert bool((out == 0).all())
    assert mhr.quantize_mxfp4(torch.empty((0, 64), device="cuda")).rows == 0
    B = mhr.quantize_mxfp4(torch.randn(64, 6, device="cuda"), axis=0)
    assert mhr.matmul_mxfp4(torch.empty((0, 64), device="cuda"), B).shape == (0, 6)


def test_quantized_product_matches_plain_product(mhr):
    """A whole layer: values of both operands multiplied by the library's fp32 product."""
    import torch

    x, w = torch.randn(70, 640, device="cuda"), torch.randn(640, 333, device="cuda")
    qx, xv = mhr.quantize_mxfp4(x, values=True)
    qw, wv = mhr.quantize_mxfp4(w, axis=0, values=True)
    got, want = mhr.matmul_mxfp4(qx, qw), mhr.matmul(xv, wv)
    S = xv.abs().double() @ wv.abs().double()
    # two fp32 sums of the same exact products, each within (K + 8) 2^-23 S
    assert bool(((got - want).abs() <= 2 * (640 + 8) * 2.0 ** -23 * S).all())


def test_offsets_past_32_bits(mhr):
    """Rows more than 2^32 bytes apart in x, the values, the packed data and C."""
    import torch

    far = 2_300_000_000
    x = torch.empty(far + 4096, dtype=torch.bfloat16, device="cuda").as_strided((2, 700), (far, 1))
    near = torch.randn(2, 700, device="cuda").bfloat16()
    x.copy_(near)
    for axis in (1, 0):
        q, v = mhr.quantize_mxfp4(x, axis=axis, values=True)
        want, wv = mhr.quantize_mxfp4(near, axis=axis, values=True)
        assert torch.equal(q.data, want.data) and torch.equal(q.scales, want.scales)
        assert torch.equal(v, wv)
    del x
    qa, qb = mhr.quantize_mxfp4(torch.randn(300, 700, device="cuda")), mhr.quantize_mxfp4(torch.randn(2, 700, device="cuda"))
    want = mhr.matmul_mxfp4(qa, qb)
    wide = torch.empty(2 * far + 4096, dtype=torch.uint8, device="cuda").as_strided((2, 352), (2 * far // 16 * 16, 1))
    wide.copy_(qb.data)
    b = mhr.MxFp4Matrix(wide, qb.scales, 2, 700)
    assert torch.equal(mhr.matmul_mxfp4(qa, b), want)
    got = mhr.matmul_mxfp4(b, qa)
    out = torch.empty(far + 4096, dtype=torch.float32, device="cuda").as_strided((2, 300), (far, 1))
    for a in (b, qb):
        out.zero_()
        assert torch.equal(mhr.matmul_mxfp4(a, qa, out=out), got)
    assert torch.allclose(got, want.t(), rtol=1e-5, atol=1e-5 * float(want.abs().max()))


def test_graph_capture(mhr):
    """Quantisation, and products that need no workspace, replay from a CUDA graph."""
    import torch

    x = torch.randn(16, 1024, device="cuda").bfloat16()
    big = torch.randn(300, 1024, device="cuda").bfloat16()
    B = mhr.quantize_mxfp4(torch.randn(1024, 384, device="cuda"), axis=0)

    def step():
        return mhr.matmul_mxfp4(x, B), mhr.matmul_mxfp4(mhr.quantize_mxfp4(big), B)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for seed in (1, 2):
        torch.manual_seed(seed)
        x.copy_(torch.randn_like(x))
        big.copy_(torch.randn_like(big))
        graph.replay()
        want = step()
        torch.cuda.synchronize()
        assert all(torch.equal(g, w) for g, w in zip(got, want))


def test_another_device_stream_argument(mhr):
    """A raw stream handle in place of the current stream."""
    import torch

    x = torch.randn(40, 512, device="cuda")
    B = mhr.quantize_mxfp4(torch.randn(512, 96, device="cuda"), axis=0)
    want = mhr.matmul_mxfp4(x, B)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out = torch.empty_like(want)
    mhr.matmul_mxfp4(x, B, out=out, stream=s.cuda_stream)
    s.synchronize()
    assert torch.equal(out, want)


def test_streams(mhr):
    """Calls on several streams at once, each with its own packed activations."""
    import torch

    B = mhr.quantize_mxfp4(torch.randn(512, 640, device="cuda"), axis=0)
    xs = [torch.randn(24 + 100 * i, 512, device="cuda") for i in range(4)]
    want = [mhr.matmul_mxfp4(x, B) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    got = []
    for _ in range(5):
        got = []
        for x, s in zip(xs, streams):
            with torch.cuda.stream(s):
                got.append(mhr.matmul_mxfp4(x, B))
    torch.cuda.synchronize()
    assert all(torch.equal(g, w) for g, w in zip(got, want))


def test_timeout_is_reported_and_cleared(mhr, kernel):
    """A first ring stage that is never filled: the call ends, the status says so, and the next
    call is right."""
    import torch

    A = mhr.quantize_mxfp4(torch.randn(20, 1024, device="cuda"))
    B = mhr.quantize_mxfp4(torch.randn(1024, 256, device="cuda"), axis=0)
    want = mhr.matmul_mxfp4(A, B)
    old = mhr.gemm_testing_set_wait_limit_ns(20_000_000)
    mhr.gemm_testing_set_inject_stall(1)
    try:
        mhr.matmul_mxfp4(A, B)
        assert mhr.gemm_check(None) == mhr.MHR_ERR_TIMEOUT
    finally:
        mhr.gemm_testing_set_inject_stall(0)
        mhr.gemm_testing_set_wait_limit_ns(old)
    assert torch.equal(mhr.matmul_mxfp4(A, B), want)
    assert mhr.gemm_check(None) == mhr.MHR_OK
