"""The experts' products and their weights' gradient on the GPU, against 64-bit numpy.

Most inputs are whole numbers of at most 3 whose sums stay below 2^24: fp32 holds every partial
sum, in any order, so results are equal to the last bit -- to the one rounding of the output type.
"""
import numpy as np
import pytest

import routed_ref as ref

pytestmark = pytest.mark.gpu

HALF_STEP = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}


def types():
    import torch

    return {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def whole(shape, dtype, seed):
    import torch

    x = np.random.default_rng(seed).integers(-3, 4, shape)
    return torch.from_numpy(x).to(types()[dtype]).cuda()


def same(got, want):
    """got is want (float64) rounded to got's type."""
    import torch

    want = torch.from_numpy(want).to(got.dtype)
    assert torch.equal(got.cpu(), want), float((got.cpu().double() - want.double()).abs().max())


def f64(t):
    return t.double().cpu().numpy()


def offsets_of(counts):
    import torch

    at = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    return at, torch.from_numpy(at).cuda()


def index(values):
    import torch

    return torch.from_numpy(np.asarray(values, np.int32)).cuda()


COUNTS = [[1], [0, 0, 3], [5, 0, 1, 70], [257, 31], [33, 300, 0, 2], [1] * 40, [513, 129, 96]]


@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("counts", COUNTS, ids=str)
@pytest.mark.parametrize("K,N", [(64, 256), (8, 8), (200, 264), (72, 600)])
def test_product(mhr, counts, K, N, transposed):
    at, offsets = offsets_of(counts)
    rows, E = int(at[-1]), len(counts)
    x = whole((rows, K), "bf16", rows + K)
    w = whole((E, N, K) if transposed else (E, K, N), "bf16", N)
    want = ref.product(f64(x), f64(w), at, rows, transposed=transposed, out=np.zeros((rows, N)))
    for out_dtype in ("bf16", "f32", "f16"):
        got = mhr.matmul_experts(x, w, offsets, transposed=transposed,
                                 out_dtype=types()[out_dtype])
        assert mhr.gemm_check(None) == mhr.MHR_OK
        same(got, want)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("counts", COUNTS, ids=str)
@pytest.mark.parametrize("K,N", [(64, 256), (8, 8), (200, 264), (536, 72)])
def test_weight_grad(mhr, counts, K, N, dtype):
    at, offsets = offsets_of(counts)
    rows = int(at[-1])
    x, g = whole((rows, K), dtype, rows + K), whole((rows, N), dtype, N)
    want = ref.weight_grad(f64(x), f64(g), at)
    for out_dtype in (dtype, "f32"):
        got = mhr.matmul_experts_grad(x, g, offsets, out_dtype=types()[out_dtype])
        assert mhr.gemm_check(None) == mhr.MHR_OK
        same(got, want)


@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("T,E,top,K,N", [(1, 8, 3, 128, 256), (50, 6, 2, 72, 136),
                                         (200, 4, 3, 264, 520), (7, 128, 8, 64, 64)])
def test_routed(mhr, T, E, top, K, N, transposed):
    """Router, sort, tokens' rows picked on the way, results back in (token, slot) order, and the
    way back, as a layer runs them."""
    import torch

    x = whole((T, K), "f16", T)
    logits = torch.randn(T, E, generator=torch.Generator().manual_seed(1)).cuda()
    experts, _ = mhr.choose_experts(logits, top)
    offsets, order = mhr.sort_by_expert(experts, E)
    at, o = offsets.cpu().numpy(), order.cpu().numpy()
    R = T * top
    w = whole((E, N, K) if transposed else (E, K, N), "f16", 2)
    kw = dict(transposed=transposed)
    same(mhr.matmul_experts(x, w, offsets, gather=order, top=top, **kw),
         ref.product(f64(x), f64(w), at, R, gather=o, top=top, out=np.zeros((R, N)), **kw))
    got = mhr.matmul_experts(x, w, offsets, gather=order, scatter=order, top=top, **kw)
    want = ref.product(f64(x), f64(w), at, R, gather=o, scatter=o, top=top, out=np.zeros((R, N)), **kw)
    same(got, want)
    # (token, slot) order: each row is its token's product with its expert
    e = experts.reshape(-1).cpu().numpy()
    for r in range(0, R, 7):
        m = f64(w)[e[r]]
        assert np.array_equal(want[r], f64(x)[r // top] @ (m.T if transposed else m))
    xs = whole((R, K), "f16", 3)
    same(mhr.matmul_experts(xs, w, offsets, scatter=order, **kw),
         ref.product(f64(xs), f64(w), at, R, scatter=o, out=np.zeros((R, N)), **kw))
    g = whole((R, N), "f16", 4)
    same(mhr.matmul_experts_grad(x, g, offsets, gather=order, top=top, out_dtype=torch.float32),
         ref.weight_grad(f64(x), f64(g), at, gather=o, top=top))
    same(mhr.matmul_experts_grad(x, g, offsets, gather=order, scatter=order, top=top,
                                 out_dtype=torch.float32),
         ref.weight_grad(f64(x), f64(g), at, gather=o, scatter=o, top=top))
    # the gradient of the tokens: the transposed product back in (token, slot) order, summed
    dx = mhr.matmul_experts(g, w, offsets, gather=order, scatter=order, transposed=not transposed,
                            out_dtype=torch.float32).reshape(T, top, K).sum(1)
    wt = f64(w) if transposed else f64(w).transpose(0, 2, 1)
    assert np.array_equal(f64(dx), (f64(g)[:, None] @ wt[e]).reshape(T, top, K).sum(1))
    assert mhr.gemm_check(None) == mhr.MHR_OK


@pytest.mark.parametrize("kind", ["product", "transposed", "grad"])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_real_values(mhr, kind, dtype):
    """Normal inputs. Products are exact in fp32; a sum of n of them, however ordered, even with
    truncation, is off by at most n 2^-23 of the sum of magnitudes; then one rounding."""
    import torch

    at, offsets = offsets_of([150, 0, 90])
    gen = torch.Generator().manual_seed(5)
    x = torch.randn(240, 520, generator=gen).to(types()[dtype]).cuda()
    for out_dtype in (dtype, "f32"):
        if kind == "grad":
            g = torch.randn(240, 304, generator=gen).to(types()[dtype]).cuda()
            got = mhr.matmul_experts_grad(x, g, offsets, out_dtype=types()[out_dtype])
            want, S = (ref.weight_grad(a, b, at) for a, b in
                       ((f64(x), f64(g)), (np.abs(f64(x)), np.abs(f64(g)))))
            n = 150
        else:
            t = kind == "transposed"
            w = torch.randn((3, 304, 520) if t else (3, 520, 304), generator=gen)
            w = w.to(types()[dtype]).cuda()
            got = mhr.matmul_experts(x, w, offsets, transposed=t, out_dtype=types()[out_dtype])
            want, S = (ref.product(a, b, at, 240, transposed=t, out=np.zeros((240, 304)))
                       for a, b in ((f64(x), f64(w)), (np.abs(f64(x)), np.abs(f64(w)))))
            n = 520
        err = np.abs(f64(got) - want)
        assert np.all(err <= n * 2.0 ** -23 * S + HALF_STEP[out_dtype] * np.abs(want))


@pytest.mark.parametrize("K,N", [(1, 1), (7, 9), (65, 129), (130, 257), (1, 300), (333, 2)])
@pytest.mark.parametrize("kind", ["product", "transposed", "grad"])
def test_odd_sizes(mhr, K, N, kind):
    """Rows that TMA cannot read are copied to scratch; odd outputs are stored one by one."""
    import torch

    at, offsets = offsets_of([3, 0, 40, 1])
    x = whole((44, K), "bf16", K)
    for out_dtype in (torch.bfloat16, torch.float32):
        if kind == "grad":
            g = whole((44, N), "bf16", N)
            same(mhr.matmul_experts_grad(x, g, offsets, out_dtype=out_dtype),
                 ref.weight_grad(f64(x), f64(g), at))
        else:
            t = kind == "transposed"
            w = whole((4, N, K) if t else (4, K, N), "bf16", 3)
            same(mhr.matmul_experts(x, w, offsets, transposed=t, out_dtype=out_dtype),
                 ref.product(f64(x), f64(w), at, 44, transposed=t, out=np.zeros((44, N))))


def test_strides_and_padding_stay(mhr):
    import torch

    at, offsets = offsets_of([20, 13])
    K, N = 80, 96
    bx = whole((33, K + 24), "bf16", 1)
    bw = whole((2, K + 3, N + 8), "bf16", 2)
    for x in (bx[:, 8:K + 8], bx[:, 3:K + 3]):            # on and off 16 bytes
        for w in (bw[:, 1:K + 1, :N], bw[:, 2:K + 2, 5:N + 5]):
            buf = torch.full((33, N + 9), 7.0, device="cuda")
            mhr.matmul_experts(x, w, offsets, out=buf[:, 4:N + 4])
            same(buf[:, 4:N + 4], ref.product(f64(x), f64(w), at, 33, out=np.zeros((33, N))))
            assert bool((buf[:, :4] == 7).all()) and bool((buf[:, N + 4:] == 7).all())
    g = whole((33, N + 24), "bf16", 4)[:, 16:N + 16]
    buf = torch.full((2, K + 2, N + 6), 7.0, dtype=torch.bfloat16, device="cuda")
    mhr.matmul_experts_grad(bx[:, 8:K + 8], g, offsets, out=buf[:, 1:K + 1, 3:N + 3])
    same(buf[:, 1:K + 1, 3:N + 3], ref.weight_grad(f64(bx[:, 8:K + 8]), f64(g), at))
    buf[:, 1:K + 1, 3:N + 3] = 7
    assert bool((buf == 7).all())


def test_rows_without_an_expert_stay(mhr):
    import torch

    at, offsets = offsets_of([4, 0, 9])
    x, w = whole((40, 64), "bf16", 1), whole((3, 64, 72), "bf16", 2)
    out = torch.full((40, 72), 7.0, device="cuda")
    mhr.matmul_experts(x, w, offsets, out=out)
    want = ref.product(f64(x), f64(w), at, 40, out=np.full((40, 72), 7.0))
    same(out, want)
    assert float(out[13:].min()) == 7
    # a gradient takes the experts' rows alone
    g = whole((40, 72), "bf16", 3)
    g[13:] = float("nan")
    same(mhr.matmul_experts_grad(x, g, offsets, out_dtype=torch.float32),
         ref.weight_grad(f64(x), f64(g), at))


def test_indices_outside(mhr):
    """They cause no access: rows of zeros, rows that are not written."""
    import torch

    at, offsets = offsets_of([10, 6])
    x, w = whole((5, 64), "bf16", 1), whole((2, 64, 64), "bf16", 2)
    gather = index([0, 9, -1, 4, 10, 11, 2 ** 31 - 1, -2 ** 31, 3, 3, 8, 2, 1, 0, 5, 7])
    scatter = index([0, 3, 2, -1, 16, 5, 6, 7, -2 ** 31, 9, 10, 2 ** 31 - 1, 12, 13, 14, 15])
    gn, sn = gather.cpu().numpy(), scatter.cpu().numpy()
    out = torch.full((16, 64), 7.0, device="cuda")
    mhr.matmul_experts(x, w, offsets, gather=gather, scatter=scatter, top=2, out=out)
    same(out, ref.product(f64(x), f64(w), at, 16, gather=gn, scatter=sn, top=2,
                          out=np.full((16, 64), 7.0)))
    g = whole((16, 72), "bf16", 3)
    same(mhr.matmul_experts_grad(x, g, offsets, gather=gather, scatter=scatter, top=2,
                                 out_dtype=torch.float32),
         ref.weight_grad(f64(x), f64(g), at, gather=gn, scatter=sn, top=2))
    # offsets that fall, or lie past the rows
    bad = index([3, 1, 99])
    out = torch.full((16, 64), 7.0, device="cuda")
    xs = whole((16, 64), "bf16", 5)
    mhr.matmul_experts(xs, w, bad, out=out)
    same(out, ref.product(f64(xs), f64(w), [1, 1, 16], 16, out=np.full((16, 64), 7.0)))
    assert mhr.gemm_check(None) == mhr.MHR_OK


def test_infinities_stay_with_their_experts(mhr):
    """Rows of another expert, and those past the last, share tiles and boxes with an expert's."""
    import torch

    at, offsets = offsets_of([5, 4])
    x, w = whole((12, 72), "bf16", 1), whole((2, 72, 72), "bf16", 2)
    x[5:] = float("inf")
    w[1] = float("nan")
    got = mhr.matmul_experts(x, w, offsets, out=torch.zeros(12, 72, device="cuda"))
    same(got[:5], ref.product(f64(x)[:5], f64(w)[:1], [0, 5], 5, out=np.zeros((5, 72))))
    assert bool(got[5:9].isnan().all()) and float(got[9:].abs().max()) == 0
    g = whole((12, 72), "bf16", 3)
    g[5:] = float("nan")
    d = mhr.matmul_experts_grad(x, g, offsets, out_dtype=torch.float32)
    same(d[:1], ref.weight_grad(f64(x)[:5], f64(g)[:5], [0, 5]))


def test_empty(mhr):
    import torch

    _, offsets = offsets_of([0, 0])
    e = dict(dtype=torch.bfloat16, device="cuda")
    assert mhr.matmul_experts(torch.zeros(0, 64, **e), torch.zeros(2, 64, 8, **e), offsets).shape == (0, 8)
    g = mhr.matmul_experts_grad(torch.zeros(0, 64, **e), torch.zeros(0, 8, **e), offsets)
    assert g.shape == (2, 64, 8) and float(g.abs().max()) == 0
    _, offsets = offsets_of([2, 1])
    out = mhr.matmul_experts(torch.zeros(3, 0, **e), torch.zeros(2, 0, 8, **e), offsets)
    assert out.shape == (3, 8) and float(out.abs().max()) == 0
    assert mhr.matmul_experts(torch.zeros(3, 8, **e), torch.zeros(2, 8, 0, **e), offsets).shape == (3, 0)
    assert mhr.matmul_experts_grad(torch.zeros(3, 0, **e), torch.zeros(3, 8, **e), offsets).shape == (2, 0, 8)
    out = mhr.matmul_experts(torch.zeros(0, 8, **e), torch.ones(2, 8, 8, **e), offsets,
                             gather=index([0, 1, 2]))
    assert float(out.abs().max()) == 0


def test_many_experts_and_far_offsets(mhr):
    import torch

    E = 1024
    counts = np.random.default_rng(1).integers(0, 3, E)
    at, offsets = offsets_of(counts)
    rows = int(at[-1])
    x, w = whole((rows, 64), "bf16", 1), whole((E, 64, 64), "bf16", 2)
    same(mhr.matmul_experts(x, w, offsets),
         ref.product(f64(x), f64(w), at, rows, out=np.zeros((rows, 64))))
    g = whole((rows, 64), "bf16", 3)
    same(mhr.matmul_experts_grad(x, g, offsets), ref.weight_grad(f64(x), f64(g), at))
    # experts, rows and outputs more than 2^32 bytes apart
    pitch = (1 << 31) + 64
    big = torch.zeros(pitch + 64 * 64, dtype=torch.bfloat16, device="cuda")
    w = torch.as_strided(big, (2, 64, 64), (pitch, 64, 1))
    w.copy_(whole((2, 64, 64), "bf16", 4))
    at, offsets = offsets_of([3, 5])
    x = whole((8, 64), "bf16", 5)
    want = ref.product(f64(x), f64(w), at, 8, out=np.zeros((8, 64)))
    same(mhr.matmul_experts(x, w, offsets), want)
    flat = torch.zeros((1 << 31) // 7 * 7 + 64, dtype=torch.bfloat16, device="cuda")
    out = torch.as_strided(flat, (8, 64), ((1 << 31) // 7, 1))
    mhr.matmul_experts(x, w, offsets, out=out)
    same(out, want)
    d = torch.as_strided(big, (2, 64, 64), (pitch, 64, 1))
    g = whole((8, 64), "bf16", 6)
    mhr.matmul_experts_grad(x, g, offsets, out=d)
    same(d, ref.weight_grad(f64(x), f64(g), at))


def test_on_another_stream_and_captured(mhr):
    import torch

    at, offsets = offsets_of([40, 0, 77])
    x, w = whole((117, 71), "bf16", 1), whole((3, 71, 65), "bf16", 2)  # (copied to scratch)
    want = ref.product(f64(x), f64(w), at, 117, out=np.zeros((117, 65)))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out = torch.empty(117, 65, device="cuda")
    mhr.matmul_experts(x, w, offsets, out=out, stream=s.cuda_stream)
    junk = [torch.full((200_000,), 7, dtype=torch.uint8, device="cuda") for _ in range(8)]
    s.synchronize()
    same(out, want)
    del junk
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = mhr.matmul_experts(x, w, offsets)
        d = mhr.matmul_experts_grad(x, out, offsets, out_dtype=torch.float32)
    x.copy_(whole((117, 71), "bf16", 9))
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    same(out, ref.product(f64(x), f64(w), at, 117, out=np.zeros((117, 65))))
    assert torch.equal(d, mhr.matmul_experts_grad(x, out, offsets, out_dtype=torch.float32))


def test_a_stalled_stage_is_a_timeout(mhr):
    """The bounded waits: both CTAs of a pair unwind, the next call is right."""
    import torch

    at, offsets = offsets_of([40, 77])
    x, w = whole((117, 520), "bf16", 1), whole((2, 520, 256), "bf16", 2)
    old = mhr.gemm_testing_set_wait_limit_ns(20_000_000)
    mhr.gemm_testing_set_inject_stall(1)
    try:
        mhr.matmul_experts(x, w, offsets)
        assert mhr.gemm_check(None) == mhr.MHR_ERR_TIMEOUT
        mhr.matmul_experts_grad(x, x, offsets)
        assert mhr.gemm_check(None) == mhr.MHR_ERR_TIMEOUT
        order = torch.arange(116, -1, -1, dtype=torch.int32, device="cuda")
        mhr.matmul_experts(x, w, offsets, gather=order)
        assert mhr.gemm_check(None) == mhr.MHR_ERR_TIMEOUT
    finally:
        mhr.gemm_testing_set_inject_stall(0)
        mhr.gemm_testing_set_wait_limit_ns(old)
    same(mhr.matmul_experts(x, w, offsets),
         ref.product(f64(x), f64(w), at, 117, out=np.zeros((117, 256))))
    assert mhr.gemm_check(None) == mhr.MHR_OK


def test_scratch_is_of_the_calls_own_stream(mhr):
    """What the current stream gave back may still be written by its work: a call on another
    stream takes its scratch from that stream's memory."""
    import torch

    n = 20_000
    at, offsets = offsets_of([9_000, 11_000])
    x, w = whole((n, 71), "bf16", 1), whole((2, 71, 65), "bf16", 2)
    out = torch.zeros((n, 65), dtype=torch.bfloat16, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())

    def held():
        return sum(g["total_size"] for g in torch.cuda.memory_snapshot()
                   if g["stream"] == s.cuda_stream)

    torch.cuda.empty_cache()
    before = held()
    mhr.matmul_experts(x, w, offsets, out=out, stream=s.cuda_stream)
    s.synchronize()
    assert held() > before
    same(out, ref.product(f64(x), f64(w), at, n, out=np.zeros((n, 65))))


def test_two_streams_at_once(mhr):
    """Calls that share the GPU, their scratch apart: all as if alone."""
    import torch

    at, offsets = offsets_of([300, 0, 500, 224])
    order = torch.arange(1023, -1, -1, dtype=torch.int32, device="cuda")
    x, w = whole((1024, 200), "bf16", 1), whole((4, 200, 328), "bf16", 2)
    x2 = whole((1024, 200), "bf16", 3)
    calls = [lambda a, **k: mhr.matmul_experts(a, w, offsets, order, **k),
             lambda a, **k: mhr.matmul_experts_grad(a, a, offsets, order, order, **k)]
    for call in calls:
        want = [call(a) for a in (x, x2)]
        streams = [torch.cuda.Stream() for _ in range(2)]
        outs = [[torch.empty_like(want[0]) for _ in range(8)] for _ in range(2)]
        for s in streams:
            s.wait_stream(torch.cuda.current_stream())
        for i in range(8):
            for j, a in enumerate((x, x2)):
                call(a, out=outs[j][i], stream=streams[j].cuda_stream)
        torch.cuda.synchronize()
        for j in range(2):
            assert all(torch.equal(o, want[j]) for o in outs[j])


@pytest.mark.parametrize("out_dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("K,N,left,pad", [(300, 200, 8, 16), (300, 199, 3, 8), (33, 330, 0, 2),
                                          (513, 97, 1, 0), (256, 257, 2, 3)])
def test_gradient_into_a_larger_matrix(mhr, out_dtype, K, N, left, pad):
    """Rows that TMA can write and rows that start anywhere, ends inside every tile."""
    import torch

    at, offsets = offsets_of([140, 0, 300])
    dtype = "f16" if out_dtype == "f16" else "bf16"
    x, g = whole((440, K), dtype, 1), whole((440, N), dtype, 2)
    buf = torch.full((3, K + 2, left + N + pad), 7.0, dtype=types()[out_dtype], device="cuda")
    out = buf[:, 1:K + 1, left:left + N]
    mhr.matmul_experts_grad(x, g, offsets, out=out)
    same(out, ref.weight_grad(f64(x), f64(g), at))
    out.fill_(7)
    assert bool((buf == 7).all())
