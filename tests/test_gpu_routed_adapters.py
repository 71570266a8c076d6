"""Low-rank adapters on the GPU, against 64-bit numpy.

Whole numbers keep every sum exact (see test_gpu_routed_product.py), so most results are equal to
the one rounding of the output type.
"""
import numpy as np
import pytest

import routed_ref as ref

pytestmark = pytest.mark.gpu

HALF_STEP = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}


def types():
    import torch

    return {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def whole(shape, dtype, seed, most=3):
    import torch

    x = np.random.default_rng(seed).integers(-most, most + 1, shape)
    return torch.from_numpy(x).to(types()[dtype]).cuda()


def f64(t):
    return t.double().cpu().numpy()


def same(got, want):
    import torch

    want = torch.from_numpy(want).to(got.dtype)
    assert torch.equal(got.cpu(), want), float((got.cpu().double() - want.double()).abs().max())


def which_of(T, L, run, seed):
    """Requests of `run` rows, some without an adapter, by entries below 0 and past the last."""
    import torch

    a = np.random.default_rng(seed).integers(-1, L + 1, -(-T // run)).repeat(run)[:T]
    a[0] = 0
    return torch.from_numpy(a.astype(np.int32)).cuda()


def case(T, K, N, L, rank, dtype, seed=0):
    return (whole((T, K), dtype, seed + 1), whole((L, rank, K), dtype, seed + 2, 1),
            whole((L, rank, N), dtype, seed + 3, 1))


@pytest.mark.parametrize("T,run", [(1, 1), (3, 1), (7, 2), (63, 1), (64, 64), (65, 1), (256, 5), (257, 5), (512, 5), (513, 5), (200, 33),
                                   (130, 1), (1000, 700), (2100, 150)])
@pytest.mark.parametrize("K,N,L,rank", [(64, 64, 3, 16), (200, 136, 5, 4), (72, 264, 1, 64),
                                        (136, 392, 9, 11), (128, 1032, 2, 100), (64, 72, 40, 128)])
def test_adapters(mhr, T, run, K, N, L, rank):
    import torch

    for dtype, out in (("bf16", "bf16"), ("f16", "f32"), ("bf16", "f32"), ("f16", "f16")):
        x, down, up = case(T, K, N, L, rank, dtype)
        y = whole((T, N), out, 4, 50)
        which = which_of(T, L, run, T)
        scales = torch.from_numpy(2.0 ** np.arange(-1, L - 1).clip(-1, 2)).float().cuda()
        got = mhr.add_adapters(y, x, down, up, which, scales)
        assert mhr.gemm_check(None) == mhr.MHR_OK
        assert got.dtype == y.dtype
        want = ref.adapters(f64(y), f64(x), f64(down), f64(up), which.cpu().numpy(), f64(scales))
        same(got, want)
        # in place, and without scales
        z = y.clone()
        assert mhr.add_adapters(z, x, down, up, which, out=z) is not None
        same(z, ref.adapters(f64(y), f64(x), f64(down), f64(up), which.cpu().numpy()))


@pytest.mark.parametrize("T", [2, 150, 270])
@pytest.mark.parametrize("K,N,rank", [(1, 1, 1), (7, 9, 3), (65, 129, 8), (131, 2, 16), (9, 300, 33)])
def test_odd_sizes(mhr, T, K, N, rank):
    for out in ("bf16", "f32"):
        x, down, up = case(T, K, N, 3, rank, "bf16")
        y, which = whole((T, N), out, 4, 50), which_of(T, 3, 1, 1)
        same(mhr.add_adapters(y, x, down, up, which),
             ref.adapters(f64(y), f64(x), f64(down), f64(up), which.cpu().numpy()))


@pytest.mark.parametrize("T", [4, 300])
@pytest.mark.parametrize("dtype,out", [("bf16", "bf16"), ("bf16", "f32"), ("f16", "f16"),
                                       ("f16", "f32")])
@pytest.mark.parametrize("size", [1.0, 2.0 ** -7])
def test_real_values(mhr, T, dtype, out, size):
    """Products are exact in fp32; sums of n of them, however ordered, are off by at most n 2^-23
    of the sum of magnitudes. Between the sums v is held to 2^-16 for 16-bit results (two terms of
    8 bits each, less a bit for the second's sign and rounding) or 2^-20 for fp32 ones (three, or
    two of 11 bits on the row's own power of two), of the row's largest."""
    import torch

    gen = torch.Generator().manual_seed(T)
    K, N, L, rank = 1000, 264, 4, 24

    def normal(*shape):
        return torch.randn(*shape, generator=gen)

    x = (normal(T, K) * size).to(types()[dtype]).cuda()
    down = (normal(L, rank, K) * K ** -0.5).to(types()[dtype]).cuda()
    up, y = normal(L, rank, N).to(types()[dtype]).cuda(), normal(T, N).to(types()[out]).cuda()
    which, scales = which_of(T, L, 3, 1), (0.5 + torch.rand(L, generator=gen)).cuda()
    got = f64(mhr.add_adapters(y, x, down, up, which, scales))
    w = which.cpu().numpy()
    want = ref.adapters(f64(y), f64(x), f64(down), f64(up), w, f64(scales))
    held = 2.0 ** -20 if out == "f32" else 2.0 ** -16
    bound = HALF_STEP[out] * np.abs(want)
    for t, a in enumerate(w):
        if 0 <= a < L:
            s, d, u = float(scales[a]), f64(down[a]), f64(up[a])
            v = d @ f64(x[t])
            off = K * 2.0 ** -23 * (np.abs(d) @ np.abs(f64(x[t]))) + held * np.abs(v).max()
            bound[t] += s * (off @ np.abs(u) + (rank + 4) * 2.0 ** -23 * (np.abs(v) @ np.abs(u)))
            bound[t] += 2.0 ** -23 * np.abs(f64(y[t]))
    assert np.all(np.abs(got - want) <= bound), float((np.abs(got - want) / bound).max())


@pytest.mark.parametrize("T", [3, 140, 270])
def test_strides_and_padding_stay(mhr, T):
    import torch

    K, N, L, rank = 80, 96, 3, 12
    bx, bd = whole((T, K + 24), "bf16", 1), whole((L, rank + 3, K + 8), "bf16", 2, 1)
    bu, by = whole((L, rank + 1, N + 16), "bf16", 3, 1), whole((T, N + 8), "f32", 4, 50)
    which = which_of(T, L, 2, 1)
    for o in (0, 8, 3):
        x, down = bx[:, o:K + o], bd[:, 1:rank + 1, :K]
        up, y = bu[:, :rank, o:N + o], by[:, o // 2:N + o // 2]
        buf = torch.full((T, N + 9), 7.0, device="cuda")
        mhr.add_adapters(y, x, down, up, which, out=buf[:, 4:N + 4])
        same(buf[:, 4:N + 4], ref.adapters(f64(y), f64(x), f64(down), f64(up), which.cpu().numpy()))
        assert bool((buf[:, :4] == 7).all()) and bool((buf[:, N + 4:] == 7).all())


@pytest.mark.parametrize("T", [5, 200, 520])
def test_none_and_empty(mhr, T):
    import torch

    x, down, up = case(T, 64, 72, 3, 8, "bf16")
    y = whole((T, 72), "bf16", 4, 50)
    none = torch.full((T,), -1, dtype=torch.int32, device="cuda")
    assert torch.equal(mhr.add_adapters(y, x, down, up, none), y)
    z = y.clone()
    mhr.add_adapters(z, x, down, up, none + 4, out=z)
    assert torch.equal(z, y)
    which = which_of(T, 3, 1, 1)
    same(mhr.add_adapters(y, x[:, :0], down[:, :, :0], up, which), f64(y))
    assert mhr.add_adapters(y[:, :0], x, down, up[:, :, :0], which).shape == (T, 0)
    assert mhr.add_adapters(y[:0], x[:0], down, up, which[:0]).shape == (0, 72)


@pytest.mark.parametrize("T", [6, 200, 520])
def test_infinities_stay_in_their_rows(mhr, T):
    import torch

    x, down, up = case(T, 64, 72, 2, 8, "bf16")
    y, which = whole((T, 72), "f32", 4, 50), which_of(T, 2, 1, 1)
    clean = mhr.add_adapters(y, x, down, up, which)
    x[1], which[1] = float("nan"), 1
    x[2], which[2] = float("inf"), 0
    x[3], which[3] = float("nan"), -1
    got = mhr.add_adapters(y, x, down, up, which)
    assert bool(got[1].isnan().all()) and not bool(got[2].isfinite().any())
    assert torch.equal(got[3], y[3])
    assert torch.equal(got[4:], clean[4:]) and torch.equal(got[0], clean[0])


def test_far_offsets(mhr):
    """Adapters, rows and results more than 2^32 bytes apart."""
    import torch

    pitch = (1 << 31) + 64
    big = torch.zeros(pitch + 16 * 64, dtype=torch.bfloat16, device="cuda")
    for T in (2, 130, 530):
        x, down, up = case(T, 64, 64, 2, 16, "bf16")
        d = torch.as_strided(big, (2, 16, 64), (pitch, 64, 1))
        y, which = whole((T, 64), "bf16", 4, 50), which_of(T, 2, 1, 1)
        want = mhr.add_adapters(y, x, down, up, which)
        d.copy_(down)
        assert torch.equal(mhr.add_adapters(y, x, d, up, which), want)
        d.copy_(up)
        assert torch.equal(mhr.add_adapters(y, x, down, d, which), want)
        out = torch.as_strided(big, (T, 64), ((1 << 31) // T // 8 * 8 + 8, 1))
        mhr.add_adapters(y, x, down, up, which, out=out)
        assert torch.equal(out, want)


@pytest.mark.parametrize("T", [6, 300])
def test_on_another_stream_and_captured(mhr, T):
    import torch

    x, down, up = case(T, 71, 65, 3, 8, "bf16")
    y, which = whole((T, 65), "f32", 4, 50), which_of(T, 3, 2, 1)
    want = ref.adapters(f64(y), f64(x), f64(down), f64(up), which.cpu().numpy())
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out = torch.empty_like(y)
    mhr.add_adapters(y, x, down, up, which, out=out, stream=s.cuda_stream)
    junk = [torch.full((200_000,), 7, dtype=torch.uint8, device="cuda") for _ in range(8)]
    s.synchronize()
    same(out, want)
    del junk
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = mhr.add_adapters(y, x, down, up, which)
    which.copy_(which_of(T, 3, 1, 9))
    graph.replay()
    graph.replay()
    same(out, ref.adapters(f64(y), f64(x), f64(down), f64(up), which.cpu().numpy()))


@pytest.mark.parametrize("run", [1, 600])
def test_a_stalled_stage_is_a_timeout(mhr, run):
    """The bounded waits: the whole cluster unwinds, the next call is right."""
    x, down, up = case(600, 1024, 1024, 2, 16, "bf16")
    y, which = whole((600, 1024), "bf16", 4, 50), which_of(600, 2, run, 1).clamp(min=0)
    want = mhr.add_adapters(y, x, down, up, which)
    old = mhr.gemm_testing_set_wait_limit_ns(20_000_000)
    mhr.gemm_testing_set_inject_stall(1)
    try:
        mhr.add_adapters(y, x, down, up, which)
        assert mhr.gemm_check(None) == mhr.MHR_ERR_TIMEOUT
    finally:
        mhr.gemm_testing_set_inject_stall(0)
        mhr.gemm_testing_set_wait_limit_ns(old)
    assert mhr.add_adapters(y, x, down, up, which).equal(want)
    assert mhr.gemm_check(None) == mhr.MHR_OK
