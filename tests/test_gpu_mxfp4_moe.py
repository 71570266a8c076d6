"""The mixture-of-experts layer on the GPU against 64-bit numpy."""
import numpy as np
import pytest

import mxfp4_ref as ref

pytestmark = pytest.mark.gpu


def layer(T, E, top, H, I, seed, favoured=0):
    """x and router as float64 bf16 values whose chosen experts are clear of ties by 1e-4 (fp32
    sums of H products of order 1 / sqrt(H) stay within H 2^-24 of that order), packed experts."""
    import torch

    for attempt in range(50):
        rng = np.random.default_rng(seed + 1000 * attempt)
        bf = lambda a: torch.from_numpy(a).bfloat16().double().numpy()  # noqa: E731
        x = bf(rng.standard_normal((T, H)))
        router = bf(rng.standard_normal((E, H)) * H ** -0.5)
        if favoured:  # experts that every token chooses: logits from 4 on
            x[:, 0] = 2
            first = E // 3
            router[first:first + favoured] = 0
            router[first:first + favoured, 0] = bf(2 + np.arange(favoured) / 16)
        order = np.sort(x @ router.T, 1)[:, ::-1]
        if E == 1 or np.min(order[:, :top + 1][:, :-1] - order[:, :top + 1][:, 1:]) > 1e-4:
            break
    else:
        raise AssertionError("no clear routing found")
    up, ups, upv = ref.random_packed(2 * E * I, H, seed + 1, 122 - int(np.log2(H) / 2), 126 - int(np.log2(H) / 2))
    down, downs, downv = ref.random_packed(E * H, I, seed + 2, 122 - int(np.log2(I) / 2), 126 - int(np.log2(I) / 2))
    return x, router, (up, ups, upv), (down, downs, downv)


def expected(x, router, upv, downv, top, E, H, I):
    """y, its error bound, experts and weights, from the definition in 64 bits.

    The bound: gate and up are fp32 sums over H (at most H / 16 + 64 roundings of 2^-22 of the sum
    of magnitudes); |silu'| <= 1.1 and silu is off by a few units (2^-20); h is rounded to no
    less than 11 bits (2^-11); the down sums likewise over I and top; weights carry 2^-18; y is rounded to bf16."""
    T = x.shape[0]
    logits = x @ router.T
    experts = np.argsort(-logits, axis=1, kind="stable")[:, :top]
    chosen = np.take_along_axis(logits, experts, 1)
    w = np.exp(chosen - chosen[:, :1])
    w /= w.sum(1, keepdims=True)
    y, bound = np.zeros((T, H)), np.zeros((T, H))
    for t in range(T):
        for k in range(top):
            e = experts[t, k]
            G, U = upv[2 * e * I:(2 * e + 1) * I], upv[(2 * e + 1) * I:(2 * e + 2) * I]
            D = downv[e * H:(e + 1) * H]
            g, u = G @ x[t], U @ x[t]
            eg = (H / 16 + 64) * 2.0 ** -22 * (np.abs(G) @ np.abs(x[t]))
            eu = (H / 16 + 64) * 2.0 ** -22 * (np.abs(U) @ np.abs(x[t]))
            s = g / (1 + np.exp(-g))
            h = s * u
            eh = 1.1 * eg * (np.abs(u) + eu) + np.abs(s) * eu + (2.0 ** -11 + 2.0 ** -20) * np.abs(h)
            y[t] += w[t, k] * (D @ h)
            mag = np.abs(D) @ np.abs(h)
            bound[t] += w[t, k] * (np.abs(D) @ eh + ((I / 16 + 64) * 2.0 ** -22 + 2.0 ** -18) * mag)
    bound += 2.0 ** -8 * (np.abs(y) + bound) + 1e-30
    return y, bound, experts, w


def run_case(mhr, T, E, top, H, I, seed=0, shift=0, favoured=0):
    import torch

    x, router, (up, ups, upv), (down, downs, downv) = layer(T, E, top, H, I, seed, favoured)
    dev = lambda a: torch.from_numpy(a).cuda()  # noqa: E731

    def strided(a):  # a bf16 matrix in a wider buffer, `shift` elements in
        buf = torch.full((a.shape[0], a.shape[1] + 2 * shift), 9.0, dtype=torch.bfloat16, device="cuda")
        v = buf[:, shift:shift + a.shape[1]]
        v.copy_(dev(a))
        return v

    out = strided(np.zeros((T, H)))
    y, experts, weights = mhr.moe_mxfp4(strided(x), strided(router),
                                        mhr.MxFp4Matrix(dev(up), dev(ups), 2 * E * I, H),
                                        mhr.MxFp4Matrix(dev(down), dev(downs), E * H, I), top, out=out)
    assert mhr.gemm_check(None) == mhr.MHR_OK
    want, bound, want_e, want_w = expected(x, router, upv, downv, top, E, H, I)
    assert np.array_equal(experts.cpu().numpy(), want_e)
    assert np.allclose(weights.cpu().numpy(), want_w, rtol=2e-5, atol=0)  # exp of logits off by ~1e-6
    err = np.abs(y.double().cpu().numpy() - want)
    assert np.all(err <= bound), float((err / bound).max())
    if shift:
        base = out._base if out._base is not None else out
        assert bool((base[:, :shift] == 9).all()) and bool((base[:, -shift:] == 9).all())
    return y, experts, weights


CASES = [(1, 1, 1, 32, 32), (1, 4, 2, 64, 32), (1, 32, 4, 1024, 512), (2, 8, 8, 96, 200), (3, 5, 3, 257, 33),
         (5, 16, 4, 520, 129), (8, 60, 6, 1000, 300), (9, 12, 2, 384, 640), (16, 128, 8, 256, 128),
         (17, 3, 2, 320, 96), (33, 64, 4, 264, 72), (64, 4, 4, 192, 160), (64, 128, 8, 512, 256),
         (64, 500, 1, 64, 40), (64, 2, 1, 2048, 100), (7, 20, 16, 130, 1000)]


@pytest.mark.parametrize("T,E,top,H,I", CASES)
def test_layer(mhr, T, E, top, H, I):
    run_case(mhr, T, E, top, H, I, seed=T + E + H)


@pytest.mark.parametrize("shift", [1, 8])
def test_layer_strides(mhr, shift):
    run_case(mhr, 6, 10, 3, 200, 96, shift=shift)
    run_case(mhr, 20, 10, 3, 256, 96, shift=shift)


@pytest.mark.parametrize("T,E,top,H,I,shift", [
    (50, 61, 3, 203, 40, 0), (50, 61, 3, 203, 40, 1), (64, 45, 2, 2104, 33, 8),
    (41, 120, 4, 4100, 16, 0), (17, 511, 1, 31, 8, 0)])
def test_more_logits_than_warps(mhr, T, E, top, H, I, shift):
    """Ragged sets of tokens and experts, rows that take no 16-byte loads, several rounds of K."""
    run_case(mhr, T, E, top, H, I, seed=H, shift=shift)


def test_more_columns_than_are_staged_at_once(mhr):
    """Every token on the same experts and wide rows: several passes over an expert's pairs."""
    run_case(mhr, 64, 2, 2, 8192, 96, seed=5)
    run_case(mhr, 40, 1, 1, 128, 9000, seed=6)


@pytest.mark.parametrize("T,E,top,H,I,favoured", [
    (64, 340, 16, 13000, 2, 8),   # columns too long for shared memory in one part of K, and more
                                  # passes over experts than any other shape has
    (64, 20, 16, 16384, 8, 0),
    (64, 20, 8, 8, 16384, 4),     # the same of the down product
    (64, 24, 16, 40, 13000, 8),
    (1, 16, 16, 16384, 16, 0)])
def test_longest_columns(mhr, T, E, top, H, I, favoured):
    run_case(mhr, T, E, top, H, I, seed=T + E, favoured=favoured)


def test_ties_go_to_the_lowest_expert(mhr):
    import torch

    T, E, H, I = 3, 40, 64, 32
    x = torch.randn(T, H, device="cuda").bfloat16()
    row = torch.randn(1, H, device="cuda").bfloat16()
    up = mhr.quantize_mxfp4(torch.randn(2 * E * I, H, device="cuda"))
    down = mhr.quantize_mxfp4(torch.randn(E * H, I, device="cuda"))
    _, experts, weights = mhr.moe_mxfp4(x, row.expand(E, H).contiguous(), up, down, 5)
    assert experts.tolist() == [[0, 1, 2, 3, 4]] * T
    assert bool((weights == 0.2).all())


def test_zero_token_and_zero_rows(mhr):
    """A token of zeros: equal logits, a zero output; weights of zero codes give zero."""
    import torch

    E, H, I = 6, 96, 64
    x = torch.randn(4, H, device="cuda").bfloat16()
    x[2] = 0
    up = mhr.quantize_mxfp4(torch.randn(2 * E * I, H, device="cuda"))
    down = mhr.quantize_mxfp4(torch.randn(E * H, I, device="cuda"))
    router = torch.randn(E, H, device="cuda").bfloat16()
    y, experts, _ = mhr.moe_mxfp4(x, router, up, down, 2)
    assert experts[2].tolist() == [0, 1] and bool((y[2] == 0).all()) and bool((y[0] != 0).any())
    zero = mhr.quantize_mxfp4(torch.zeros(2 * E * I, H, device="cuda"))
    assert bool((mhr.moe_mxfp4(x, router, zero, down, 2)[0] == 0).all())
    assert mhr.moe_mxfp4(x[:0], router, up, down, 2)[0].shape == (0, H)


def test_nan_token_stays_in_its_row(mhr):
    import torch

    E, H, I = 6, 96, 64
    x = torch.randn(5, H, device="cuda").bfloat16()
    up = mhr.quantize_mxfp4(torch.randn(2 * E * I, H, device="cuda"))
    down = mhr.quantize_mxfp4(torch.randn(E * H, I, device="cuda"))
    router = torch.randn(E, H, device="cuda").bfloat16()
    want = mhr.moe_mxfp4(x, router, up, down, 2)[0]
    bad = x.clone()
    bad[3, 10] = float("nan")
    got = mhr.moe_mxfp4(bad, router, up, down, 2)[0]
    keep = [0, 1, 2, 4]
    assert torch.equal(got[keep], want[keep]) and bool(torch.isnan(got[3]).all())


@pytest.mark.parametrize("size", [2.0 ** -60, 2.0 ** 40])
def test_magnitudes_far_from_one(mhr, size):
    """Tokens and weights whose products leave f16's range: the powers of two take them back.
    (Gates far from zero: silu is the gate itself, or next to nothing.)"""
    import torch

    E, H, I = 4, 128, 64
    x = torch.randn(3, H, device="cuda").bfloat16()
    router = torch.randn(E, H, device="cuda").bfloat16()
    up = mhr.quantize_mxfp4(torch.randn(2 * E * I, H, device="cuda"))
    down = mhr.quantize_mxfp4(torch.randn(E * H, I, device="cuda"))
    big = (x.float() * size).bfloat16()
    y, experts, weights = mhr.moe_mxfp4(big, router, up, down, 1)
    upv = ref.values(*ref.unpack(up.data.cpu().numpy(), up.scales.cpu().numpy(), H), H)
    downv = ref.values(*ref.unpack(down.data.cpu().numpy(), down.scales.cpu().numpy(), I), I)
    bx = big.double().cpu().numpy()
    for t in range(3):
        e = int(experts[t, 0])
        g, u = (upv[(2 * e + i) * I:(2 * e + 1 + i) * I] @ bx[t] for i in (0, 1))
        h = g * np.where(g > 0, 1.0, 0.0) * u if size > 1 else g * 0.5 * u
        want = downv[e * H:(e + 1) * H] @ h
        mag = np.abs(downv[e * H:(e + 1) * H]) @ np.abs(h)
        err = np.abs(y[t].double().cpu().numpy() - want)
        # h to 11 bits, sums within (H + I) 2^-22 of magnitudes that cancel by up to 2^6, y to 8
        assert np.all(err <= 2.0 ** -8 * np.abs(want) + 2.0 ** -9 * mag)


def test_repeats_bit_for_bit_and_leaves_its_counters_clear(mhr):
    first = run_case(mhr, 12, 16, 4, 640, 384, seed=3)[0].clone()
    for _ in range(4):
        assert bool((run_case(mhr, 12, 16, 4, 640, 384, seed=3)[0] == first).all())


def test_layer_between_products_on_several_streams(mhr):
    """The layer's counters outlive other calls' use of the same workspace; streams keep theirs."""
    import torch

    E, H, I = 16, 256, 128
    up = mhr.quantize_mxfp4(torch.randn(2 * E * I, H, device="cuda"))
    down = mhr.quantize_mxfp4(torch.randn(E * H, I, device="cuda"))
    router = torch.randn(E, H, device="cuda").bfloat16()
    xs = [torch.randn(t, H, device="cuda").bfloat16() for t in (1, 9, 30)]
    want = [mhr.moe_mxfp4(x, router, up, down, 4)[0] for x in xs]
    a = torch.randn(600, 700, device="cuda")
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    for _ in range(3):
        got = []
        for x, s in zip(xs, streams):
            with torch.cuda.stream(s):
                mhr.matmul(a, a.t().contiguous(), "3xtf32")
                got.append(mhr.moe_mxfp4(x, router, up, down, 4)[0])
        torch.cuda.synchronize()
        assert all(torch.equal(g, w) for g, w in zip(got, want))


def test_timeout_is_reported_and_cleared(mhr):
    """A block that never arrives at the grid barrier (as the test hook has it): the others give
    up after the limit, the status says so, and the next call is right."""
    import torch

    E, H, I = 8, 128, 64
    x = torch.randn(2, H, device="cuda").bfloat16()
    up = mhr.quantize_mxfp4(torch.randn(2 * E * I, H, device="cuda"))
    down = mhr.quantize_mxfp4(torch.randn(E * H, I, device="cuda"))
    router = torch.randn(E, H, device="cuda").bfloat16()
    want = mhr.moe_mxfp4(x, router, up, down, 2)[0]
    old = mhr.gemm_testing_set_wait_limit_ns(20_000_000)
    mhr.gemm_testing_set_inject_stall(1)
    try:
        mhr.moe_mxfp4(x, router, up, down, 2)
        assert mhr.gemm_check(None) == mhr.MHR_ERR_TIMEOUT
    finally:
        mhr.gemm_testing_set_inject_stall(0)
        mhr.gemm_testing_set_wait_limit_ns(old)
    assert torch.equal(mhr.moe_mxfp4(x, router, up, down, 2)[0], want)
    assert mhr.gemm_check(None) == mhr.MHR_OK
