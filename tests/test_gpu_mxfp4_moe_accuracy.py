"""How many bits the mixture-of-experts layer keeps, where the rounding of y to bf16 cannot hide it.

x and the inner vector h reach the tensor cores as eight e2m1 values a block of 32: with a first
unit s, max <= 6 s < 2 max, the first leaves at most s, the second (unit s / 4) at most s / 8 and
each further one an eighth of that, so that eight leave s 2^-21 < 2^-22 max, or 2^-129 (a quarter of
the smallest unit, 2^-127) where that is more. Everything else is fp32.
"""
import numpy as np
import pytest

import mxfp4_ref as ref

pytestmark = pytest.mark.gpu

FLOOR = 2.0 ** -129


def bf16(a):
    import torch

    return torch.from_numpy(np.asarray(a, np.float64)).bfloat16().double().numpy()


def matrix(codes, scales):
    """(packed matrix on the GPU, its float64 values)."""
    import torch

    import memory_hierarchy_reuse_gb300 as m

    rows, cols = codes.shape
    data, tiled = ref.pack(codes, scales)
    return (m.MxFp4Matrix(torch.from_numpy(data).cuda(), torch.from_numpy(tiled).cuda(), rows, cols),
            ref.values(codes, scales, cols))


def sparse(rng, rows, cols, exponent, taboo=None):
    """Codes with two nonzero columns a row, none of them in `taboo`, and scales 2^exponent."""
    codes = np.zeros((rows, cols), np.uint8)
    allowed = np.array([c for c in range(cols) if taboo is None or c not in taboo])
    at = allowed[rng.integers(0, len(allowed), (rows, 2))]
    codes[np.arange(rows)[:, None], at] = rng.integers(1, 8, (rows, 2)) + 8 * rng.integers(0, 2, (rows, 2))
    return codes, np.full((rows, cols // 32), 127 + exponent, np.uint8)


def left_over(w, v, ev):
    """What the terms of a vector v (known to within ev) leave of w v, a row of w at a time."""
    largest = (np.abs(v) + ev).reshape(-1, 32).max(1)
    return np.maximum(2.0 ** -22 * largest, FLOOR).repeat(32) @ np.abs(w).T


def expected(x, G, U, D):
    """One expert's output for a token and its bound, from the definition in 64 bits. fp32 sums: at
    most (K / 16 + 64) roundings of 2^-22 of the magnitudes (64-column MMAs, K parts, terms). silu
    and its product with up: exp within 1 ulp, a sum, a quotient and a product within half, of
    which |silu| has at most 2.5 x 2^-23 in all, 2^-21 with the half ulps of gate and up."""
    H, I = len(x), len(G)
    sums = (H / 16 + 64) * 2.0 ** -22
    g, u = G @ x, U @ x
    eg = left_over(G, x, 0) + sums * (np.abs(G) @ np.abs(x))
    eu = left_over(U, x, 0) + sums * (np.abs(U) @ np.abs(x))
    s = g / (1 + np.exp(-g))
    h = s * u
    eh = 1.1 * eg * (np.abs(u) + eu) + np.abs(s) * eu + 2.0 ** -21 * np.abs(h)
    y = D @ h
    bound = np.abs(D) @ eh + left_over(D, h, eh) + (I / 16 + 64) * 2.0 ** -22 * (np.abs(D) @ np.abs(h))
    return y, bound


def check(y, want, bound):
    got = y.double().cpu().numpy()
    bound = bound + 2.0 ** -8 * (np.abs(want) + bound)  # the rounding to bf16
    err = np.abs(got - want)
    assert np.all(err <= bound), float((err / bound).max())


@pytest.mark.parametrize("T,E,top,H,I", [(1, 2, 1, 256, 96), (3, 3, 2, 2048, 64), (20, 4, 2, 544, 192),
                                         (64, 2, 2, 128, 32), (16, 1, 1, 256, 64), (17, 1, 1, 256, 64),
                                         (22, 1, 1, 512, 64), (23, 1, 1, 1024, 96), (45, 1, 1, 256, 64)])
def test_small_values_beside_loud_ones(mhr, T, E, top, H, I):
    """A value 2^12 times the others in every block of x, and of h, that no weight multiplies: y is
    made of what the first terms leave."""
    import torch

    rng = np.random.default_rng(T + H)
    loud_x = set(b * 32 + b * 5 % 32 for b in range(H // 32))
    loud_h = set(b * 32 + b * 7 % 32 for b in range(I // 32))
    x = rng.standard_normal((T, H))
    x[:, sorted(loud_x)] *= 2.0 ** 12
    x = bf16(x)
    router = bf16(rng.standard_normal((E, H)) * H ** -0.5)
    router[:, sorted(loud_x)] = 0
    codes, scales = sparse(rng, 2 * E * I, H, -2, loud_x)
    scales.reshape(E, 2, I, -1)[:, :, sorted(loud_h)] += 6  # gate and up rows of the loud h
    up, upv = matrix(codes, scales)
    down, downv = matrix(*sparse(rng, E * H, I, 0, loud_h))
    y, experts, weights = mhr.moe_mxfp4(torch.from_numpy(x).bfloat16().cuda(),
                                        torch.from_numpy(router).bfloat16().cuda(), up, down, top)
    assert mhr.gemm_check(None) == mhr.MHR_OK
    upv, downv = upv.reshape(E, 2, I, H), downv.reshape(E, H, I)
    for t in range(T):
        want, bound = np.zeros(H), np.zeros(H)
        for e, w in zip(experts[t].tolist(), weights[t].double().tolist()):
            v, b = expected(x[t], upv[e, 0], upv[e, 1], downv[e])
            want, bound = want + w * v, bound + w * (b + 2.0 ** -22 * np.abs(v))
        check(y[t], want, bound)


def test_silu_of_gates_far_below_zero(mhr):
    """Pairs of inner values that cancel to 16 bits, one of a gate from -10 to -85 and one of a gate
    of 32 (whose silu is 32): what is left shows the error of the first's silu."""
    import torch

    n, H, I = 32, 128, 64
    gates = bf16(-np.linspace(10, 85, n))
    silu = gates / (1 + np.exp(-gates))
    shift = np.ceil(np.log2(16 / np.abs(silu))).astype(int)  # h in [16, 32)
    h = silu * np.exp2(shift)
    high = bf16(-h / 32)
    low = bf16(-h / 32 - high)
    # x: a gate of 32 and a one, the gates, the high and the low parts of the others' up values
    x = np.zeros((1, H))
    x[0, :2], x[0, 32:64], x[0, 64:96], x[0, 96:] = (32, 1), gates, high, low
    j = np.arange(n)
    codes, scales = np.zeros((2 * I, H), np.uint8), np.full((2 * I, H // 32), 127, np.uint8)
    codes[j, 32 + j] = 2               # (code 2: one)
    codes[n + j, 0] = 2
    codes[I + j, 1], scales[I + j, 0] = 2, 127 + shift
    codes[I + n + j, 64 + j] = codes[I + n + j, 96 + j] = 2
    up, _ = matrix(codes, scales)
    codes = np.zeros((H, I), np.uint8)
    codes[j, j] = codes[j, n + j] = 2
    down, _ = matrix(codes, np.full((H, I // 32), 127, np.uint8))
    y, _, weights = mhr.moe_mxfp4(torch.from_numpy(x).bfloat16().cuda(),
                                  torch.zeros(1, H, device="cuda").bfloat16(), up, down, 1)
    assert mhr.gemm_check(None) == mhr.MHR_OK and float(weights) == 1
    want = h + 32 * (high + low)
    # silu and its product 2.5 x 2^-23 (gate and up are exact); both h in 8 terms 2^-22 of at most
    # 32; the sums of the terms, eight of them twice, 2^-23 each of at most 64
    bound = 2.5 * 2.0 ** -23 * 32 + 2 * 2.0 ** -22 * 32 + 4 * 2.0 ** -23 * 64
    check(y[0, :n], want, np.full(n, bound))
    assert bool((y[0, n:] == 0).all())


@pytest.mark.parametrize("m", [96, 104, 108, 112, 116, 120, 124, 126])
def test_blocks_near_the_smallest_numbers(mhr, m):
    """x of some 2^-m times weights of some 2^m, and the same of h."""
    import torch

    rng = np.random.default_rng(m)
    T, H, I = 3, 64, 64
    x = bf16(rng.standard_normal((T, H)) * np.exp2(-m))
    up, upv = matrix(*sparse(rng, 2 * I, H, m))
    down, downv = matrix(*sparse(rng, H, I, 0))
    router = torch.zeros(1, H, device="cuda").bfloat16()
    y = mhr.moe_mxfp4(torch.from_numpy(x).bfloat16().cuda(), router, up, down, 1)[0]
    for t in range(T):
        check(y[t], *expected(x[t], upv[:I], upv[I:], downv))
    x = bf16(rng.standard_normal((T, H)))
    up, upv = matrix(*sparse(rng, 2 * I, H, -(m // 2)))
    down, downv = matrix(*sparse(rng, H, I, m))
    y = mhr.moe_mxfp4(torch.from_numpy(x).bfloat16().cuda(), router, up, down, 1)[0]
    assert mhr.gemm_check(None) == mhr.MHR_OK
    for t in range(T):
        check(y[t], *expected(x[t], upv[:I], upv[I:], downv))


@pytest.mark.parametrize("value", [float("inf"), float("-inf"), float("nan")])
def test_infinite_token(mhr, value):
    """Its logits are infinities or NaN, so its weights and y are NaN; other tokens keep theirs."""
    import torch

    rng = np.random.default_rng(2)
    T, E, H, I = 5, 6, 96, 64
    x = torch.from_numpy(bf16(rng.standard_normal((T, H)))).bfloat16().cuda()
    router = torch.from_numpy(bf16(rng.standard_normal((E, H)))).bfloat16().cuda()
    up, _ = matrix(*sparse(rng, 2 * E * I, H, -2))
    down, _ = matrix(*sparse(rng, E * H, I, 0))
    want = mhr.moe_mxfp4(x, router, up, down, 2)
    x[3, 40] = value
    y, experts, weights = mhr.moe_mxfp4(x, router, up, down, 2)
    keep = [0, 1, 2, 4]
    assert all(torch.equal(g[keep], w[keep]) for g, w in zip((y, experts, weights), want))
    assert bool(torch.isnan(y[3]).all()) and bool(torch.isnan(weights[3]).all())
    assert bool(((experts >= 0) & (experts < E)).all())


def test_the_most_segments(mhr):
    """The shape whose blocks get the most runs of items that share an expert and a part of K:
    64 tokens in one call against 8 at a time (both fp32 sums rounded to bf16, in other orders)."""
    import torch

    E, top, H, I = 512, 8, 15700, 16
    gen = torch.Generator(device="cuda").manual_seed(1)

    def packed(rows, cols):
        codes = torch.randint(0, 256, (rows, -(-cols // 32) * 16), dtype=torch.uint8, device="cuda", generator=gen)
        if cols % 32:
            codes[:, cols // 2:] = 0  # (cols even: the last block's columns past cols)
        return mhr.MxFp4Matrix(codes, torch.randint(118, 122, (mhr.mxfp4_scale_bytes(rows, cols),),
                                                    dtype=torch.uint8, device="cuda", generator=gen), rows, cols)

    up, down = packed(2 * E * I, H), packed(E * H, I)
    x = torch.randn(64, H, device="cuda", generator=gen).bfloat16()
    router = torch.randn(E, H, device="cuda", generator=gen).bfloat16()
    x[:, :8] = 8
    router[:8, :8] += 64  # eight experts that every token chooses
    y, experts, _ = mhr.moe_mxfp4(x, router, up, down, top)
    assert mhr.gemm_check(None) == mhr.MHR_OK
    assert bool((experts.sort(1)[0] == torch.arange(8, device="cuda")).all())
    parts = torch.cat([mhr.moe_mxfp4(x[i:i + 8], router, up, down, top)[0] for i in range(0, 64, 8)])
    assert float((y.float() - parts.float()).norm() / parts.float().norm()) < 2.0 ** -8
