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


@pytest.mark.parametrize("T", [6, 300, 700])
@pytest.mark.parametrize("rank", [1, 8, 16, 70])
@pytest.mark.parametrize("dtype,out", [("bf16", "bf16"), ("bf16", "f32"), ("f16", "f16")])
def test_infinities_of_x_are_the_definitions(mhr, T, rank, dtype, out):
    """Which outputs are an infinity, of which sign, and which are NaN does not depend on how many
    rows there are, or on the rank's being no multiple of 16."""
    import torch

    rng = np.random.default_rng(rank)
    K, N = 72, 136
    x = rng.integers(-3, 4, (T, K)).astype(np.float32)
    x[1, 5], x[2, 71], x[4, 0] = np.inf, -np.inf, np.nan
    down = rng.choice([-1.0, 1.0], (2, rank, K)).astype(np.float32)
    up = rng.choice([-1.0, 1.0], (2, rank, N)).astype(np.float32)
    up[:, :, :N // 2] = down[:, :, 5:6]  # columns in which a row's infinities have one sign
    x, down, up = (torch.from_numpy(t).to(types()[dtype]).cuda() for t in (x, down, up))
    y = torch.from_numpy(rng.integers(-50, 51, (T, N))).to(types()[out]).cuda()
    which = (torch.arange(T, dtype=torch.int32, device="cuda") // 3) % 2
    which[5] = -1
    with np.errstate(invalid="ignore"):
        want = ref.adapters(f64(y), f64(x), f64(down), f64(up), which.cpu().numpy())
    assert np.isinf(want[1]).sum() >= N // 2 and np.isnan(want[4]).all()
    same(mhr.add_adapters(y, x, down, up, which), want)


@pytest.mark.parametrize("T", [6, 300])
@pytest.mark.parametrize("dtype,out", [("bf16", "f32"), ("f16", "f16"), ("f16", "f32")])
def test_an_infinity_of_down_leaves_the_other_sums(mhr, T, dtype, out):
    """Beside it, sums that fp16 does not hold."""
    import torch

    rng = np.random.default_rng(7)
    K, N, rank = 64, 72, 12
    x = 64.0 * rng.integers(1, 4, (T, K))
    down = 256.0 * rng.choice([-1.0, 1.0], (2, rank, K))
    down[0, 4, 3] = np.inf
    up = rng.choice([-1.0, 1.0], (2, rank, N))
    x, down, up = (torch.from_numpy(t).to(types()[dtype]).cuda() for t in (x, down, up))
    y = torch.zeros(T, N, dtype=types()[out], device="cuda")
    which = (torch.arange(T, dtype=torch.int32, device="cuda") // 3) % 2
    want = ref.adapters(f64(y), f64(x), f64(down), f64(up), which.cpu().numpy())
    assert np.isinf(want[:3]).all() and np.abs(want[3:6]).max() > 2.0 ** 17
    same(mhr.add_adapters(y, x, down, up, which), want)


@pytest.mark.parametrize("T", [6, 300])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("exponent", [-126, -115, -100, 100, 112, 118])
def test_adapters_of_far_scales(mhr, T, dtype, exponent):
    """Sums between the products next to either end of fp32's range. All values are whole numbers
    times a power of two, and no larger than 2^127."""
    import torch

    rng = np.random.default_rng(3)
    K, N, rank = 64, 72, 5
    x, down, up = (torch.from_numpy(rng.integers(-3, 4, s)).to(types()[dtype]).cuda()
                   for s in ((T, K), (2, rank, K), (2, rank, N)))
    if exponent > 0:
        up = up * 2.0 ** -12
    y = torch.zeros(T, N, device="cuda")
    which = (torch.arange(T, dtype=torch.int32, device="cuda") // 3) % 2
    scales = torch.full((2,), 2.0 ** exponent, device="cuda")
    assert float(scales[0]) == 2.0 ** exponent
    got = mhr.add_adapters(y, x, down, up, which, scales)
    want = ref.adapters(f64(y), f64(x), f64(down), f64(up), which.cpu().numpy(), f64(scales))
    assert bool(np.abs(want).max() < 2.0 ** 127)
    same(got, want)


def parts_of(offsets, rows):
    """Where each expert's rows start and end, by the header's words."""
    parts, last = [], 0
    for a, b in zip(offsets[:-1], offsets[1:]):
        a, b = (min(max(v, 0), rows) for v in (a, b))
        start = max(a, last)
        parts.append((start, max(b, start)))
        if b > a:
            last = max(last, b)
    return parts


FALLING = [[0, 10, 0, 10], [0, 5, 3, 10], [3, 1, 99], [-7, 4, -1, 6, 2, 9], [9, 0, 4, 3, 8, 8, 1],
           [0] + [7, 3] * 60 + [16], list(range(16, -1, -1))]


@pytest.mark.parametrize("rows", [16, 400])
@pytest.mark.parametrize("offsets", FALLING, ids=lambda o: str(o[:7]))
def test_offsets_that_fall(mhr, offsets, rows):
    """No position belongs to two experts: products and gradients repeat, and count it once."""
    import torch

    scale = rows // 16
    at = [v * scale for v in offsets]
    E = len(at) - 1
    rng = np.random.default_rng(E)
    x, w, g = (torch.from_numpy(rng.integers(-3, 4, s)).bfloat16().cuda()
               for s in ((rows, 72), (E, 72, 136), (rows, 136)))
    o = torch.tensor(at, dtype=torch.int32, device="cuda")
    parts = parts_of(at, rows)
    owner = np.zeros(rows, int)
    for start, end in parts:
        owner[start:end] += 1
    assert owner.max() <= 1
    for out_dtype in (torch.bfloat16, torch.float32):
        out = torch.full((rows, 136), 7.0, dtype=out_dtype, device="cuda")
        mhr.matmul_experts(x, w, o, out=out)
        want = np.full((rows, 136), 7.0)
        for e, part in enumerate(parts):
            ref.product(f64(x), f64(w)[e:e + 1], part, rows, out=want)
        same(out, want)
        d = mhr.matmul_experts_grad(x, g, o, out_dtype=out_dtype)
        same(d, np.concatenate([ref.weight_grad(f64(x), f64(g), part) for part in parts]))
    # an operand that is copied first: the same rows
    odd = torch.zeros(E, 72, 137, dtype=torch.bfloat16, device="cuda")[:, :, 1:]
    odd.copy_(w)
    again = torch.full((rows, 136), 7.0, device="cuda")
    mhr.matmul_experts(x, odd, o, out=again)
    same(again, want)
    assert mhr.gemm_check(None) == mhr.MHR_OK


def chosen(mhr, x, bias, top, score, **kw):
    import torch

    e, _ = mhr.choose_experts(torch.from_numpy(x).cuda(), top, score, torch.from_numpy(bias).cuda(),
                              **kw)
    want, _ = ref.choose(x.astype(np.float64), top, score, bias.astype(np.float64), **kw)
    assert np.array_equal(e.cpu().numpy(), want)
    return want


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E", [40, 300])
@pytest.mark.parametrize("apart", [1e-8, 0])
def test_a_far_score_behind_the_first_rejected_key(mhr, score, E, apart):
    """The last chosen and the first rejected key have scores near zero, which 32 bits tell apart
    (or they are the same); behind them, within its own error of both, comes a high score with a negative bias."""
    T, high = 1000, E - 2
    x = np.full((T, E), -30, np.float32)
    bias = np.full(E, -5, np.float32)
    x[:, 3], bias[3] = (1.5, 1) if score == "sigmoid" else (0.1, 1)
    x[:, high] = (score == "sigmoid") + np.random.default_rng(2).uniform(-4e-7, 4e-7, T)
    s = ref.scores(x.astype(np.float64), score)[:, high]
    bias[5], bias[E // 2], bias[high] = 0.01, 0.01 - apart, 0.01 - s.mean()
    want = chosen(mhr, x, bias, 2, score)
    assert set(want[:, 1]) == {5, high}  # the case is what it says


def test_a_far_score_behind_32_candidates(mhr):
    """The same, behind more near keys than a warp has lanes."""
    T, E, high = 500, 128, 100
    x = np.full((T, E), -30, np.float32)
    bias = np.full(E, -5, np.float32)
    x[:, 3], bias[3] = 1.5, 1
    bias[10], bias[11], bias[12:60] = 0.01, 0.01 - 1e-9, 0.01 - 6e-9
    x[:, high] = 1 + np.random.default_rng(2).uniform(-4e-7, 4e-7, T)
    s = ref.scores(x.astype(np.float64), "sigmoid")[:, high]
    bias[high] = 0.01 - s.mean()
    want = chosen(mhr, x, bias, 2, "sigmoid")
    assert {10, high} <= set(want[:, 1])


@pytest.mark.parametrize("depth", [80, 86, 98])
def test_scores_far_below_the_best(mhr, depth):
    """Biases as small as softmax scores of e^-depth, whose argument 32 bits round."""
    rng = np.random.default_rng(1)
    T, E = 20000, 40
    x = np.full((T, E), -200, np.float32)
    x[:, 0] = 40
    step = 2.0 ** -18 if depth < 90 else 2.0 ** -9
    x[:, 3] = 40 - depth + step * rng.integers(-40, 41, T)
    x[:, E - 2] = 39.5 - depth + step * rng.integers(-40, 41, T)
    bias = np.zeros(E, np.float32)
    bias[E - 2] = np.exp(-float(depth)) - np.exp(-depth - 0.5)
    want = chosen(mhr, x, bias, 2, "softmax")
    assert set(want[:, 1]) == {3, E - 2}


@pytest.mark.parametrize("renormalize", [True, False])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("T,E,top", [(5, 8, 3), (70, 60, 6), (33, 128, 8), (40, 512, 16)])
def test_choose_grad_term_by_term(mhr, T, E, top, dtype, score, renormalize):
    """Each element against the size of its own terms, so that a small one counts as a large one
    does. In parts of 2^-24, for |l| <= 8: a score or share is off by 44 of it at most (expf 4, its
    argument 16, sums 21, quotient and product 3); g less its mean by 44 + 16 + 1 of the mean's
    terms; 1 - s, the scale and the last sum by 8 more: 44 + 61 + 8 < 120. Then the type's
    rounding, of fp16 half a step of its subnormals at least."""
    import torch

    rng = np.random.default_rng(T + E)
    x = torch.from_numpy(np.clip(rng.standard_normal((T, E)) * 1.5, -8, 8)).to(types()[dtype]).cuda()
    g = rng.standard_normal((T, top)).astype(np.float32)
    kw = dict(score=score, renormalize=renormalize)
    e, _ = mhr.choose_experts(x, top, **kw)
    got = f64(mhr.choose_experts_grad(x, e, torch.from_numpy(g).cuda(), scale=2.5, **kw))
    x64, at, g = f64(x), e.long().cpu().numpy(), g.astype(np.float64)
    want = ref.choose_grad(x64, at, g, scale=2.5, **kw)
    s = ref.scores(x64, score)
    chosen = np.take_along_axis(s, at, 1)
    total = chosen.sum(1, keepdims=True) if renormalize else 1.0
    mean = (chosen / total * np.abs(g)).sum(1, keepdims=True)
    of = np.zeros((T, E))  # |g| of the chosen, and the mean where it takes part
    np.put_along_axis(of, at, np.abs(g) + (mean if renormalize else 0), 1)
    if score == "softmax" and not renormalize:
        of += mean
    size = 2.5 * s / total * of * (1 - s if score == "sigmoid" else 1)
    step = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}[dtype]
    floor = 2.0 ** -25 if dtype == "f16" else 0
    floor = floor + 2.0 ** -46 * size.sum(1, keepdims=True)
    assert np.all(np.abs(got - want) <= 120 * 2.0 ** -24 * size + step * np.abs(want) + floor)


@pytest.mark.parametrize("out", ["bf16", "f16", "f32"])
def test_long_sums_of_adapters_are_cut(mhr, out):
    """x down^T of 32768 positive terms, less itself in three bf16 values: its error is left. A
    cluster has up to 8 CTAs of up to 4 accumulators, 64 steps of 16 terms each. A step truncates
    by a unit, 2^-23 of the sum so far at most: 64 / 2 of those on average over a growing sum, and
    8 more for what adds up the parts and multiplies them."""
    import torch

    T, K, N = 300, 32768, 64
    gen = torch.Generator().manual_seed(4)
    x, down = torch.rand(T, K, generator=gen).bfloat16(), torch.zeros(1, 4, K).bfloat16()
    down[0, 0] = torch.rand(K, generator=gen).bfloat16()
    down[0, 0, :3] = 0
    v = x.double() @ down[0, 0].double()
    rest = v.clone()
    for i in range(3):
        x[:, i], down[0, i + 1, i] = rest.bfloat16(), 1
        rest -= rest.bfloat16().double()
    up = torch.tensor([1.0, -1.0, -1.0, -1.0]).bfloat16()[None, :, None].repeat(1, 1, N)
    y = torch.zeros(T, N, dtype=types()[out], device="cuda")
    which = torch.zeros(T, dtype=torch.int32, device="cuda")
    got = mhr.add_adapters(y, x.cuda(), down.cuda(), up.contiguous().cuda(), which)
    assert float(rest.abs().max()) < 2.0 ** -24 * float(v.min())
    err = (got.double().cpu().abs() / v[:, None]).mean()
    assert float(err) <= (32 + 8) * 2.0 ** -23, float(err)


@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("out_dtype", ["bf16", "f32"])
def test_a_rows_product_does_not_go_by_the_rows_beside_it(mhr, out_dtype, transposed):
    """Alone, in a tile of few rows, and in the largest: to the last bit."""
    import torch

    gen = torch.Generator(device="cuda").manual_seed(6)
    x = torch.randn(700, 1000, generator=gen, device="cuda").bfloat16()
    w = torch.randn(2, 264, 1000, generator=gen, device="cuda").bfloat16()
    if not transposed:
        w = w.transpose(1, 2).contiguous()
    kw = dict(transposed=transposed, out_dtype=types()[out_dtype])

    def first(rows):
        at = torch.tensor([0, rows, 700], dtype=torch.int32, device="cuda")
        return mhr.matmul_experts(x, w, at, **kw)[:rows]

    whole = first(700)
    for rows in (1, 33, 129, 260):
        assert torch.equal(first(rows), whole[:rows])
    order = torch.arange(700, dtype=torch.int32, device="cuda")
    few = torch.tensor([0, 40, 40], dtype=torch.int32, device="cuda")
    assert torch.equal(mhr.matmul_experts(x, w, few, gather=order[:40], **kw), whole[:40])
