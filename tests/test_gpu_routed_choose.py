"""The router, its gradient and the sort by expert on the GPU, against 64-bit numpy (routed_ref)."""
import numpy as np
import pytest

import routed_ref as ref

pytestmark = pytest.mark.gpu


def types():
    import torch

    return {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def half_step(dtype):
    return {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}[dtype]


# Weights in fp32 from logits held exactly: expf (2 ulp) of a difference that is rounded
# (|l| <= 16 here: 16 * 2^-24 relative), sums of up to 16 + 5 roundings, a division and two
# products: less than 2 * 2^-23 + 16 * 2^-24 + 24 * 2^-24 = 44 * 2^-24.
WEIGHTS = 44 * 2.0 ** -24


def check(mhr, x, top, **kw):
    """x: a CUDA tensor; bias in kw as numpy."""
    import torch

    bias = kw.pop("bias", None)
    gpu = None if bias is None else torch.from_numpy(bias.astype(np.float32)).cuda()
    e, w = mhr.choose_experts(x, top, bias=gpu, **kw)
    x64 = x.double().cpu().numpy()
    b64 = None if bias is None else bias.astype(np.float32).astype(np.float64)
    want_e, want_w = ref.choose(x64, top, bias=b64, **kw)
    assert e.dtype == torch.int32 and w.dtype == torch.float32
    assert np.array_equal(e.cpu().numpy(), want_e)
    got = w.double().cpu().numpy()
    assert np.array_equal(np.isnan(got), np.isnan(want_w))
    fine = ~np.isnan(want_w)
    assert np.all(np.abs(got - want_w)[fine] <= WEIGHTS * np.abs(want_w)[fine] + 2.0 ** -126)
    return e, w


def normal(T, E, dtype, seed, std=1.5):
    import torch

    x = np.random.default_rng(seed).standard_normal((T, E)) * std
    return torch.from_numpy(np.clip(x, -8, 8)).to(types()[dtype]).cuda()


@pytest.mark.parametrize("renormalize", [True, False])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("T,E,top", [(1, 1, 1), (3, 2, 2), (5, 8, 3), (70, 60, 6), (33, 128, 8),
                                     (9, 257, 16), (17, 512, 16)])
def test_choose(mhr, T, E, top, dtype, score, renormalize):
    x = normal(T, E, dtype, T + E)
    check(mhr, x, top, score=score, renormalize=renormalize)
    bias = np.random.default_rng(1).standard_normal(E) * 0.1
    check(mhr, x, top, score=score, renormalize=renormalize, bias=bias, scale=2.5)


@pytest.mark.parametrize("group_score", ["max", "top2"])
@pytest.mark.parametrize("bias", [True, False])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,groups,group_top,top",
                         [(256, 8, 4, 8), (64, 32, 5, 4), (60, 12, 3, 6), (63, 7, 2, 16),
                          (17, 17, 4, 3), (512, 2, 1, 16), (510, 17, 2, 9), (96, 3, 1, 5),
                          (40, 5, 5, 8)])
def test_choose_in_groups(mhr, E, groups, group_top, top, score, bias, group_score):
    b = np.random.default_rng(2).standard_normal(E) * 0.1 if bias else None
    for dtype in ("f32", "bf16"):
        check(mhr, normal(40, E, dtype, E), top, score=score, bias=b, groups=groups,
              group_top=group_top, group_score=group_score)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_ties_go_to_the_lowest_index(mhr, score):
    import torch

    x = torch.randint(0, 3, (64, 96), generator=torch.Generator().manual_seed(3)).float().cuda()
    check(mhr, x, 16, score=score)
    check(mhr, x, 16, score=score, bias=np.zeros(96))
    check(mhr, x, 9, score=score, groups=8, group_top=3, group_score="top2")
    check(mhr, x, 9, score=score, groups=8, group_top=3)
    x = torch.zeros(4, 50, device="cuda")
    x[:, ::2] = -0.0  # equal to 0
    e, _ = check(mhr, x, 7, score=score)
    assert e[0].tolist() == list(range(7))


@pytest.mark.parametrize("groups", [1, 8])
def test_neighbours_that_32_bits_do_not_tell_apart(mhr, groups):
    """Keys whose order only 64 bits give: a bias that undoes the scores' differences but for
    parts of 2^-26 and less."""
    import torch

    rng = np.random.default_rng(5)
    E, T = 128, 200
    x = rng.uniform(-3, 3, E).astype(np.float32)
    bias = (0.75 - ref.scores(x.astype(np.float64)[None], "sigmoid")[0]).astype(np.float32)
    rows = np.repeat(x[None], T, 0)
    rows[:, rng.integers(0, E, T)] += np.float32(2.0 ** -21)
    kw = dict(score="sigmoid", bias=bias, groups=groups, group_top=max(1, groups // 2),
              group_score="top2")
    check(mhr, torch.from_numpy(rows).cuda(), 8, **kw)
    keys = ref.scores(rows.astype(np.float64), "sigmoid") + bias.astype(np.float64)
    near = np.diff(np.sort(keys[0])[-9:])
    assert near.max() < 2.0 ** -24  # the case is what it says


@pytest.mark.parametrize("E,groups", [(20, 1), (128, 1), (128, 4), (300, 1)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_a_few_such_neighbours(mhr, E, groups, score):
    """Some of the best keys in runs of such neighbours, the others far off."""
    import torch

    rng = np.random.default_rng(7)
    T, top = 300, 8
    x = rng.uniform(-3, 3, (T, E)).astype(np.float32)
    x[:, E // 2:] = x[0, E // 2:]  # one row's bias undoes the differences in all
    x -= x.mean()
    bias = np.zeros(E, np.float32)
    if score == "softmax":  # alike sums: the other half's logits are low
        x[:, :E // 2] -= 30
    s = ref.scores(x.astype(np.float64), score)[0]
    run = np.arange(E // 2, E // 2 + 6)
    bias[run] = (s.max() + 0.5 - s[run]).astype(np.float32)
    bias[run[3:]] -= 0.1
    check(mhr, torch.from_numpy(x).cuda(), top, score=score, bias=bias, groups=groups,
          group_top=max(1, groups - 1))
    keys = np.sort(s + bias)[::-1]
    assert np.diff(-keys[:3]).max() < 2.0 ** -23 and keys[2] - keys[3] > 0.05


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [True, False])
def test_masked_and_special_logits(mhr, score, renormalize):
    import torch

    inf, nan = float("inf"), float("nan")
    x = normal(10, 48, "f32", 6)
    x[0, 5:] = -inf           # fewer experts than asked for are left
    x[1] = -inf               # none is: weights of zero
    x[2] = torch.finfo(torch.float32).min
    x[3, 7] = nan
    x[4, 9] = inf if score == "sigmoid" else 8.0
    x[5, ::2] = -inf
    x[6, 3:] = torch.finfo(torch.float32).min
    x[7] = -500.0 - torch.arange(48, device="cuda") / 8  # scores that 32 bits do not hold
    x[8] = nan
    kw = dict(score=score, renormalize=renormalize)
    e, w = check(mhr, x, 8, **kw)
    assert e[1].tolist() == list(range(8)) and float(w[1].abs().sum()) == 0
    assert e[8].tolist() == list(range(8)) and bool(w[8].isnan().all())
    if renormalize:
        assert abs(float(w[7].sum()) - 1) < 1e-5
    bias = np.random.default_rng(1).standard_normal(48) * 0.1
    x[3, 7] = 0.0
    x[8] = 0.0
    check(mhr, x, 8, bias=bias, **kw)
    check(mhr, x, 8, groups=6, group_top=2, **kw)


def test_choose_strided_unaligned_and_far(mhr):
    import torch

    big = normal(30, 300, "bf16", 8)
    check(mhr, big[:, 1:65], 4)
    check(mhr, big[::2, :64], 4, groups=8, group_top=3)
    check(mhr, big[3:4, 7:8], 1)
    assert mhr.choose_experts(big[:0], 3)[0].shape == (0, 3)
    # rows whose offsets pass 2^31 elements
    far = torch.zeros(1, dtype=torch.bfloat16, device="cuda")
    pitch = (1 << 31) // 3 + 8
    wide = torch.zeros(3 * pitch + 64, dtype=torch.bfloat16, device="cuda")
    x = torch.as_strided(wide, (4, 64), (pitch, 1))
    x.copy_(normal(4, 64, "bf16", 9))
    check(mhr, x, 8)
    del far, wide


GRADS = [(s, r) for s in ("softmax", "sigmoid") for r in (True, False)]


@pytest.mark.parametrize("score,renormalize", GRADS)
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("T,E,top", [(1, 1, 1), (5, 8, 3), (70, 60, 6), (33, 128, 8), (9, 257, 16),
                                     (6, 512, 16)])
def test_choose_grad(mhr, T, E, top, dtype, score, renormalize):
    import torch

    x = normal(T, E, dtype, T * E)
    e, _ = mhr.choose_experts(x, top, score=score)
    g = np.random.default_rng(T).standard_normal((T, top)).astype(np.float32)
    got = mhr.choose_experts_grad(x, e, torch.from_numpy(g).cuda(), score=score,
                                  renormalize=renormalize, scale=2.5)
    assert got.dtype == x.dtype
    want = ref.choose_grad(x.double().cpu().numpy(), e.cpu().numpy(), g.astype(np.float64),
                           score, renormalize, 2.5)
    err = np.abs(got.double().cpu().numpy() - want)
    # as WEIGHTS, of scale * |g| at most twice over (g less its mean), times the score; then the
    # rounding to the logits' type
    size = 2.5 * 2 * np.abs(g).max(1, keepdims=True)
    floor = 2.0 ** -25 if dtype == "f16" else 0  # half a step of fp16's subnormals
    assert np.all(err <= 2 * WEIGHTS * size + half_step(dtype) * np.abs(want) + floor)


@pytest.mark.parametrize("score,renormalize", GRADS)
def test_choose_grad_against_differences(mhr, score, renormalize):
    """Of the forward call's own weights, in fp32."""
    import torch

    T, E, top, h = 12, 40, 5, 2.0 ** -7
    x = normal(T, E, "f32", 4)
    kw = dict(score=score, renormalize=renormalize)
    e, _ = mhr.choose_experts(x, top, **kw)
    g = torch.randn(T, top, generator=torch.Generator().manual_seed(1)).cuda()
    got = mhr.choose_experts_grad(x, e, g, **kw)

    def loss(x):
        w = ref.choose(x.double().cpu().numpy(), top, **kw)
        assert np.array_equal(w[0], e.cpu().numpy())  # the choice is held
        return (w[1] * g.double().cpu().numpy()).sum(1)

    checked = 0
    for c in range(E):
        d = torch.zeros_like(x)
        d[:, c] = h
        try:
            diff = (loss(x + d) - loss(x - d)) / (2 * h)
        except AssertionError:
            continue  # the step changes the choice
        # third derivatives of a score are below 1: h^2 / 6 of |g|, twice over
        assert np.all(np.abs(got[:, c].double().cpu().numpy() - diff) <= h * h * float(g.abs().max()) + 1e-5)
        checked += 1
    assert checked > 4


@pytest.mark.parametrize("score,renormalize", GRADS)
def test_choose_grad_of_odd_rows(mhr, score, renormalize):
    import torch

    x = normal(6, 50, "f32", 11)
    x[0] = float("-inf")
    x[1, 3:] = float("-inf")
    x[2] = torch.finfo(torch.float32).min
    e, _ = mhr.choose_experts(x, 6, score=score)
    e[3, 2] = e[3, 0]         # one expert twice
    e[4, 1], e[4, 3] = -1, 50  # entries outside
    e[5] = -1
    g = torch.randn(6, 6, generator=torch.Generator().manual_seed(2)).cuda()
    got = mhr.choose_experts_grad(x, e, g, score=score, renormalize=renormalize)
    want = ref.choose_grad(x.double().cpu().numpy(), e.cpu().numpy(), g.double().cpu().numpy(),
                           score, renormalize)
    rows = [0, 1, 3, 4, 5] if score == "sigmoid" and renormalize else range(6)
    for t in rows:  # (row 2's sigmoids are 0 in 64 bits, and their shares with them)
        assert np.allclose(got[t].double().cpu().numpy(), want[t], rtol=1e-5, atol=1e-5), t
    # out with a pitch of its own, off 16 bytes
    buf = torch.full((6, 61), 7.0, device="cuda")
    mhr.choose_experts_grad(x, e, g, score=score, renormalize=renormalize, out=buf[:, 3:53])
    assert torch.equal(buf[:, 3:53], got)
    assert bool((buf[:, :3] == 7).all()) and bool((buf[:, 53:] == 7).all())


@pytest.mark.parametrize("n,count", [(0, 5), (1, 1), (8, 128), (31, 3), (64, 128), (1000, 60),
                                     (4096, 1), (4097, 256), (50000, 512), (131072, 256),
                                     (300001, 1024)])
def test_sort(mhr, n, count):
    import torch

    rng = np.random.default_rng(n)
    e = rng.integers(-2, count + 2, n).astype(np.int32)
    offsets, order = mhr.sort_by_expert(torch.from_numpy(e).cuda(), count)
    want = ref.sort(e, count)
    assert np.array_equal(offsets.cpu().numpy(), want[0])
    assert np.array_equal(order.cpu().numpy(), want[1])


def test_sort_of_equal_and_of_outside_entries(mhr):
    import torch

    for e in (np.zeros(9999), np.full(777, -1), np.full(50, 2 ** 31 - 1)):
        offsets, order = mhr.sort_by_expert(torch.from_numpy(e.astype(np.int32)).cuda(), 7)
        want = ref.sort(e.astype(np.int64), 7)
        assert np.array_equal(offsets.cpu().numpy(), want[0])
        assert np.array_equal(order.cpu().numpy(), want[1])


def test_on_another_stream_and_captured(mhr):
    import torch

    x = normal(300, 96, "f32", 13)
    want = check(mhr, x, 6, score="sigmoid")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        e, w = mhr.choose_experts(x, 6, score="sigmoid")
    s.synchronize()
    assert torch.equal(e, want[0]) and torch.equal(w, want[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        e, w = mhr.choose_experts(x, 6, score="sigmoid")
        offsets, order = mhr.sort_by_expert(e, 96)
        d = mhr.choose_experts_grad(x, e, w, score="sigmoid")
    x.copy_(normal(300, 96, "f32", 14))
    graph.replay()
    want = mhr.choose_experts(x, 6, score="sigmoid")
    assert torch.equal(e, want[0]) and torch.equal(w, want[1])
    assert torch.equal(d, mhr.choose_experts_grad(x, e, w, score="sigmoid"))
    again = mhr.sort_by_expert(e, 96)
    assert torch.equal(offsets, again[0]) and torch.equal(order, again[1])
