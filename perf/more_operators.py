"""Cases for the operators that go by an index per row: routing, its sort, the experts' products
and low-rank adapters.

* ``choose``: the router of a mixture of experts: scores (softmax or sigmoid) of T x E logits, a bias
  for balance that takes part in the choice alone, a choice of groups first, the top experts in
  descending order (ties to the lowest index) and their weights; ``choose_grad``: the gradient of the
  logits for one of the weights;
* ``sort``: the rows of all experts one expert after the other: the stable order of the (token, slot)
  pairs, and where each expert's part starts;
* ``experts``: ``out[p] = x[row of p] W_e`` over those parts -- forward, with the tokens' rows picked on
  the way (``gather``) or results put back in (token, slot) order (``scatter``), with the transposed
  weights, as the gradient of x is; ``experts_grad``: the gradient of the weights;
* ``adapters``: ``out = y + scale_a (x down_a^T) up_a``, each row with the low-rank adapter of its request.
"""
import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


# ------------------------------------------------------------------------------------- the cases
def listed():
    return [
        # one token of a decoding step: nothing but latency
        dict(name="choose 1x256 sigmoid", op="choose", T=1, E=256, top=8, dtype="f32",
             score="sigmoid", bias=True, groups=8, group_top=4, group_score="top2",
             renormalize=True, scale=2.5),
        # a batch of prompts, the bias-balanced choice in groups
        dict(name="choose 16384x256 sigmoid", op="choose", T=16384, E=256, top=8, dtype="f32",
             score="sigmoid", bias=True, groups=8, group_top=4, group_score="top2",
             renormalize=True, scale=2.5),
        # a training step's way back through a plain softmax router, every logit with a gradient
        dict(name="choose grad 8192x128 softmax", op="choose_grad", T=8192, E=128, top=8,
             dtype="bf16", score="softmax", bias=False, groups=1, group_top=1, group_score="max",
             renormalize=False, scale=1.0),
        # the pairs of a small decoding batch
        dict(name="sort 64 pairs", op="sort", T=8, E=128, top=8),
        # the pairs of a batch of prompts
        dict(name="sort 131072 pairs", op="sort", T=16384, E=256, top=8),
        # one token through its experts' up products: their weights' bytes
        dict(name="experts 1 token", op="experts", T=1, E=128, top=8, K=2048, N=1536, dtype="bf16",
             gather=True, scatter=False, transposed=False),
        # a short prompt, sizes that end inside every tile
        dict(name="experts 333 tokens", op="experts", T=333, E=60, top=6, K=2600, N=1416,
             dtype="f16", gather=True, scatter=False, transposed=False),
        # the largest: a training batch's gradient of the experts' inputs, back in token order
        dict(name="experts 4096 tokens transposed", op="experts", T=4096, E=128, top=8, K=1536,
             N=4096, dtype="bf16", gather=False, scatter=True, transposed=True),
        # the same step's gradient of smaller experts' weights, held in fp32 as optimisers do
        dict(name="experts grad 2048 tokens", op="experts_grad", T=2048, E=64, top=8, K=2048,
             N=1408, dtype="bf16", out="f32", gather=True),
        # one token of one request
        dict(name="adapters 1 token", op="adapters", T=1, K=4096, N=4096, L=32, rank=16,
             dtype="bf16", out="bf16", run=1),
        # a decoding batch of as many requests, some without an adapter, a wide projection
        dict(name="adapters 48 tokens", op="adapters", T=48, K=4096, N=11008, L=64, rank=16,
             dtype="f16", out="f16", run=1),
        # prompts of some requests in one batch
        dict(name="adapters 8192 tokens", op="adapters", T=8192, K=4096, N=4096, L=8, rank=64,
             dtype="bf16", out="bf16", run=700),
    ]


def draw(rng):
    def log(lo, hi, multiple=1):
        return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random() / multiple)) * multiple))

    op = rng.choice(["choose", "choose_grad", "sort", "experts", "experts_grad", "adapters"])
    if op in ("choose", "choose_grad"):
        groups = rng.choice([1, 1, 4, 8])
        size = log(4, 256 // groups)
        group_top = rng.randint(1, groups)
        score = rng.choice(["softmax", "sigmoid"])
        return dict(op=op, T=log(1, 16384), E=groups * size,
                    top=rng.randint(1, min(10, group_top * size)),
                    dtype=rng.choice(["f32", "bf16", "f16"]), score=score,
                    bias=rng.choice([True, False]), groups=groups, group_top=group_top,
                    group_score=rng.choice(["max", "top2"]), renormalize=rng.choice([True, False]),
                    scale=rng.choice([1.0, 2.5]))
    if op == "sort":
        E = log(4, 256)
        return dict(op=op, T=log(1, 16384), E=E, top=rng.randint(1, min(8, E)))
    if op in ("experts", "experts_grad"):
        E = log(4, 128)
        m = rng.choice([1, 8, 64])
        case = dict(op=op, T=log(1, 4096), E=E, top=rng.randint(1, min(8, E)), K=log(64, 4096, m),
                    N=log(64, 1536, m), dtype=rng.choice(["bf16", "f16"]),
                    gather=rng.choice([True, False]))
        if op == "experts":
            return dict(case, scatter=rng.choice([True, False]), transposed=rng.choice([True, False]))
        return dict(case, out=rng.choice(["f32", "same"]))
    T = log(1, 8192)
    m = rng.choice([1, 8, 64])
    return dict(op=op, T=T, K=log(64, 4096, m), N=log(64, 4096, m), L=log(1, 64),
                rank=rng.choice([4, 8, 11, 16, 32, 64]), dtype=rng.choice(["bf16", "f16"]),
                out=rng.choice(["same", "f32"]), run=rng.choice([1, 1 + T // 11, 700]))


def touched(rows, of, each=1):
    """Expected number of ``of`` bins that ``rows`` rows reach, each of them ``each`` bins."""
    return of * (1 - (1 - each / of) ** rows)


def work(case):
    op, T = case["op"], case["T"]
    if op in ("choose", "choose_grad"):
        n, size = T * case["E"], DTYPES[case["dtype"]].itemsize
        pairs = 8 * T * case["top"]
        if op == "choose":
            return {"bytes": n * size + pairs + 4 * case["E"] * case["bias"], "flops": 10 * n}
        # a gradient for the chosen alone asks for their logits only
        whole = case["score"] == "softmax" and not case["renormalize"]
        read = n * size if whole else T * case["top"] * size
        return {"bytes": read + n * size + pairs, "flops": 10 * n}
    if op == "sort":
        return {"bytes": 8 * T * case["top"] + 4 * case["E"] + 4, "flops": 4 * T * case["top"]}
    if op in ("experts", "experts_grad"):
        R, K, N = T * case["top"], case["K"], case["N"]
        rows = T if case["gather"] else R
        if op == "experts":
            weights = touched(T, case["E"], case["top"]) * K * N
            return {"bytes": 2 * (rows * K + weights + R * N), "flops": 2 * R * K * N}
        size = 4 if case["out"] == "f32" else 2
        return {"bytes": 2 * (rows * K + R * N) + size * case["E"] * K * N, "flops": 2 * R * K * N}
    K, N, r = case["K"], case["N"], case["rank"]
    size = 4 if case["out"] == "f32" else 2
    adapters = touched(-(-T // case["run"]), case["L"]) * r * (K + N)
    return {"bytes": 2 * (T * K + adapters) + 2 * size * T * N, "flops": 2 * T * r * (K + N)}


# ------------------------------------------------------------------------------------ the inputs
def normal(shape, gen, std=1.0, dtype=torch.float32):
    return torch.randn(shape, generator=gen, device="cuda", dtype=dtype).mul_(std)


def activations(rows, cols, gen, dtype):
    """Normal values with the few large channels that hidden states have."""
    x = normal((rows, cols), gen)
    loud = torch.rand((cols,), generator=gen, device="cuda") < 0.01
    return torch.where(loud, x * 12, x).to(dtype)


def routed(T, E, top, gen):
    """Experts of T tokens as a router picks them, some more popular than others."""
    score = normal((T, E), gen) + normal((E,), gen, 0.7)
    return torch.sort(score, descending=True, stable=True)[1][:, :top].int()


def options(case):
    return {k: case[k] for k in ("score", "groups", "group_top", "group_score", "renormalize",
                                 "scale")}


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op, T = case["op"], case["T"]
    if op in ("choose", "choose_grad"):
        logits = normal((T, case["E"]), gen, 1.5).to(DTYPES[case["dtype"]])
        bias = normal((case["E"],), gen, 0.05) if case["bias"] else None
        s = dict(case, logits=logits, bias=bias)
        if op == "choose_grad":
            s["experts"] = plain_choose(s)[0]
            s["grad"] = normal((T, case["top"]), gen)
        return s
    if op == "sort":
        return dict(case, experts=routed(T, case["E"], case["top"], gen))
    if op in ("experts", "experts_grad"):
        E, top, K, N = (case[k] for k in ("E", "top", "K", "N"))
        dtype = DTYPES[case["dtype"]]
        offsets, order = plain_sort(routed(T, E, top, gen), E)
        s = dict(case, offsets=offsets, order=order,
                 capacity=int((offsets[1:] - offsets[:-1]).max()))  # rows of the fullest expert
        s["x"] = activations(T if case["gather"] else T * top, K, gen, dtype)
        if op == "experts":
            shape = (E, N, K) if case["transposed"] else (E, K, N)
            s["w"] = normal(shape, gen, K ** -0.5, dtype)
        else:
            s["grad"] = normal((T * top, N), gen, 0.1).to(dtype)
        return s
    K, N, L, r = (case[k] for k in ("K", "N", "L", "rank"))
    dtype = DTYPES[case["dtype"]]
    out = DTYPES[case["out"]] if case["out"] != "same" else dtype
    # the requests' rows lie together; one in sixteen requests but the first has no adapter
    requests = -(-T // case["run"])
    which = torch.randint(0, L, (requests,), generator=gen, device="cuda")
    none = torch.rand((requests,), generator=gen, device="cuda") < 1 / 16
    none[0] = False
    which = torch.where(none, -1, which).repeat_interleave(case["run"])[:T].int()
    return dict(case, x=activations(T, K, gen, dtype), y=normal((T, N), gen).to(out),
                down=normal((L, r, K), gen, K ** -0.5, dtype), up=normal((L, r, N), gen, 0.3, dtype),
                which=which.contiguous(), scales=0.5 + torch.rand((L,), generator=gen, device="cuda"))


# ----------------------------------------------------------------------------------- plain forms
def plain_scores(s):
    x = s["logits"].double()
    if s["score"] == "sigmoid":
        return 1 / (1 + torch.exp(-x))
    e = torch.exp(x - x.amax(-1, keepdim=True))
    return e / e.sum(-1, keepdim=True)


def plain_choose(s):
    """Scores in 64 bits: neighbours that differ in their last bits decide between experts."""
    scores = plain_scores(s)
    T, E = scores.shape
    G, size = s["groups"], E // s["groups"]
    key = scores + s["bias"].double() if s["bias"] is not None else scores
    best = torch.sort(key.reshape(T, G, size), dim=-1, descending=True)[0]
    best = best[..., :2].sum(-1) if s["group_score"] == "top2" else best[..., 0]
    best = torch.sort(best, dim=-1, descending=True, stable=True)[1][:, :s["group_top"]]
    open_ = torch.zeros((T, G), dtype=torch.bool, device=key.device).scatter(1, best, True)
    key = torch.where(open_.repeat_interleave(size, 1), key, -float("inf"))
    experts = torch.sort(key, dim=-1, descending=True, stable=True)[1][:, :s["top"]]
    weights = torch.gather(scores, 1, experts)
    if s["renormalize"]:
        weights = weights / weights.sum(-1, keepdim=True)
    return experts.int(), (weights * s["scale"]).float()


def plain_choose_grad(s):
    at, g, c = s["experts"].long(), s["grad"], s["scale"]
    x = s["logits"].float()
    if s["score"] == "softmax":
        e = torch.exp(x - x.amax(-1, keepdim=True))
        scores = e / e.sum(-1, keepdim=True)
    else:
        scores = 1 / (1 + torch.exp(-x))
    chosen = torch.gather(scores, 1, at)
    if s["renormalize"]:
        total = chosen.sum(-1, keepdim=True)
        share = chosen / total
        of_chosen = c * (g - (share * g).sum(-1, keepdim=True)) / total
    else:
        of_chosen = c * g
    of_scores = torch.zeros_like(x).scatter(1, at, of_chosen)
    if s["score"] == "softmax":
        grad = scores * (of_scores - (scores * of_scores).sum(-1, keepdim=True))
    else:
        grad = of_scores * scores * (1 - scores)
    return grad.to(s["logits"].dtype)


def plain_sort(experts, E):
    flat = experts.reshape(-1).long()
    order = torch.sort(flat, stable=True)[1]
    counts = torch.zeros((E,), dtype=torch.int64, device=flat.device).scatter_add(
        0, flat, torch.ones_like(flat))
    offsets = torch.zeros((E + 1,), dtype=torch.int32, device=flat.device)
    offsets[1:] = counts.cumsum(0)
    return offsets, order.int()


def padded(s):
    """Each expert's rows (E x capacity positions), and which of them there are."""
    at = s["offsets"][:-1, None] + torch.arange(s["capacity"], device="cuda")
    there = at < s["offsets"][1:, None]
    return torch.where(there, at, 0).long(), there


def plain_experts(s):
    at, there = padded(s)
    rows = s["order"].long()[at] // s["top"] if s["gather"] else at
    w = s["w"].float()
    out = s["x"].float()[rows] @ (w.transpose(1, 2) if s["transposed"] else w)
    to = s["order"].long()[at] if s["scatter"] else at
    result = torch.empty((s["order"].numel(), s["N"]), dtype=s["x"].dtype, device="cuda")
    result[to[there]] = out[there].to(s["x"].dtype)
    return result


def plain_experts_grad(s):
    at, there = padded(s)
    rows = s["order"].long()[at] // s["top"] if s["gather"] else at
    x = s["x"].float()[rows] * there.unsqueeze(-1)
    out = x.transpose(1, 2) @ s["grad"].float()[at]
    return out if s["out"] == "f32" else out.to(s["x"].dtype)


def plain_adapters(s):
    """All adapters on every row, and none but the row's own kept between the two products."""
    L, r, K = s["down"].shape
    v = (s["x"].float() @ s["down"].float().reshape(L * r, K).t()).reshape(-1, L, r)
    mine = s["which"].unsqueeze(1) == torch.arange(L, device="cuda")
    v = torch.where(mine.unsqueeze(-1), v * s["scales"].reshape(1, L, 1), 0.0)
    return (s["y"].float() + v.reshape(-1, L * r) @ s["up"].float().reshape(L * r, -1)).to(s["y"].dtype)


# --------------------------------------------------------------------------------------- a pass
def run(s):
    op = s["op"]
    if own:
        import memory_hierarchy_reuse_gb300 as mhr
        order = s.get("order")
        if op == "choose":
            return mhr.choose_experts(s["logits"], s["top"], bias=s["bias"], **options(s))
        if op == "choose_grad":
            return mhr.choose_experts_grad(s["logits"], s["experts"], s["grad"], score=s["score"],
                                           renormalize=s["renormalize"], scale=s["scale"])
        if op == "sort":
            return mhr.sort_by_expert(s["experts"], s["E"])
        if op == "experts":
            return mhr.matmul_experts(s["x"], s["w"], s["offsets"],
                                      gather=order if s["gather"] else None, top=s["top"],
                                      scatter=order if s["scatter"] else None,
                                      transposed=s["transposed"])
        if op == "experts_grad":
            return mhr.matmul_experts_grad(
                s["x"], s["grad"], s["offsets"], gather=order if s["gather"] else None,
                top=s["top"], out_dtype=torch.float32 if s["out"] == "f32" else s["x"].dtype)
        return mhr.add_adapters(s["y"], s["x"], s["down"], s["up"], s["which"], s["scales"])
    if op == "sort":
        return plain_sort(s["experts"], s["E"])
    return {"choose": plain_choose, "choose_grad": plain_choose_grad, "experts": plain_experts,
            "experts_grad": plain_experts_grad, "adapters": plain_adapters}[op](s)


# ----------------------------------------------------------------------------------- in 64 bits
def exact_scores(logits, score):
    if score == "sigmoid":
        return np.where(logits >= 0, 1 / (1 + np.exp(-np.abs(logits))),
                        np.exp(-np.abs(logits)) / (1 + np.exp(-np.abs(logits))))
    e = np.exp(logits - logits.max(1, keepdims=True))
    return e / e.sum(1, keepdims=True)


def exact_choose(case, s):
    x = s["logits"].double().cpu().numpy()
    scores = exact_scores(x, case["score"])
    key = scores + (s["bias"].double().cpu().numpy() if case["bias"] else 0)
    T, E = key.shape
    G = case["groups"]
    if G > 1:
        grouped = np.sort(key.reshape(T, G, E // G), -1)[:, :, ::-1]
        value = grouped[:, :, 0] if case["group_score"] == "max" else grouped[:, :, :2].sum(-1)
        rank = np.argsort(np.argsort(-value, 1, kind="stable"), 1, kind="stable")
        key = np.where(np.repeat(rank < case["group_top"], E // G, 1), key, -np.inf)
    experts = np.argsort(-key, 1, kind="stable")[:, :case["top"]]
    weights = np.take_along_axis(scores, experts, 1)
    if case["renormalize"]:
        weights = weights / weights.sum(1, keepdims=True)
    return torch.from_numpy(experts.astype(np.int32)), torch.from_numpy(weights * case["scale"])


def exact_choose_grad(case, s):
    """The derivative by the weights' logarithms: d log w / d logit, one chosen expert at a time."""
    x, at = s["logits"].double().cpu().numpy(), s["experts"].cpu().numpy()
    g = s["grad"].double().cpu().numpy()
    scores = exact_scores(x, case["score"])
    chosen = np.take_along_axis(scores, at, 1)
    weights = chosen / chosen.sum(1, keepdims=True) if case["renormalize"] else chosen
    weights = weights * case["scale"]
    own_slope = 1 - chosen if case["score"] == "sigmoid" else np.ones_like(chosen)
    grad = np.zeros_like(x)
    rows = np.arange(x.shape[0])
    gw = (g * weights).sum(1)
    for j in range(at.shape[1]):
        grad[rows, at[:, j]] += g[:, j] * weights[:, j] * own_slope[:, j]
        if case["renormalize"]:
            grad[rows, at[:, j]] -= gw * weights[:, j] / case["scale"] * own_slope[:, j]
    if case["score"] == "softmax" and not case["renormalize"]:
        grad -= gw[:, None] * scores
    return torch.from_numpy(grad)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "choose":
        return exact_choose(case, s)
    if op == "choose_grad":
        return exact_choose_grad(case, s)
    if op == "sort":
        flat = s["experts"].cpu().numpy().reshape(-1)
        offsets = np.searchsorted(np.sort(flat), np.arange(case["E"] + 1))
        return (torch.from_numpy(offsets.astype(np.int32)),
                torch.from_numpy(np.argsort(flat, kind="stable").astype(np.int32)))
    if op in ("experts", "experts_grad"):
        at = s["offsets"].tolist()
        order = s["order"].long()
        if op == "experts":
            out = torch.empty((order.numel(), case["N"]), dtype=torch.float64, device="cuda")
        else:
            out = torch.zeros((case["E"], case["K"], case["N"]), dtype=torch.float64, device="cuda")
        for e in range(case["E"]):
            p = torch.arange(at[e], at[e + 1], device="cuda")
            x = s["x"][order[p] // case["top"] if case["gather"] else p].double()
            if op == "experts_grad":
                out[e] = x.t() @ s["grad"][p].double()
            elif p.numel():
                w = s["w"][e].double()
                out[order[p] if case["scatter"] else p] = x @ (w.t() if case["transposed"] else w)
        return out
    out = s["y"].double()
    for a in range(case["L"]):
        t = torch.nonzero(s["which"] == a).flatten()
        v = s["x"][t].double() @ s["down"][a].double().t()
        out[t] += float(s["scales"][a]) * (v @ s["up"][a].double())
    return out
