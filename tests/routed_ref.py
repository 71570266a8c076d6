"""The routed operators in 64-bit numpy, one row at a time where that is the definition."""
import numpy as np


def scores(x, kind):
    """softmax or sigmoid of the rows of float64 x; a row of -inf has scores of zero."""
    with np.errstate(invalid="ignore", over="ignore"):
        if kind == "sigmoid":
            e = np.exp(-np.abs(x))
            return np.where(x >= 0, 1 / (1 + e), e / (1 + e))
        m = x.max(1, keepdims=True)
        none = m == -np.inf
        e = np.exp(x - np.where(none, 0, m))
        return np.where(none, 0, e / np.where(none, 1, e.sum(1, keepdims=True)))


def best(keys, n):
    """Indices of the n largest of a list, descending, ties to the lowest, NaN largest."""
    k = [(np.inf, 1) if np.isnan(v) else (v, 0) for v in keys]
    return sorted(range(len(k)), key=lambda i: (-k[i][1], -k[i][0], i))[:n]


def choose(x, top, score="softmax", bias=None, groups=1, group_top=1, group_score="max",
           renormalize=True, scale=1.0):
    s = scores(x, score)
    T, E = x.shape
    size = E // groups
    experts = np.zeros((T, top), np.int32)
    weights = np.zeros((T, top))
    for t in range(T):
        with_bias = s[t] + (0 if bias is None else bias)
        keys = x[t] if bias is None else with_bias
        open_ = range(groups)
        if groups > 1:
            worth = []
            for g in range(groups):
                if group_score == "max":
                    k = keys[g * size:(g + 1) * size]
                    worth.append(k[best(k, 1)[0]])
                else:
                    k = with_bias[g * size:(g + 1) * size]
                    worth.append(k[best(k, 2)].sum())
            open_ = best(worth, group_top)
        members = [e for g in sorted(open_) for e in range(g * size, (g + 1) * size)]
        experts[t] = [members[i] for i in best(keys[members], top)]
        if not renormalize:
            weights[t] = s[t, experts[t]] * scale
            continue
        l = x[t, experts[t]]
        if score == "softmax":
            weights[t] = scores(l[None], "softmax")[0] * scale
        elif l.max() < -700:  # sigmoid(l) = e^l there, which 64 bits cannot hold either
            weights[t] = scores(l[None], "softmax")[0] * scale
        else:
            weights[t] = s[t, experts[t]] / s[t, experts[t]].sum() * scale
    return experts, weights


def choose_grad(x, experts, g, score="softmax", renormalize=True, scale=1.0):
    """By the chain rule through the scores, duplicates added up, entries outside left out."""
    s = scores(x, score)
    T, E = x.shape
    out = np.zeros((T, E))
    for t in range(T):
        j = [i for i in range(experts.shape[1]) if 0 <= experts[t, i] < E]
        at, gj = experts[t, j], g[t, j]
        sj = s[t, at]
        if renormalize:
            total = sj.sum()
            ds = scale * (gj - (sj * gj).sum() / total) / total if total else 0 * sj
        else:
            ds = scale * gj
        of = np.zeros(E)
        np.add.at(of, at, ds)
        if score == "softmax":
            out[t] = s[t] * (of - (s[t] * of).sum())
        else:
            out[t] = of * s[t] * (1 - s[t])
    return out


def sort(experts, count):
    flat = np.where((experts >= 0) & (experts < count), experts, count).reshape(-1)
    offsets = np.searchsorted(np.sort(flat), np.arange(count + 1))
    return offsets.astype(np.int32), np.argsort(flat, kind="stable").astype(np.int32)


def product(x, w, offsets, rows, gather=None, scatter=None, top=1, transposed=False, out=None):
    """`out` (float64, left as it is where nothing is written) for float64 x and w."""
    for e in range(w.shape[0]):
        for q in range(offsets[e], offsets[e + 1]):
            r = q if gather is None else (gather[q] // top if gather[q] >= 0 else -1)
            to = q if scatter is None else scatter[q]
            if 0 <= to < out.shape[0]:
                row = x[r] if 0 <= r < x.shape[0] else np.zeros(x.shape[1])
                out[to] = row @ (w[e].T if transposed else w[e])
    return out


def weight_grad(x, g, offsets, gather=None, scatter=None, top=1):
    E = len(offsets) - 1
    out = np.zeros((E, x.shape[1], g.shape[1]))
    for e in range(E):
        for q in range(offsets[e], offsets[e + 1]):
            r = q if gather is None else (gather[q] // top if gather[q] >= 0 else -1)
            to = q if scatter is None else scatter[q]
            if 0 <= r < x.shape[0] and 0 <= to < g.shape[0]:
                out[e] += np.outer(x[r], g[to])
    return out


def adapters(y, x, down, up, which, scales=None):
    out = y.copy()
    for t, a in enumerate(which):
        if 0 <= a < down.shape[0]:
            out[t] += (1 if scales is None else scales[a]) * ((x[t] @ down[a].T) @ up[a])
    return out
