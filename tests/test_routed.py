"""The routed operators' checks of arguments, without a GPU: refusals come before any CUDA call."""
import pytest

P, Q, R, S = 0x10000, 0x20000000, 0x40000000, 0x60000000  # fake, disjoint, aligned addresses


@pytest.fixture(scope="module")
def mhr():
    from memory_hierarchy_reuse_gb300 import build as b

    b.build()
    import memory_hierarchy_reuse_gb300 as m

    m.load()
    return m


def refused(mhr, name, args, bad):
    """Each change of one argument of a call is refused as invalid."""
    f = getattr(mhr.load(), name)
    for change in bad:
        a = dict(args, **change)
        assert f(*a.values()) == mhr.MHR_ERR_INVALID_ARG, change


def test_choose_refusals(mhr):
    args = dict(dtype=0, logits=P, T=4, E=16, ld=16, score=0, bias=None, groups=4, group_top=2,
                group_score=0, top=3, renormalize=1, scale=1.0, experts=Q, weights=R, stream=None)
    refused(mhr, "gemm_routed_choose", args, [
        dict(dtype=3), dict(dtype=-1), dict(logits=None), dict(T=-1), dict(E=0), dict(E=516, ld=516),
        dict(ld=15), dict(score=2), dict(groups=0), dict(groups=3), dict(E=64, ld=64, groups=64),
        dict(group_top=0), dict(group_top=5), dict(group_score=2), dict(top=0), dict(top=9),
        dict(E=32, ld=32, group_top=4, top=17), dict(experts=None), dict(weights=None),
        dict(logits=P + 2), dict(experts=Q + 2), dict(experts=R), dict(weights=P), dict(bias=Q),
        dict(bias=R + 3), dict(T=1 << 40)])
    assert mhr.load().gemm_routed_choose(*dict(args, T=0, logits=None).values()) == mhr.MHR_OK


def test_choose_grad_refusals(mhr):
    args = dict(dtype=1, logits=P, ld=16, experts=Q, grad=R, T=4, E=16, top=3, score=0,
                renormalize=1, scale=1.0, out=S, ldg=16, stream=None)
    refused(mhr, "gemm_routed_choose_grad", args, [
        dict(dtype=3), dict(logits=None), dict(experts=None), dict(grad=None), dict(out=None),
        dict(T=-1), dict(E=0), dict(E=1024, ld=1024, ldg=1024), dict(top=0), dict(top=17),
        dict(ld=15), dict(ldg=15), dict(score=-1), dict(out=P), dict(out=Q), dict(out=R),
        dict(out=S + 1), dict(grad=R + 2)])
    assert mhr.load().gemm_routed_choose_grad(*dict(args, T=0).values()) == mhr.MHR_OK


def test_sort_refusals(mhr):
    args = dict(experts=P, n=100, E=16, offsets=Q, order=R, stream=None)
    refused(mhr, "gemm_routed_sort", args, [
        dict(n=-1), dict(n=1 << 31), dict(E=0), dict(E=1025), dict(experts=None),
        dict(offsets=None), dict(order=None), dict(offsets=P), dict(order=P), dict(order=Q),
        dict(order=R + 2)])


def test_tensor_calls_refuse(mhr):
    """What the tensor-level calls say before they look for a GPU."""
    import torch

    x = torch.zeros(4, 16)
    e = torch.zeros(4, 3, dtype=torch.int32)
    g = torch.zeros(4, 3)
    for error, match, call in [
            (TypeError, "logits must be a tensor", lambda: mhr.choose_experts([1.0], 1)),
            (TypeError, "logits must be float32", lambda: mhr.choose_experts(x.double(), 1)),
            (ValueError, "2-D", lambda: mhr.choose_experts(x[0], 1)),
            (ValueError, "row-major", lambda: mhr.choose_experts(x.t(), 1)),
            (ValueError, "score", lambda: mhr.choose_experts(x, 1, score="tanh")),
            (ValueError, "CUDA", lambda: mhr.choose_experts(x, 1)),
            (TypeError, "experts must be int32",
             lambda: mhr.choose_experts_grad(x, e.long(), g)),
            (TypeError, "grad_weights must be float32",
             lambda: mhr.choose_experts_grad(x, e, g.half())),
            (ValueError, "T x top", lambda: mhr.choose_experts_grad(x, e[:3], g[:3])),
            (ValueError, "T x top", lambda: mhr.choose_experts_grad(x, e, g[:, :2].contiguous())),
            (ValueError, "contiguous", lambda: mhr.choose_experts_grad(x, e[:, :2], g)),
            (ValueError, "count", lambda: mhr.sort_by_expert(e, 0)),
            (TypeError, "int32", lambda: mhr.sort_by_expert(g, 5)),
            (ValueError, "CUDA", lambda: mhr.sort_by_expert(e, 5))]:
        with pytest.raises(error, match=match):
            call()
