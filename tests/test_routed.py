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


def product_args():
    return dict(dtype=1, x=P, x_rows=20, ldx=64, gather=None, top=1, w=Q, ldw=64, stride_w=4096,
                transposed=0, offsets=R, E=3, out_dtype=1, out=S, out_rows=20, ldo=64,
                scatter=None, rows=20, K=64, N=64, scratch=None, scratch_bytes=0, stream=None)


def test_product_refusals(mhr):
    refused(mhr, "gemm_routed_product", product_args(), [
        dict(dtype=0), dict(dtype=3), dict(out_dtype=3), dict(x=None), dict(w=None), dict(out=None),
        dict(offsets=None), dict(E=0), dict(E=1025), dict(top=0), dict(rows=-1), dict(K=-1),
        dict(N=-1), dict(x_rows=19), dict(out_rows=21), dict(ldx=63), dict(ldw=63), dict(ldo=63),
        dict(stride_w=4095), dict(out=P), dict(out=Q), dict(out=R), dict(x=P + 1), dict(out=S + 1),
        dict(offsets=R + 2), dict(gather=0x50000001), dict(scatter=0x50000002), dict(gather=S),
        dict(scatter=S), dict(rows=1 << 31, x_rows=1 << 31, out_rows=1 << 31),
        # a copy is needed (pitch, address, stride), and no scratch or too little is there
        dict(ldx=65), dict(x=P + 2), dict(stride_w=4100), dict(ldw=66, stride_w=66 * 64),
        dict(ldx=65, scratch=0x70000000, scratch_bytes=2559),
        dict(ldx=65, scratch=0x70000008, scratch_bytes=1 << 20),
        dict(ldx=65, scratch=S, scratch_bytes=1 << 20), dict(ldx=65, scratch=P, scratch_bytes=1 << 20)])
    f = mhr.load().gemm_routed_product
    for nothing in (dict(rows=0, x_rows=0, out_rows=0), dict(N=0, ldw=0, ldo=0),
                    dict(out_rows=0, scatter=0x50000000)):
        assert f(*dict(product_args(), **nothing).values()) == mhr.MHR_OK, nothing


def test_weight_grad_refusals(mhr):
    args = dict(dtype=1, x=P, x_rows=20, ldx=64, gather=None, top=1, grad=Q, grad_rows=20, ldg=64,
                scatter=None, offsets=R, E=3, out_dtype=0, out=S, ldo=64, stride_o=4096, rows=20,
                K=64, N=64, scratch=None, scratch_bytes=0, stream=None)
    refused(mhr, "gemm_routed_weight_grad", args, [
        dict(dtype=0), dict(out_dtype=-1), dict(x=None), dict(grad=None), dict(out=None),
        dict(offsets=None), dict(E=0), dict(top=-1), dict(x_rows=21), dict(grad_rows=21),
        dict(ldx=63), dict(ldg=63), dict(ldo=63), dict(stride_o=4095), dict(out=P), dict(out=Q),
        dict(out=R), dict(out=S + 2), dict(ldg=68), dict(grad=Q + 2), dict(ldx=68)])
    f = mhr.load().gemm_routed_weight_grad
    assert f(*dict(args, K=0, out=None).values()) == mhr.MHR_OK


def test_scratch(mhr):
    f = mhr.load().gemm_routed_product_scratch
    args = dict(x=P, x_rows=20, ldx=64, gathered=0, w=Q, ldw=64, stride_w=4096, transposed=0, E=3,
                rows=20, K=64, N=64)
    for change, bytes_ in [
            (dict(), 0), (dict(ldx=72), 0), (dict(ldx=65), 20 * 128), (dict(x=P + 2), 20 * 128),
            (dict(x_rows=1, ldx=65, gathered=1), 0),                 # one row has no pitch
            (dict(gathered=1), 0), (dict(gathered=1, rows=257), 258 * 128),
            (dict(gathered=1, rows=300, ldx=65), 300 * 128), (dict(w=Q + 2), 3 * 64 * 128),
            (dict(ldw=66, stride_w=66 * 64), 3 * 64 * 128), (dict(stride_w=4100), 3 * 64 * 128),
            (dict(E=1, stride_w=1), 0), (dict(N=60, ldw=65), 3 * 64 * 128),
            (dict(transposed=1, N=60, ldw=65), 3 * 60 * 128), (dict(ldx=65, w=Q + 2), 212 * 128),
            (dict(rows=0, ldx=65), 0), (dict(K=0, ldx=65), 0), (dict(E=0), -1), (dict(rows=-1), -1),
            (dict(gathered=1, rows=(1 << 31) - 512, K=(1 << 31) - 512, N=(1 << 31) - 512, E=1024,
                  w=Q + 2), -1)]:
        assert f(*dict(args, **change).values()) == bytes_, change
    f = mhr.load().gemm_routed_weight_grad_scratch
    args = dict(x=P, x_rows=20, ldx=64, gathered=0, grad=Q, grad_rows=20, ldg=64, scattered=0,
                rows=20, K=64, N=64)
    for change, bytes_ in [(dict(), 0), (dict(gathered=1), 20 * 128),
                           (dict(gathered=1, scattered=1, rows=50), 100 * 128),
                           (dict(ldg=65), 20 * 128), (dict(rows=0, gathered=1), 0),
                           (dict(K=-1), -1)]:
        assert f(*dict(args, **change).values()) == bytes_, change


def test_adapters_refusals(mhr):
    args = dict(dtype=1, x=P, ldx=64, down=Q, ldd=64, stride_d=1024, up=R, ldu=64, stride_u=1024,
                which=0x50000000, scales=None, L=3, rank=16, out_dtype=1, y=S, ldy=64,
                out=0x70000000, ldo=64, T=20, K=64, N=64, scratch=None, scratch_bytes=0,
                stream=None)
    refused(mhr, "gemm_routed_adapters", args, [
        dict(dtype=0), dict(out_dtype=3), dict(x=None), dict(down=None), dict(up=None),
        dict(which=None), dict(y=None), dict(out=None), dict(L=0), dict(L=1025), dict(rank=0),
        dict(rank=129), dict(T=-1), dict(T=1 << 31), dict(K=-1), dict(N=-1), dict(ldx=63),
        dict(ldd=63), dict(ldu=63), dict(ldy=63), dict(ldo=63), dict(stride_d=1023),
        dict(stride_u=1000), dict(out=P), dict(out=Q), dict(out=R), dict(out=0x50000000),
        dict(out=S + 64), dict(out=S, ldo=72), dict(scales=0x70000000), dict(x=P + 1),
        dict(y=S + 1), dict(which=0x50000002), dict(scales=0x50001001)])
    f = mhr.load().gemm_routed_adapters
    for nothing in (dict(T=0), dict(N=0, ldu=0, ldy=0, ldo=0)):
        assert f(*dict(args, **nothing).values()) == mhr.MHR_OK
    sizes = [v for k, v in args.items()
             if k not in ("which", "scales", "y", "ldy", "out", "ldo", "scratch",
                          "scratch_bytes", "stream")]
    assert mhr.load().gemm_routed_adapters_scratch(*sizes) >= 0
    sizes[10] = 129  # the rank
    assert mhr.load().gemm_routed_adapters_scratch(*sizes) == -1


def test_tensor_calls_refuse(mhr):
    """What the tensor-level calls say before they look for a GPU."""
    import torch

    x = torch.zeros(4, 16)
    e = torch.zeros(4, 3, dtype=torch.int32)
    g = torch.zeros(4, 3)
    h, w = x.bfloat16(), torch.zeros(2, 16, 8, dtype=torch.bfloat16)
    o = torch.zeros(3, dtype=torch.int32)
    r = torch.zeros(2, 5, 16, dtype=torch.bfloat16)
    which = torch.zeros(4, dtype=torch.int32)
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
            (ValueError, "CUDA", lambda: mhr.sort_by_expert(e, 5)),
            (TypeError, "both be", lambda: mhr.matmul_experts(x, w, o)),
            (TypeError, "both be", lambda: mhr.matmul_experts(h.half(), w, o)),
            (ValueError, "3-D", lambda: mhr.matmul_experts(h, w[0], o)),
            (ValueError, "row-major", lambda: mhr.matmul_experts(h, w.transpose(1, 2), o)),
            (ValueError, "overlap", lambda: mhr.matmul_experts(h, w[:1].expand(2, 16, 8), o)),
            (TypeError, "offsets must be int32", lambda: mhr.matmul_experts(h, w, o.long())),
            (ValueError, "CUDA", lambda: mhr.matmul_experts(h, w, o)),
            (TypeError, "both be", lambda: mhr.matmul_experts_grad(h, x, o)),
            (ValueError, "CUDA", lambda: mhr.matmul_experts_grad(h, h, o)),
            (TypeError, "y must be", lambda: mhr.add_adapters(x.int(), h, r, r, which)),
            (TypeError, "both be", lambda: mhr.add_adapters(x, x, r, r, which)),
            (TypeError, "both be", lambda: mhr.add_adapters(x, h, r, r.half(), which)),
            (ValueError, "sizes differ", lambda: mhr.add_adapters(x, h, r, r[:, :4], which)),
            (ValueError, "sizes differ", lambda: mhr.add_adapters(x[:3], h, r, r, which)),
            (TypeError, "which must be int32", lambda: mhr.add_adapters(x, h, r, r, which.long())),
            (ValueError, "of T values", lambda: mhr.add_adapters(x, h, r, r, which[:2])),
            (ValueError, "CUDA", lambda: mhr.add_adapters(x, h, r, r, which))]:
        with pytest.raises(error, match=match):
            call()
