"""The 4-bit operators without a GPU: refusals at the C ABI and in the tensor-level calls."""
import numpy as np
import pytest

import mxfp4_ref as ref

P, Q, R, S, T = (0x10000000 * i for i in range(1, 6))  # fake, disjoint, aligned addresses
F32, BF16 = 0, 1


@pytest.fixture(scope="module")
def lib():
    from memory_hierarchy_reuse_gb300 import build as b

    b.build()
    import memory_hierarchy_reuse_gb300 as m

    return m.load()


def test_scale_bytes(lib):
    import memory_hierarchy_reuse_gb300 as m

    for rows, cols in [(1, 1), (128, 128), (129, 128), (128, 129), (1000, 4100), (0, 5)]:
        want = -(-rows // 128) * -(-cols // 128) * 512
        assert lib.gemm_mxfp4_scale_bytes(rows, cols) == want == m.mxfp4_scale_bytes(rows, cols)
    assert lib.gemm_mxfp4_scale_bytes(-1, 4) == -1
    assert lib.gemm_mxfp4_scale_bytes(4, 1 << 40) == -1


def test_quantize_refusals(lib):
    # dtype, X, rows, cols, ldx, transpose, data, ldd, scales, values, ldv
    good = [F32, P, 8, 64, 64, 0, Q, 32, R, S, 64]
    bad = [{0: 3}, {0: -1}, {1: None}, {1: P + 2}, {2: -1}, {3: -1}, {4: 63}, {6: None}, {6: Q + 8},
           {7: 24}, {7: 16}, {7: 40}, {8: None}, {8: R + 4}, {9: P}, {9: S + 2}, {10: 63}, {8: Q},
           {6: P}, {8: P + 16}, {2: 1 << 40}, {4: 1 << 62}, {5: 1, 7: 0}, {9: Q}, {9: R}]
    for change in bad:
        args = [change.get(i, v) for i, v in enumerate(good)]
        assert lib.gemm_mxfp4_quantize(*args, None) == 1, change
    for change in ({2: 0}, {3: 0}):
        args = [change.get(i, v) for i, v in enumerate(good)]
        assert lib.gemm_mxfp4_quantize(*args, None) == 0


def test_product_refusals(lib):
    # c_dtype, A, A_scales, Bt, Bt_scales, C, M, N, K, lda, ldb, ldc
    good = [BF16, P, Q, R, S, T, 8, 16, 64, 32, 32, 16]
    bad = [{0: 7}, {1: None}, {2: None}, {3: None}, {4: None}, {5: None}, {1: P + 8}, {2: Q + 8},
           {3: R + 1}, {4: S + 4}, {5: T + 1}, {6: -1}, {7: -1}, {8: -1}, {9: 16}, {9: 40}, {10: 16},
           {10: 33}, {11: 15}, {5: P}, {5: Q}, {5: R + 16}, {5: S}, {8: 1 << 33}, {11: 1 << 62},
           {9: 1 << 45}]
    for change in bad:
        args = [change.get(i, v) for i, v in enumerate(good)]
        assert lib.gemm_mxfp4(*args, None) == 1, change
    for change in ({6: 0}, {7: 0}):
        args = [change.get(i, v) for i, v in enumerate(good)]
        assert lib.gemm_mxfp4(*args, None) == 0
    # a_dtype, A, c_dtype, Bt, Bt_scales, C, M, N, K, lda, ldb, ldc
    good = [BF16, P, BF16, R, S, T, 8, 16, 64, 64, 32, 16]
    bad = [{0: 4}, {2: 4}, {1: None}, {1: P + 1}, {9: 63}, {3: None}, {4: None}, {5: None}, {5: P},
           {5: R}, {5: S}, {10: 16}, {11: 15}, {6: -1}, {8: -2}]
    for change in bad:
        args = [change.get(i, v) for i, v in enumerate(good)]
        assert lib.gemm_mxfp4_quantized(*args, None) == 1, change


def test_moe_refusals(lib):
    # x, ldx, router, ldr, up, up_s, ldu, down, down_s, ldd, y, ldy, experts, weights, T, E, top, H, I
    a = [0x10000000 * i for i in range(1, 10)]
    good = [a[0], 64, a[1], 64, a[2], a[3], 32, a[4], a[5], 16, a[6], 64, a[7], a[8], 2, 4, 2, 64, 32]
    bad = [{0: None}, {0: a[0] + 1}, {1: 63}, {2: None}, {3: 63}, {4: None}, {4: a[2] + 8}, {5: None},
           {6: 16}, {6: 40}, {7: None}, {8: a[5] + 4}, {9: 8}, {10: None}, {11: 63}, {12: None},
           {12: a[7] + 2}, {13: None}, {14: -1}, {14: 65}, {15: 0}, {15: 513}, {16: 0}, {16: 5},
           {15: 32, 16: 17}, {17: 0}, {17: 16385}, {18: 0}, {18: 16385}, {10: a[0]}, {10: a[2]},
           {12: a[8]}, {13: a[6]}, {12: a[4]}]
    for change in bad:
        args = [change.get(i, v) for i, v in enumerate(good)]
        assert lib.gemm_mxfp4_moe(*args, None) == 1, change
    assert lib.gemm_mxfp4_moe(*[{14: 0}.get(i, v) for i, v in enumerate(good)], None) == 0


def test_moe_tensor_level_refusals():
    import torch

    import memory_hierarchy_reuse_gb300 as m

    byte = lambda *n: torch.zeros(n, dtype=torch.uint8)  # noqa: E731
    x, router = torch.zeros(2, 64).bfloat16(), torch.zeros(4, 64).bfloat16()
    up, down = m.MxFp4Matrix(byte(256, 32), byte(1024), 256, 64), m.MxFp4Matrix(byte(256, 16), byte(1024), 256, 32)
    for args, kw in [((x.float(), router, up, down, 2), {}), ((x, router.float(), up, down, 2), {}),
                     ((x[:, :32], router, up, down, 2), {}), ((x, router[:3], up, down, 2), {}),
                     ((x, router, up._replace(cols=32), down, 2), {}),
                     ((x, router, up, down._replace(cols=16), 2), {}),
                     ((x, router, up, down, 2), {"out": torch.zeros(2, 64)}),
                     ((x, router, up, down, 2), {})]:
        with pytest.raises((TypeError, ValueError)):
            m.moe_mxfp4(*args, **kw)


def test_tensor_level_refusals():
    import torch

    import memory_hierarchy_reuse_gb300 as m

    with pytest.raises(TypeError):
        m.quantize_mxfp4(torch.zeros(4, 4, dtype=torch.int32))
    with pytest.raises(ValueError):
        m.quantize_mxfp4(torch.zeros(4, 4, 4))
    with pytest.raises(ValueError):
        m.quantize_mxfp4(torch.zeros(4, 64).t())
    with pytest.raises(ValueError):
        m.quantize_mxfp4(torch.zeros(4, 4), axis=2)
    with pytest.raises(ValueError):
        m.quantize_mxfp4(torch.zeros(4, 4))  # not on a GPU
    byte = lambda *n: torch.zeros(n, dtype=torch.uint8)  # noqa: E731
    a, b = m.MxFp4Matrix(byte(4, 32), byte(512), 4, 64), m.MxFp4Matrix(byte(6, 32), byte(512), 6, 64)
    for bad_a, bad_b, kw in [(a, b._replace(cols=32), {}), (a._replace(rows=5), b, {}),
                             (a._replace(scales=byte(511)), b, {}), (a, b._replace(data=byte(6, 31)), {}),
                             (a, b, {"out": torch.zeros(6, 4)}), (a, b, {"out_dtype": torch.int32}),
                             (a._replace(data=torch.zeros(4, 32)), b, {}),
                             (torch.zeros(4, 64, dtype=torch.float64), b, {}), (a, b, {})]:
        with pytest.raises((TypeError, ValueError)):
            m.matmul_mxfp4(bad_a, bad_b, **kw)


def test_rows_that_overlap_are_refused():
    import torch

    import memory_hierarchy_reuse_gb300 as m

    with pytest.raises(ValueError):
        m.quantize_mxfp4(torch.zeros(1, 64).expand(4, 64))
    with pytest.raises(ValueError):
        m.quantize_mxfp4(torch.zeros(200).as_strided((4, 64), (32, 1)))


def test_reference_format_round_trip():
    """The numpy statement that the GPU tests compare with: packing, the tile order against a
    second way of writing it, and rounding at the ties."""
    codes, scales = ref.quantize(np.random.default_rng(0).standard_normal((150, 300)))
    data, tiled = ref.pack(codes, scales)
    c2, s2 = ref.unpack(data, tiled, 300)
    assert np.array_equal(c2, codes) and np.array_equal(s2, scales)
    padded = np.zeros((256, 12), np.uint8)
    padded[:150, :10] = scales
    again = padded.reshape(2, 4, 32, 3, 4).transpose(0, 3, 2, 1, 4).reshape(-1)
    assert np.array_equal(again, tiled)
    ties = np.array([[4.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -0.25, 6.5, 7.9] + [0] * 21])
    codes, scales = ref.quantize(ties)
    want = [4, 0, 1, 1, 2, 2, 4, 4, 0, 6, 6]
    assert scales[0, 0] == 127 and list(ref.values(codes, scales, 11)[0]) == want
