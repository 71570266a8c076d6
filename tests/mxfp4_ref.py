"""Plain numpy statement of the 4-bit format and operators, in 64 bits."""
import numpy as np

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def cdiv(a, b):
    return -(-a // b)


def quantize(x):
    """(codes rows x 32 * blocks, scale codes rows x blocks) of a float64 matrix, element by
    element from the definition: nearest of the eight magnitudes, ties to the even code."""
    rows, cols = x.shape
    blocks = cdiv(cols, 32)
    x = np.pad(np.asarray(x, np.float64), ((0, 0), (0, blocks * 32 - cols)))
    x = x.reshape(rows, blocks, 32)
    bad = ~np.isfinite(x).all(-1)
    x = np.where(bad[..., None], 0.0, x)
    amax = np.abs(x).max(-1)
    _, e = np.frexp(amax)  # amax = f 2^e, f in [0.5, 1): floor(log2 amax) = e - 1
    scale = np.where(amax > 0, np.clip(e - 3 + 127, 0, 254), 0)
    y = np.abs(np.ldexp(x, 127 - scale[..., None]))
    d = np.abs(y[..., None] - E2M1)
    best = d.min(-1, keepdims=True)
    # among equally near codes the even one (neighbours differ in parity)
    code = np.where(d == best, np.arange(8) + 100 * (np.arange(8) % 2), 1000).argmin(-1)
    code = code + 8 * (np.signbit(x) & (code > 0))
    return code.reshape(rows, blocks * 32).astype(np.uint8), np.where(bad, 255, scale).astype(np.uint8)


def values(codes, scales, cols):
    v = np.where(codes & 8, -1.0, 1.0) * E2M1[codes & 7]
    s = np.where(scales == 255, np.nan, np.ldexp(1.0, scales.astype(int) - 127))
    return (v.reshape(*scales.shape, 32) * s[..., None]).reshape(codes.shape)[:, :cols]


def pack(codes, scales):
    """(data, tiled scales) as mhr_mxfp4.h lays them out, padding zero."""
    rows, blocks = scales.shape
    data = (codes[:, 0::2] | (codes[:, 1::2] << 4)).astype(np.uint8)
    kt = cdiv(blocks, 4)
    tiled = np.zeros(cdiv(rows, 128) * kt * 512, np.uint8)
    r, b = np.arange(rows)[:, None], np.arange(blocks)[None]
    tiled[((r // 128) * kt + b // 4) * 512 + r % 32 * 16 + r % 128 // 32 * 4 + b % 4] = scales
    return data, tiled


def unpack(data, tiled, cols):
    """(codes, scale codes) of the first `cols` columns."""
    rows, blocks = data.shape[0], cdiv(cols, 32)
    data = data[:, :blocks * 16]
    codes = np.stack([data & 15, data >> 4], -1).reshape(rows, blocks * 32)
    kt = cdiv(blocks, 4)
    r, b = np.arange(rows)[:, None], np.arange(blocks)[None]
    return codes, tiled[((r // 128) * kt + b // 4) * 512 + r % 32 * 16 + r % 128 // 32 * 4 + b % 4]


def random_packed(rows, cols, seed, lo=118, hi=128):
    """A packed matrix of uniform codes with scales 2^(lo-127) .. 2^(hi-128), and its values."""
    rng = np.random.default_rng(seed)
    blocks = cdiv(cols, 32)
    codes = rng.integers(0, 16, (rows, blocks * 32), dtype=np.uint8)
    codes[:, cols:] = 0
    scales = rng.integers(lo, hi, (rows, blocks)).astype(np.uint8)
    return *pack(codes, scales), values(codes, scales, cols)


# Error bounds of a product with fp32 sums: every product of two values is exact; the MMAs add
# 64 columns at a time to an fp32 accumulator, each addition off by at most one unit in the last
# place of a partial sum (2^-23 of the sum of magnitudes), the split K parts add 8 more roundings,
# and a factor 2 covers the order within an MMA. Then C is rounded once to its type.
def product_bound(K, S, ref, dtype):
    bound = 2 * (cdiv(K, 64) + 8) * 2.0 ** -23 * S
    if dtype == "bf16":
        bound = bound + (np.abs(ref) + bound) * 2.0 ** -8
    elif dtype == "f16":
        bound = bound + (np.abs(ref) + bound) * 2.0 ** -11 + 2.0 ** -24
    return bound
