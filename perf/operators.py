"""Cases for the 4-bit operators: quantisation, product, and the mixture-of-experts layer.

Microscaled 4-bit floats (MXFP4): a value is an e2m1 code (0, 0.5, 1, 1.5, 2, 3, 4, 6 and a sign)
times a power of two shared by 32 consecutive values, so a value costs 4.25 bits. A matrix of
``rows`` x ``cols`` is two byte arrays:

* ``data``: ``rows`` x 16 * ceil(cols / 32) bytes, two codes a byte, the even column in the low half;
* ``scales``: one e8m0 byte (2^(code - 127)) per row and block of 32 columns, in tiles of 128 rows x
  4 blocks of 512 bytes: byte ``(row % 32) * 16 + (row % 128) // 32 * 4 + block % 4`` of tile
  ``(row // 128) * ceil(blocks / 4) + block // 4``.

Three operators, each with its plain form in elementary torch operations:

* ``quantize``: a matrix into that form, blocks along its rows or down its columns; the values that
  the codes stand for are returned, as training with rounded weights or activations uses them;
* ``product``: ``C = A B`` for 4-bit A and B with bf16 C; A as bf16 activations that are quantised
  on the way (``prequantized`` false), or in 4 bits already;
* ``moe``: a whole mixture-of-experts layer for a few tokens: softmax routing, the top experts'
  gated products over 4-bit weights, and their weighted sum.
"""
import numpy as np
import torch

own = False

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


# ------------------------------------------------------------------------------------- the cases
def listed():
    return [
        # one token's activations before a 4-bit product: nothing but latency
        dict(name="quantize 1x4096 bf16", op="quantize", rows=1, cols=4096, axis=1, dtype="bf16"),
        # activations of a prompt, a ragged number of rows
        dict(name="quantize 2000x8192 bf16", op="quantize", rows=2000, cols=8192, axis=1,
             dtype="bf16"),
        # a master weight in fp32, stored K x N as the library's products take it, blocks along K
        dict(name="quantize cols 8192x11008 f32", op="quantize", rows=8192, cols=11008, axis=0,
             dtype="f32"),
        # a single token through a square layer
        dict(name="product 1x4096x4096", op="product", M=1, N=4096, K=4096, prequantized=False),
        # a small decoding batch through a wide layer
        dict(name="product 24x11008x4096", op="product", M=24, N=11008, K=4096,
             prequantized=False),
        # a short prompt with every size ragged
        dict(name="product 333x5000x4104", op="product", M=333, N=5000, K=4104,
             prequantized=False),
        # a prompt through a square layer, activations quantised by the layer before
        dict(name="product 4096x4096x4096", op="product", M=4096, N=4096, K=4096,
             prequantized=True),
        # the largest: a training-sized batch, activations quantised on the way
        dict(name="product 8192x8192x8192", op="product", M=8192, N=8192, K=8192,
             prequantized=False),
        # one token, few small experts
        dict(name="moe 1 token 32 experts", op="moe", T=1, E=32, top=4, H=1024, I=512),
        # a small decoding batch over many narrow experts
        dict(name="moe 8 tokens 128 experts", op="moe", T=8, E=128, top=8, H=2048, I=768),
        # sizes that end inside every tile
        dict(name="moe 13 tokens 60 experts", op="moe", T=13, E=60, top=6, H=2600, I=1416),
        # the most tokens that the layer takes in one call, nearly every expert's weights read
        dict(name="moe 64 tokens 128 experts", op="moe", T=64, E=128, top=8, H=4096, I=1536),
    ]


def draw(rng):
    def log(lo, hi, multiple=1):
        return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random() / multiple)) * multiple))

    op = rng.choice(["quantize", "product", "moe"])
    if op == "quantize":
        return dict(op=op, rows=log(1, 8192), cols=log(32, 11008, rng.choice([1, 8, 32])),
                    axis=rng.choice([0, 1]), dtype=rng.choice(["bf16", "f16", "f32"]))
    if op == "product":
        return dict(op=op, M=log(1, 8192), N=log(64, 8192, rng.choice([1, 8, 64])),
                    K=log(64, 8192, rng.choice([1, 8, 64])),
                    prequantized=rng.choice([True, False]))
    E = log(4, 128)
    return dict(op=op, T=log(1, 64), E=E, top=min(E, rng.randint(1, 8)),
                H=log(256, 4096, rng.choice([1, 8, 64])), I=log(64, 1536, rng.choice([1, 8, 64])))


def packed_bytes(rows, cols):
    """Codes and scales of a 4-bit matrix."""
    blocks = -(-cols // 32)
    return rows * blocks * 17


def work(case):
    if case["op"] == "quantize":
        n, size = case["rows"] * case["cols"], DTYPES[case["dtype"]].itemsize
        packed = packed_bytes(case["rows"], case["cols"]) if case["axis"] == 1 else \
            packed_bytes(case["cols"], case["rows"])
        return {"bytes": 2 * size * n + packed, "flops": 4 * n}
    if case["op"] == "product":
        M, N, K = case["M"], case["N"], case["K"]
        a = packed_bytes(M, K) if case["prequantized"] else 2 * M * K
        return {"bytes": a + packed_bytes(N, K) + 2 * M * N, "flops": 2 * M * N * K}
    T, E, top, H, I = (case[k] for k in ("T", "E", "top", "H", "I"))
    touched = E * (1 - (1 - top / E) ** T)  # expected number of experts that some token takes
    weights = touched * (packed_bytes(2 * I, H) + packed_bytes(H, I))
    return {"bytes": weights + 2 * E * H + 4 * T * H + 8 * T * top,
            "flops": 2 * T * E * H + 6 * T * top * H * I}


# --------------------------------------------------------------- the format, in plain operations
def plain_codes(x):
    """(e2m1 codes, e8m0 codes) of a rows x cols fp32 matrix, blocks of 32 along the rows."""
    rows, cols = x.shape
    blocks = -(-cols // 32)
    x = torch.nn.functional.pad(x, (0, blocks * 32 - cols)).reshape(rows, blocks, 32)
    amax = x.abs().amax(-1)
    # the block's power of two: floor(log2(amax)) - 2 (6 = 1.5 * 2^2 is the largest code)
    exponent = torch.frexp(amax).exponent - 3
    code = torch.where(amax > 0, (exponent + 127).clamp(0, 254), 0)
    y = torch.ldexp(x, (127 - code).unsqueeze(-1))
    a = y.abs()
    # round to nearest, ties to the even code; above 5 saturates to 6
    e2m1 = ((a > 0.25).byte() + (a >= 0.75).byte() + (a > 1.25).byte() + (a >= 1.75).byte()
            + (a > 2.5).byte() + (a >= 3.5).byte() + (a > 5).byte())
    e2m1 = e2m1 + 8 * (torch.signbit(y) & (e2m1 > 0)).byte()
    return e2m1.reshape(rows, blocks * 32), code.byte()


def plain_values(e2m1, code):
    """fp32 values of e2m1 codes and their blocks' e8m0 codes."""
    lut = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=e2m1.device)
    v = lut[e2m1.int()].reshape(*code.shape, 32)
    return torch.ldexp(v, (code.int() - 127).unsqueeze(-1)).reshape(e2m1.shape)


def pack(e2m1, code):
    """(data, scales) in the layout above."""
    rows, blocks = code.shape
    data = e2m1[:, 0::2] | (e2m1[:, 1::2] << 4)
    tiles = torch.nn.functional.pad(code, (0, -blocks % 4, 0, -rows % 128))
    tiles = tiles.reshape(tiles.shape[0] // 128, 4, 32, tiles.shape[1] // 4, 4)
    return data.contiguous(), tiles.permute(0, 3, 2, 1, 4).contiguous().reshape(-1)


def unpack(data, scales):
    """(e2m1 codes, e8m0 codes) of a packed matrix."""
    rows, blocks = data.shape[0], data.shape[1] // 16
    e2m1 = torch.stack((data & 15, data >> 4), -1).reshape(rows, blocks * 32)
    tiles = scales.reshape(-(-rows // 128), -(-blocks // 4), 32, 4, 4).permute(0, 3, 2, 1, 4)
    return e2m1, tiles.reshape(-(-rows // 128) * 128, -(-blocks // 4) * 4)[:rows, :blocks]


# ------------------------------------------------------------------------------------ the inputs
def normal(shape, gen, std=1.0):
    return torch.randn(shape, generator=gen, device="cuda") * std


def activations(rows, cols, gen):
    """Normal values with the few large channels that hidden states have."""
    x = normal((rows, cols), gen)
    loud = torch.rand((cols,), generator=gen, device="cuda") < 0.01
    return torch.where(loud, x * 12, x)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    if case["op"] == "quantize":
        if case["axis"] == 1:
            x = activations(case["rows"], case["cols"], gen)
        else:
            x = normal((case["rows"], case["cols"]), gen, case["rows"] ** -0.5)
        return dict(case, x=x.to(DTYPES[case["dtype"]]))
    if case["op"] == "product":
        M, N, K = case["M"], case["N"], case["K"]
        a = activations(M, K, gen).bfloat16()
        a = pack(*plain_codes(a.float())) if case["prequantized"] else a
        return dict(case, a=a, b=pack(*plain_codes(normal((N, K), gen, K ** -0.5))))
    T, E, H, I = (case[k] for k in ("T", "E", "H", "I"))
    up = [plain_codes(normal((2 * I, H), gen, H ** -0.5)) for _ in range(E)]
    up = pack(torch.cat([c for c, _ in up]), torch.cat([s for _, s in up]))
    down = [plain_codes(normal((H, I), gen, I ** -0.5)) for _ in range(E)]
    down = pack(torch.cat([c for c, _ in down]), torch.cat([s for _, s in down]))
    return dict(case, x=activations(T, H, gen).bfloat16(),
                router=normal((E, H), gen, H ** -0.5).bfloat16(), up=up, down=down)


# --------------------------------------------------------------------------------------- a pass
def run_quantize(s):
    if own:
        import memory_hierarchy_reuse_gb300 as mhr
        return mhr.quantize_mxfp4(s["x"], axis=s["axis"], values=True)[1]
    x = s["x"].float() if s["axis"] == 1 else s["x"].float().t().contiguous()
    v = plain_values(*plain_codes(x))[:, : x.shape[1]]
    return (v if s["axis"] == 1 else v.t()).to(s["x"].dtype).contiguous()


def run_product(s):
    if own:
        import memory_hierarchy_reuse_gb300 as mhr
        a = mhr.MxFp4Matrix(*s["a"], s["M"], s["K"]) if s["prequantized"] else s["a"]
        b = mhr.MxFp4Matrix(*s["b"], s["N"], s["K"])
        return mhr.matmul_mxfp4(a, b, out_dtype=torch.bfloat16)
    a = plain_values(*(unpack(*s["a"]) if s["prequantized"] else plain_codes(s["a"].float())))
    b = plain_values(*unpack(*s["b"]))
    return (a @ b.t()).bfloat16()


def run_moe(s):
    T, E, top, H, I = (s[k] for k in ("T", "E", "top", "H", "I"))
    if own:
        import memory_hierarchy_reuse_gb300 as mhr
        up = mhr.MxFp4Matrix(*s["up"], 2 * E * I, H)
        down = mhr.MxFp4Matrix(*s["down"], E * H, I)
        y, experts, weights = mhr.moe_mxfp4(s["x"], s["router"], up, down, top)
        return {"y": y, "experts": experts, "weights": weights}
    x = s["x"].float()
    probs = torch.softmax(x @ s["router"].float().t(), -1)
    probs, experts = torch.sort(probs, descending=True, stable=True)
    probs, experts = probs[:, :top], experts[:, :top]
    weights = probs / probs.sum(-1, keepdim=True)
    codes, scales = unpack(*s["up"])
    up_c, up_s = codes.reshape(E, 2 * I, -1), scales.reshape(E, 2 * I, -1)
    codes, scales = unpack(*s["down"])
    down_c, down_s = codes.reshape(E, H, -1), scales.reshape(E, H, -1)
    if T * top < E:  # few experts: each (token, expert) pair's own weights
        flat = experts.reshape(-1)
        w = plain_values(up_c[flat], up_s[flat])[..., :H]
        h = w @ x.repeat_interleave(top, 0).unsqueeze(-1)
        gate, value = h[:, :I], h[:, I:]
        h = gate / (1 + torch.exp(-gate)) * value
        y = (plain_values(down_c[flat], down_s[flat])[..., :I] @ h).reshape(T, top, H)
        y = (y * weights.unsqueeze(-1)).sum(1)
    else:  # every expert's weights once, for all tokens, and the chosen ones' part of the sum
        h = x @ plain_values(up_c, up_s)[..., :H].transpose(1, 2)
        gate, value = h[..., :I], h[..., I:]
        h = gate / (1 + torch.exp(-gate)) * value
        y = h @ plain_values(down_c, down_s)[..., :I].transpose(1, 2)
        share = torch.zeros((T, E), device=x.device).scatter(1, experts, weights)
        y = (y * share.t().unsqueeze(-1)).sum(0)
    return {"y": y.bfloat16(), "experts": experts.int(), "weights": weights}


def run(state):
    return {"quantize": run_quantize, "product": run_product, "moe": run_moe}[state["op"]](state)


# ----------------------------------------------------------------------------------- in 64 bits
def exact_rounded(x):
    """The values that a float64 matrix is rounded to, blocks of 32 along the rows: the nearest
    e2m1 multiple of the block's power of two, by the spacing of the binade it falls in."""
    rows, cols = x.shape
    pad = -cols % 32
    x = torch.cat([x, x.new_zeros((rows, pad))], 1).reshape(rows, -1, 32)
    amax = x.abs().amax(-1, keepdim=True)
    top = torch.floor(torch.log2(torch.where(amax > 0, amax, 1.0)))
    top = torch.where(torch.exp2(top) > amax, top - 1, top)
    top = torch.where(torch.exp2(top + 1) <= amax, top + 1, top)
    unit = torch.exp2((top - 2).clamp(min=-127.0))
    y = x / unit
    # e2m1 is spaced 0.5 below 2, 1 from 2 to 4 and 2 from 4 to 6
    step = torch.where(y.abs() < 2, 0.5, torch.where(y.abs() < 4, 1.0, 2.0))
    y = (torch.round(y / step) * step).clamp(-6, 6) * unit
    return y.reshape(rows, -1)[:, :cols]


def exact_unpacked(data, scales, cols):
    """float64 values of a packed matrix, by each byte's place."""
    rows, blocks = data.shape[0], data.shape[1] // 16
    table = torch.tensor(E2M1, dtype=torch.float64, device=data.device)
    table = torch.cat([table, -table])
    k = torch.arange(cols, device=data.device)
    r = torch.arange(rows, device=data.device).unsqueeze(1)
    nibble = (data[:, k // 2].int() >> (k % 2 * 4).int()) & 15
    b = torch.arange(blocks, device=data.device)
    at = (r // 128 * (-(-blocks // 4)) + b // 4) * 512 + r % 32 * 16 + r % 128 // 32 * 4 + b % 4
    unit = torch.exp2(scales[at].double() - 127)
    return table[nibble] * unit.repeat_interleave(32, 1)[:, :cols]


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "quantize":
        x = s["x"].double()
        return exact_rounded(x) if case["axis"] == 1 else exact_rounded(x.t()).t().contiguous()
    if case["op"] == "product":
        a = exact_unpacked(*s["a"], case["K"]) if case["prequantized"] else \
            exact_rounded(s["a"].double())
        return a @ exact_unpacked(*s["b"], case["K"]).t()
    T, E, top, H, I = (case[k] for k in ("T", "E", "top", "H", "I"))
    x = s["x"].double()
    logits = (x @ s["router"].double().t()).cpu().numpy()
    experts = np.argsort(-logits, axis=1, kind="stable")[:, :top]
    chosen = np.take_along_axis(logits, experts, 1)
    weights = np.exp(chosen - chosen[:, :1])
    weights /= weights.sum(1, keepdims=True)
    # unpacked expert by expert: codes by rows of the whole array, scales by their place in it
    y = torch.zeros((T, H), dtype=torch.float64, device="cuda")
    for e in np.unique(experts):
        t, k = np.nonzero(experts == e)
        gate_up = exact_part(*s["up"], e * 2 * I, 2 * I, H)
        h = x[t] @ gate_up.t()
        h = h[:, :I] * torch.sigmoid(h[:, :I]) * h[:, I:]
        part = h @ exact_part(*s["down"], e * H, H, I).t()
        y[t] += part * torch.from_numpy(weights[t, k]).cuda().unsqueeze(1)
    return {"y": y, "experts": torch.from_numpy(experts.astype(np.int32)),
            "weights": torch.from_numpy(weights)}


def exact_part(data, scales, row, rows, cols):
    """float64 values of ``rows`` rows from ``row`` on: whole tiles of 128 rows around them."""
    first, last = row // 128 * 128, min(data.shape[0], -(-(row + rows) // 128) * 128)
    tile_bytes = -(-(data.shape[1] // 16) // 4) * 512
    part = scales[first // 128 * tile_bytes:-(-last // 128) * tile_bytes]
    return exact_unpacked(data[first:last], part, cols)[row - first:row - first + rows]
