"""Cases and plain forms of the 4-bit microscaled matrices and of dropout.

`listed()` and `draw()` give cases, `prepare()` a user's inputs on the GPU,
`run()` one pass (the plain form in elementary torch operations, or the calls
of the package where `own` is true), `exact()` the same outputs in float64
from the definition, and `work()` the bytes and operations of a pass.

A microscaled matrix holds signed 4-bit floating-point elements (one bit of
mantissa, two of exponent: 0, 0.5, 1, 1.5, 2, 3, 4, 6) in blocks of 32 along
its rows, each block with a power of two as its scale (8 bits, biased by 127;
255 stands for NaN).  Element 2j of a row is the low half of byte j.

Activations are feature-major (features x tokens), as in the layers of the
package.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "f16": 2, "bf16": 2}
BLOCK = 32


# ----------------------------------------------------------------- cases --

def _quantize(name, dtype, rows, cols, tokens_first=False):
    return {"name": name, "op": "quantize", "dtype": dtype, "rows": rows, "cols": cols,
            "tokens_first": tokens_first}


def _layer(name, op, dtype, tokens, n_in, n_out):
    return {"name": name, "op": op, "dtype": dtype, "tokens": tokens, "in": n_in, "out": n_out}


def _dropout(name, dtype, rows, cols, p):
    return {"name": name, "op": "dropout", "dtype": dtype, "rows": rows, "cols": cols, "p": p}


def listed():
    return [
        # a wide layer's weights taken into four bits and read back
        _quantize("quantize-weights", "bf16", 11008, 4096),
        # activations of a prompt of odd length, blocks along the features
        _quantize("quantize-tokens-f16", "f16", 2047, 4096, True),
        # serving: one token through a frozen 4096 x 4096 layer
        _layer("matmul-1", "matmul", "bf16", 1, 4096, 4096),
        # serving: a decode batch of 32 requests, wide output
        _layer("matmul-32-f16", "matmul", "f16", 32, 4096, 11008),
        # a mixed batch of odd length on a layer of odd sizes
        _layer("matmul-ragged-f16", "matmul", "f16", 2011, 4090, 4097),
        # long prompts, the largest product
        _layer("matmul-prompt", "matmul", "bf16", 8192, 4096, 11008),
        # training through a frozen layer: the gradient of its input
        _layer("gradient-train", "gradient", "bf16", 4096, 4096, 4096),
        # the same at full precision on a small layer
        _layer("gradient-f32", "gradient", "f32", 512, 2048, 2048),
        # a small batch with activations in four bits too
        _layer("matmul4-batch", "matmul4", "f16", 300, 4096, 4096),
        # long prompts with activations in four bits
        _layer("matmul4-prompt", "matmul4", "bf16", 8192, 4096, 11008),
        # dropout beside a few tokens' adapters, odd rows, both directions
        _dropout("dropout-ragged-f32", "f32", 4096, 257, 0.1),
        # dropout of a training batch's activations, both directions
        _dropout("dropout-train", "bf16", 11008, 8192, 0.05),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quantize", "matmul", "matmul", "gradient", "matmul4", "dropout"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    if op == "quantize":
        return {"op": op, "dtype": dtype, "rows": _log_int(rng, 1, 11008),
                "cols": _log_int(rng, 64, 4096), "tokens_first": rng.random() < 0.5}
    if op == "dropout":
        return {"op": op, "dtype": dtype, "rows": _log_int(rng, 1, 11008),
                "cols": _log_int(rng, 1, 8192), "p": rng.choice([0.0, 0.05, 0.1, 0.5, 0.9])}
    tokens = _log_int(rng, 1, 8192)
    if dtype == "f32":
        tokens = min(tokens, 2048)
    return {"op": op, "dtype": dtype, "tokens": tokens,
            "in": _log_int(rng, 128, 4096) if rng.random() < 0.5 else 64 * _log_int(rng, 2, 64),
            "out": _log_int(rng, 128, 11008) if rng.random() < 0.5 else 64 * _log_int(rng, 2, 172)}


# ---------------------------------------------------------------- inputs --

def _package():
    import unstructured_sparse_linear_amd as S
    return S


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dt = DTYPES[case["dtype"]]

    def normal(shape, std):
        return (torch.randn(shape, generator=g, device="cuda") * std).to(dt)

    if case["op"] == "quantize":
        rows, cols = case["rows"], case["cols"]
        if case["tokens_first"]:
            # activations [features, tokens]: a few features are much larger than the others
            big = torch.rand(cols, 1, generator=g, device="cuda") < 0.01
            x = normal((cols, rows), 1.0) * torch.where(big, 20.0, 1.0).to(dt)
            return {"case": case, "w": x.t()}
        return {"case": case, "w": normal((rows, cols), cols ** -0.5)}
    if case["op"] == "dropout":
        shape = (case["rows"], case["cols"])
        # the seed and the step of a training run, kept on the device
        state = torch.randint(0, 1 << 40, (2,), generator=g, device="cuda", dtype=torch.int64)
        return {"case": case, "x": normal(shape, 1.0), "dy": normal(shape, shape[1] ** -0.5),
                "state": state}
    n_in, n_out, T = case["in"], case["out"], case["tokens"]
    # the frozen weights, quantised when they were loaded
    codes, scales = _encode(torch.randn((n_out, n_in), generator=g, device="cuda") * n_in ** -0.5)
    s = {"case": case, "codes": codes, "scales": scales,
         "x": normal((n_out, T), T ** -0.5) if case["op"] == "gradient" else normal((n_in, T), 1.0)}
    if own:
        s["W"] = _package().Mx4Matrix(codes, scales, n_in)
    return s


# ------------------------------------------------------ plain operations --

def _blocks(w):
    """[rows, blocks, 32] in f32, zeros past the last column."""
    rows, cols = w.shape
    pad = -cols % BLOCK
    w = w.float()
    if pad:
        w = torch.cat([w, w.new_zeros(rows, pad)], 1)
    return w.reshape(rows, -1, BLOCK)


def _indices(w):
    """Element indices 0..15 and biased scales of each block."""
    b = _blocks(w)
    top = b.abs().amax(2)
    finite = torch.isfinite(top)
    # 2^(e - 1) <= top < 2^e; the largest element, 6, has exponent 2
    e = torch.frexp(torch.where(finite, top, 1.0)).exponent
    code = torch.clamp(e - 3 + 127, 0, 254)
    code = torch.where(top == 0, 127, code)
    a = b.abs() * torch.ldexp(torch.ones_like(top), 127 - code)[:, :, None]
    # halves go to the element with an even mantissa
    i = ((a > 0.25).int() + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5)
         + (a > 5.0))
    i = i + 8 * torch.signbit(b)
    code = torch.where(finite, code, 255)
    return torch.where(finite[:, :, None], i, 0), code


def _encode(w):
    i, code = _indices(w)
    i = i.reshape(i.shape[0], -1, 2)
    return (i[:, :, 0] + 16 * i[:, :, 1]).to(torch.uint8), code.to(torch.uint8)


_ELEMENTS = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def _values(i, code, cols):
    """f32 values of element indices [rows, blocks, 32]."""
    m = (i & 7).float()
    v = torch.where(m < 4, m * 0.5, torch.where(m < 6, m - 2.0, 2.0 * m - 8.0))
    v = torch.where(i >= 8, -v, v)
    scale = torch.ldexp(torch.ones_like(code, dtype=torch.float32), code.int() - 127)
    scale = torch.where(code == 255, math.nan, scale)
    return (v * scale[:, :, None]).reshape(i.shape[0], -1)[:, :cols]


def _decode(codes, scales, cols):
    i = torch.stack([codes & 15, codes >> 4], 2).reshape(codes.shape[0], -1, BLOCK).int()
    return _values(i, scales.int(), cols)


_M0, _M1, _W0, _W1 = 0xD2511F53, 0xCD9E8D57, 0x9E3779B9, 0xBB67AE85
_LOW = 0xFFFFFFFF


def _random16(rows, cols, state):
    """Philox 4x32 of seven rounds (Salmon, Moraes, Dror and Shaw, 2011): 16 random
    bits for each element, eight to a counter (column / 8, row, step)."""
    seed, step = state[0], state[1]
    c = torch.arange((cols + 7) // 8, device="cuda")[None, :]
    r = torch.arange(rows, device="cuda")[:, None]
    c0, c1 = torch.broadcast_tensors(c, r)
    c2, c3 = step & _LOW, (step >> 32) & _LOW
    k0, k1 = seed & _LOW, (seed >> 32) & _LOW
    for _ in range(7):
        p0, p1 = c0 * _M0, c2 * _M1
        c0, c1, c2, c3 = (((p1 >> 32) & _LOW) ^ c1 ^ k0, p1 & _LOW,
                          ((p0 >> 32) & _LOW) ^ c3 ^ k1, p0 & _LOW)
        k0, k1 = (k0 + _W0) & _LOW, (k1 + _W1) & _LOW
    words = torch.stack([c0, c1, c2, c3], 2)
    halves = torch.stack([words & 0xFFFF, words >> 16], 3)
    return halves.reshape(rows, -1)[:, :cols]


def _plain(s):
    case, dt = s["case"], DTYPES[s["case"]["dtype"]]
    if case["op"] == "quantize":
        i, code = _indices(s["w"])
        return _values(i, code, case["cols"]).to(dt)
    if case["op"] == "dropout":
        limit = int(math.floor(case["p"] * 65536 + 0.5))
        keep = _random16(case["rows"], case["cols"], s["state"]) >= limit
        scale = torch.tensor(65536 / (65536 - limit), dtype=torch.float32, device="cuda")
        zero = scale.new_zeros(())
        return [torch.where(keep, t.float() * scale, zero).to(dt) for t in (s["x"], s["dy"])]
    W = _decode(s["codes"], s["scales"], case["in"])
    x = s["x"].float()
    if case["op"] == "gradient":
        return (W.t() @ x).to(dt)
    if case["op"] == "matmul4":
        i, code = _indices(s["x"].t())
        x = _values(i, code, case["in"]).t()
    return (W @ x).to(dt)


def run(state):
    if not own:
        return _plain(state)
    S, case = _package(), state["case"]
    dt = DTYPES[case["dtype"]]
    if case["op"] == "quantize":
        return S.mx4_dequantize(S.mx4_quantize(state["w"]), dt)
    if case["op"] == "dropout":
        return [S.dropout(t, case["p"], state["state"]) for t in (state["x"], state["dy"])]
    if case["op"] == "gradient":
        return S.mx4_matmul(state["W"], state["x"], transposed=True)
    if case["op"] == "matmul4":
        return S.mx4_matmul(state["W"], S.mx4_quantize(state["x"].t()), out_dtype=dt)
    return S.mx4_matmul(state["W"], state["x"])


# ------------------------------------------------------- the definition --

def _rounded(w):
    """What stands for w in float64: each element of a block to the nearest of its grid,
    whose step doubles at 2 and at 4 times the block's scale."""
    rows, cols = w.shape
    out = torch.empty(rows, cols, dtype=torch.float64, device=w.device)
    for first in range(0, cols, BLOCK):
        b = w[:, first:first + BLOCK].double()
        top = b.abs().amax(1, keepdim=True)
        scale = torch.exp2(torch.clamp(torch.floor(torch.log2(top)) - 2.0, min=-127.0))
        a = b / torch.where(top == 0, 1.0, scale)
        step = torch.where(a.abs() < 2, 0.5, torch.where(a.abs() < 4, 1.0, 2.0))
        out[:, first:first + BLOCK] = (torch.clamp(torch.round(a / step) * step, -6.0, 6.0)
                                       * torch.where(top == 0, 1.0, scale))
    return out


def _weights(s, cols):
    table = torch.tensor(_ELEMENTS + [-v for v in _ELEMENTS], dtype=torch.float64, device="cuda")
    codes, W = s["codes"].long(), None
    W = torch.empty(codes.shape[0], 2 * codes.shape[1], dtype=torch.float64, device="cuda")
    W[:, 0::2], W[:, 1::2] = table[codes % 16], table[codes // 16]
    return (W * torch.exp2(s["scales"].double() - 127).repeat_interleave(BLOCK, 1))[:, :cols]


def _uniform(rows, cols, seed, step):
    """The random halves of every element, from the generator's definition on words of
    16 bits (so that no product passes 63 bits)."""
    def product(a, m):
        lo, hi = a * (m & 0xFFFF), a * (m >> 16)
        total = lo + ((hi & 0xFFFF) << 16)
        return (hi >> 16) + (total >> 32), total & _LOW

    groups = -(-cols // 8)
    n = torch.arange(rows * groups, device="cuda")
    v = [n % groups, n // groups, torch.full_like(n, step % 2**32),
         torch.full_like(n, step // 2**32)]
    for i in range(7):
        k = [(seed % 2**32 + i * _W0) % 2**32, (seed // 2**32 + i * _W1) % 2**32]
        h0, l0 = product(v[0], _M0)
        h1, l1 = product(v[2], _M1)
        v = [h1 ^ v[1] ^ k[0], l1, h0 ^ v[3] ^ k[1], l0]
    out = torch.empty(rows, groups, 8, dtype=torch.int32, device="cuda")
    for i in range(8):
        out[:, :, i] = ((v[i // 2] >> (16 * (i % 2))) % 65536).reshape(rows, groups)
    return out.reshape(rows, 8 * groups)[:, :cols]


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "quantize":
        return _rounded(s["w"])
    if case["op"] == "dropout":
        limit = round(case["p"] * 65536)
        step, key = int(s["state"][1]), int(s["state"][0])
        dropped = _uniform(case["rows"], case["cols"], key, step) < limit
        return [(t.double() * 65536 / (65536 - limit)).masked_fill_(dropped, 0.0)
                for t in (s["x"], s["dy"])]
    W = _weights(s, case["in"])
    if case["op"] == "gradient":
        return torch.mm(W.t().contiguous(), s["x"].double())
    x = s["x"].double()
    if case["op"] == "matmul4":
        x = _rounded(s["x"].t()).t().contiguous()
    return torch.mm(W, x)


def work(case):
    e = BYTES[case["dtype"]]
    if case["op"] == "quantize":
        n, blocks = case["rows"] * case["cols"], case["rows"] * -(-case["cols"] // BLOCK)
        # the input, the codes and scales, and the values read back
        return {"bytes": 2 * e * n + 17 * blocks, "flops": 4 * n}
    if case["op"] == "dropout":
        n = case["rows"] * case["cols"]
        return {"bytes": 4 * e * n, "flops": 2 * n}
    T, n_in, n_out = case["tokens"], case["in"], case["out"]
    weights = 17 * n_out * -(-n_in // BLOCK)
    return {"bytes": weights + e * T * (n_in + n_out), "flops": 2 * T * n_in * n_out}
