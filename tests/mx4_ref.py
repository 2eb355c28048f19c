"""Float64 definitions of the 4-bit microscaled matrices and of dropout, and the
bounds their results are held to.  Whole numbers and numpy only."""
import numpy as np
import torch

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
ELEMENTS = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6])


def quantize(w):
    """Codes [rows, 16 nb] and scales [rows, nb] of a float64 matrix, element by element."""
    rows, cols = w.shape
    nb = -(-cols // 32)
    codes, scales = np.zeros((rows, 32 * nb), np.uint8), np.empty((rows, nb), np.uint8)
    for b in range(nb):
        block = w[:, 32 * b:32 * b + 32]
        top = np.abs(block).max(1)
        with np.errstate(divide="ignore", invalid="ignore"):
            e = np.floor(np.log2(top)) - 2
        # log2 of a value just below a power of two may round up to it
        e = np.where(np.exp2(e + 2) > top, e - 1, e)
        s = np.clip(e + 127, 0, 254)
        s = np.where(top == 0, 127, s)
        s = np.where(np.isfinite(top), s, 255)
        scales[:, b] = s
        with np.errstate(invalid="ignore"):
            a = np.abs(block) / np.exp2(s - 127)[:, None]
        # the nearest element; of two equally near ones the even index
        d = np.abs(a[:, :, None] - ELEMENTS[:8])
        d = np.where(np.isnan(d), 0, d)
        i = d.argmin(2)
        up = np.minimum(i + 1, 7)
        tie = np.take_along_axis(d, up[:, :, None], 2)[:, :, 0] == d.min(2)
        i = np.where(tie & (i % 2 == 1), up, i)
        i = np.where((s == 255)[:, None], 0, i + 8 * np.signbit(block))
        codes[:, 32 * b:32 * b + block.shape[1]] = i
    return codes[:, 0::2] | (codes[:, 1::2] << 4), scales


def dequantize(codes, scales, cols):
    e = np.empty((codes.shape[0], 2 * codes.shape[1]))
    e[:, 0::2], e[:, 1::2] = ELEMENTS[codes & 15], ELEMENTS[codes >> 4]
    s = np.exp2(scales.astype(np.float64) - 127)
    s[scales == 255] = np.nan
    return (e * np.repeat(s, 32, 1))[:, :cols]


def random_mx4(rng, rows, cols, low=118, high=134):
    """Codes and scales of every kind of element."""
    nb = -(-cols // 32)
    i = rng.integers(0, 16, (rows, 32 * nb)).astype(np.uint8)
    i[:, cols:] = 0
    scales = rng.integers(low, high + 1, (rows, nb)).astype(np.uint8)
    return i[:, 0::2] | (i[:, 1::2] << 4), scales


def bound(ref, terms, magnitude, dtype):
    """How far a result may be from `ref`: f32 sums of `terms` exact products, in any
    order, each addition off by at most 2^-23 of the sum of magnitudes (truncation), and
    one rounding, of at most half a step."""
    info = torch.finfo(DTYPES[dtype])
    return (terms * 2.0 ** -23 * magnitude + info.eps / 2 * (np.abs(ref) + terms * 2.0 ** -23
            * magnitude) + info.smallest_normal * info.eps)


M0, M1, W0, W1 = 0xD2511F53, 0xCD9E8D57, 0x9E3779B9, 0xBB67AE85


def philox(counter, key, rounds=7):
    """Philox 4x32 on Python's whole numbers."""
    c, k = list(counter), list(key)
    for _ in range(rounds):
        p, q = c[0] * M0, c[2] * M1
        c = [(q >> 32) ^ c[1] ^ k[0], q & 0xffffffff, (p >> 32) ^ c[3] ^ k[1], p & 0xffffffff]
        k = [(k[0] + W0) & 0xffffffff, (k[1] + W1) & 0xffffffff]
    return c


def random16(rows, cols, seed, step, row0=0, col0=0):
    """The 16 random bits of each element of a part of a matrix."""
    r, c = np.meshgrid(np.arange(row0, row0 + rows, dtype=np.uint64),
                       np.arange(col0, col0 + cols, dtype=np.uint64), indexing="ij")
    low = np.uint64(0xffffffff)
    v = [c >> np.uint64(3), r, np.full_like(r, step & 0xffffffff), np.full_like(r, (step >> 32) & 0xffffffff)]
    k = [seed & 0xffffffff, (seed >> 32) & 0xffffffff]
    for _ in range(7):
        p, q = v[0] * np.uint64(M0), v[2] * np.uint64(M1)
        s = np.uint64(32)
        v = [(q >> s) ^ v[1] ^ np.uint64(k[0]), q & low, (p >> s) ^ v[3] ^ np.uint64(k[1]), p & low]
        k = [(k[0] + W0) & 0xffffffff, (k[1] + W1) & 0xffffffff]
    part = c & np.uint64(7)
    word = np.choose((part >> np.uint64(1)).astype(int), v)
    return ((word >> (np.uint64(16) * (part & np.uint64(1)))) & np.uint64(0xffff)).astype(np.int64)


def dropout(x, p, seed, step):
    """x (float64, a matrix) in float64: kept elements scaled in f32."""
    limit = int(np.floor(p * 65536 + 0.5))
    if limit == 65536:
        return np.zeros_like(x)
    scale = np.float64(np.float32(65536 / (65536 - limit)))
    return np.where(random16(*x.shape, seed, step) >= limit, x * scale, 0.0)
