"""64-bit plain forms of the e4m3 operators (test-side only)."""
import numpy as np
import torch

TINY = np.float32(2.0 ** -100)


def decode_table():
    """The value of every e4m3 code: sign, 4 exponent bits (bias 7), 3 fraction
    bits; exponent 0 is subnormal, code 0x7f NaN, no infinity."""
    out = np.empty(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        v = m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        if e == 15 and m == 7:
            v = np.nan
        out[c] = -v if c & 128 else v
    return out


E4M3 = decode_table()


def values(q):
    """fp64 values of e4m3 codes (uint8 or float8_e4m3fn tensor)."""
    return E4M3[q.cpu().view(torch.uint8).numpy()]


def round_e4m3(v):
    """The nearest e4m3 value of fp64 v, |v| <= 464, ties to the even code."""
    v = np.asarray(v, dtype=np.float64)
    a = np.abs(v)
    with np.errstate(divide="ignore"):
        e = np.floor(np.log2(np.where(a > 0, a, 1.0)))
    step = 2.0 ** (np.maximum(e, -6) - 3)
    return np.copysign(np.minimum(np.rint(a / step) * step, 448.0), v)


def dequantize(q, s, block=1):
    """fp64 values of codes [rows, K] with scales per 1 x 128 or 128 x 128."""
    v = values(q)
    s = s.cpu().numpy().astype(np.float64)
    if block == 128:
        s = np.repeat(s, 128, 0)[:v.shape[0]]
    return v * np.repeat(s, 128, 1)[:, :v.shape[1]]


def quantize_ref(x, block=1):
    """The codes' values and the scales of fp32-representable x [rows, K], each
    step rounded as the header states it (numpy's fp32 is IEEE)."""
    x = np.asarray(x, dtype=np.float32)
    rows, K = x.shape
    KB, RB = -(-K // 128), -(-rows // block)
    mag = np.where(np.isfinite(x), np.abs(x), np.float32(0))
    pad = np.zeros((RB * block, KB * 128), np.float32)
    pad[:rows, :K] = mag
    amax = pad.reshape(RB, block, KB, 128).max(axis=(1, 3))
    amax = np.maximum(amax, TINY)
    s = amax / np.float32(448)
    r = np.float32(448) / amax
    each = np.repeat(np.repeat(r, block, 0)[:rows], 128, 1)[:, :K]
    with np.errstate(invalid="ignore"):
        p = x * each
    q = np.where(np.isfinite(x), round_e4m3(np.where(np.isfinite(x), p, 0)), np.nan)
    return q, s


def act64(g, act):
    if act == "geglu":
        return 0.5 * g * (1 + np.tanh(np.sqrt(2 / np.pi) * (g + 0.044715 * g ** 3)))
    return g / (1 + np.exp(-g))


def sum_bound(K):
    """|error| of a product's sum over its sum of absolute products: each block's
    128 products are added in one chain (at most 128 steps), the block sums in
    another, and scaled by a rounded product of two scales; a step of the tensor
    cores may truncate, so it counts 2^-23, not 2^-24."""
    return (128 + -(-K // 128) + 4) * 2.0 ** -23
