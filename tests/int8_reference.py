"""Plain 64-bit statements of the INT8 payload with one scale per row and of its
products, in numpy, from the definitions in include/qcp.h.  They share nothing with the
library."""
import numpy as np

# the most that a rounding to a type is off, relative to the value, and the least step's half
UNIT = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}
LEAST = {"f32": 2.0 ** -150, "f16": 2.0 ** -25, "bf16": 2.0 ** -134}


def padded(n):
    return -(-n // 128) * 128


def payload(x):
    """float64 [rows, cols] (values of a 16- or 32-bit type) -> (int8 [rows, P], fp32 scales
    [rows]).  Scale and quotient are fp32 quotients: a quotient of two fp32 numbers in 64
    bits, rounded to 32, is the fp32 one (53 >= 2 * 24 + 2 bits)."""
    rows, cols = x.shape
    codes = np.zeros((rows, padded(cols)), np.int8)
    scales = np.zeros(rows, np.float32)
    if cols:
        with np.errstate(all="ignore"):
            big = np.abs(x).max(1)
            ok = np.isfinite(big)
            scales = np.where(ok, (np.where(ok, big, 0) / 127).astype(np.float32), np.float32("nan"))
            s = scales.astype(np.float64)
            live = ok & (s > 0)
            q = (np.where(live[:, None], x, 0) / np.where(live, s, 1)[:, None]).astype(np.float32)
            codes[:, :cols] = np.clip(np.rint(q), -127, 127)
    return codes, scales


def read(codes, scales, dt):
    """What a payload stands for in a type, float64: the fp32 product, rounded to it."""
    with np.errstate(all="ignore"):
        v = (codes.astype(np.float64) * scales.astype(np.float64)[:, None]).astype(np.float32)
        if dt == "f16":
            v = v.astype(np.float16)
        elif dt == "bf16":
            b = v.view(np.uint32).astype(np.uint64)
            b = (b + np.uint64(0x7FFF) + ((b >> np.uint64(16)) & np.uint64(1))) & np.uint64(0xFFFF0000)
            v = np.where(np.isnan(v), v, b.astype(np.uint32).view(np.float32))
    return v.astype(np.float64)


def product(a, b):
    """Two payloads -> float64 [M, N]: the sums are exact (below 2^53)."""
    sums = a[0].astype(np.float64) @ b[0].astype(np.float64).T
    return sums * a[1].astype(np.float64)[:, None] * b[1].astype(np.float64)[None, :]


def product_bound(want, dt):
    """Roundings of int8_matmul: of the sum, of the scales' product and of their product, each
    2^-24 of the value, and of the result to fp32 where it is subnormal; then to the type."""
    three = (1 + 2.0 ** -24) ** 3 - 1
    return np.abs(want) * (three + (0 if dt == "f32" else UNIT[dt] * (1 + three))) + LEAST["f32"] * 2 + \
        (0 if dt == "f32" else LEAST[dt])
