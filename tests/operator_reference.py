"""Plain 64-bit statements of the optimizer step and of the MXFP4 payload, in
numpy, for the tests of those operators.  They share nothing with the library
and are written from the definitions in include/qcp.h."""
import numpy as np

MASK = 0xFFFFFFFF


def mix(x):
    """The 32-bit scramble of the stochastic rounding, on Python ints or uint64 arrays."""
    m = MASK if isinstance(x, int) else np.uint64(MASK)
    s16, s15 = (16, 15) if isinstance(x, int) else (np.uint64(16), np.uint64(15))
    a, b = (0x6A09E667, 0xBB67AE85) if isinstance(x, int) else (np.uint64(0x6A09E667), np.uint64(0xBB67AE85))
    x = x ^ (x >> s16)
    x = (x * a) & m
    x = x ^ (x >> s15)
    x = (x * b) & m
    return x ^ (x >> s16)


def random_halves(places, seed, step):
    """The 16 random bits of m and of sqrt(v) at each place of the moments."""
    key = 0
    for word in (seed & MASK, (seed >> 32) & MASK, step & MASK, (step >> 32) & MASK):
        key = mix((key + word + 0x9E3779B9) & MASK)
    places = np.asarray(places, np.uint64)
    hi = places >> np.uint64(32)
    keys = (np.uint64(key) + hi * np.uint64(0x9E3779B9)) & np.uint64(MASK)
    h = mix((places & np.uint64(MASK)) ^ keys)
    return (h & np.uint64(0xFFFF)).astype(np.float64), (h >> np.uint64(16)).astype(np.float64)


def adamw(p, g, m, v, step, lr, beta1, beta2, eps, decay, scale=1.0):
    """One step in float64 -> (p, m, v)."""
    p, g, m, v = (np.asarray(t, np.float64) for t in (p, g, m, v))
    g = g * scale
    m = beta1 * m + (1 - beta1) * g
    v = beta2 * v + (1 - beta2) * g * g
    hat = np.sqrt(v / (1 - beta2 ** step)) + eps
    return p * (1 - lr * decay) - lr * (m / (1 - beta1 ** step)) / hat, m, v


def e4m3_value(codes):
    """E4M3FN bytes -> float64."""
    c = np.asarray(codes).astype(np.int64)
    e, f = (c >> 3) & 15, c & 7
    a = np.where(e == 0, f * 2.0 ** -9, (8 + f) * 2.0 ** (e - 10.0))
    return np.where(c & 128, -a, a)


def block_scale(x, G):
    """The power-of-two scale of each block of a flat float64 array."""
    big = np.abs(x.reshape(-1, G)).max(1)
    mant, power = np.frexp(big / 448)
    power = np.maximum(np.where(mant == 0.5, power - 1, power), -126)
    return np.where(big == 0, 0.0, np.ldexp(1.0, power))


def stochastic_e4m3(x, scale, half, slack=0.0):
    """|x| / scale to the E4M3 grid with the 16 random bits `half`, sign kept.
    `slack` moves the position between the two neighbours (in spacings)."""
    q = np.abs(x) / np.where(scale == 0, 1.0, scale)
    unit = 2.0 ** (np.maximum(np.frexp(q)[1] - 1, -6) - 3.0)
    return np.copysign(np.maximum(np.floor(q / unit + half / 65536 + slack), 0) * unit, x)


# ------------------------------------------------------------------ MXFP4

E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])


def padded(n):
    return -(-n // 128) * 128


def mx_payload(x):
    """float64 [rows, cols] (values of a 16- or 32-bit type) -> (codes, scales) bytes."""
    rows, cols = x.shape
    t = np.zeros((rows, padded(cols)))
    t[:, :cols] = x
    b = t.reshape(rows, -1, 32)
    with np.errstate(invalid="ignore", over="ignore"):
        big = np.abs(b).max(2)
        ok = np.isfinite(big)
        # the exponent field of the absmax in fp32: floor(log2) + 127, 0 for subnormals
        field = np.where(big >= 2.0 ** -126, np.frexp(np.where(ok, big, 1.0))[1] - 1 + 127, 0)
        e = np.where(ok, np.maximum(field - 2, 0), 255)
        a = np.abs(b) / np.where(ok, np.ldexp(1.0, e - 127), 1.0)[:, :, None]
        below = np.searchsorted(E2M1, a, side="right") - 1
        below = np.clip(below, 0, 7)
        above = np.minimum(below + 1, 7)
        d0, d1 = a - E2M1[below], E2M1[above] - a
        up = (d1 < d0) | ((d1 == d0) & (below % 2 == 1))
        code = np.where(up & (above > below), above, below) + np.where(np.signbit(b), 8, 0)
    code = code.reshape(rows, -1).astype(np.uint8)
    return code[:, 0::2] | (code[:, 1::2] << 4), e.astype(np.uint8), ok


def mx_values(codes, scales):
    """payload bytes -> float64 [lines, P]."""
    c = np.stack([codes & 15, codes >> 4], 2).reshape(codes.shape[0], -1).astype(np.int64)
    v = np.where(c & 8, -1.0, 1.0) * E2M1[c & 7]
    s = np.where(scales == 255, np.nan, np.ldexp(1.0, scales.astype(np.int64) - 127))
    return v * np.repeat(s, 32, axis=1)
