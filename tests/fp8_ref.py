"""The 8-bit block-128 definitions in 64 bits (numpy), written from the formulas."""
import numpy as np


def e4m3_values():
    """Value of every E4M3 code 0..0x7E (bias 7, three mantissa bits)."""
    v = []
    for c in range(0x7F):
        e, m = c >> 3, c & 7
        v.append(m * 2.0 ** -9 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7))
    return np.array(v)


VALUES = e4m3_values()


def to_codes(q):
    """Nearest E4M3 code of each value (ties to the even code), sign included."""
    a = np.abs(q)
    hi = np.clip(np.searchsorted(VALUES, a), 1, 0x7E)
    lo = hi - 1
    dl, dh = a - VALUES[lo], VALUES[hi] - a
    c = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    return (c | np.where(np.signbit(q), 0x80, 0)).astype(np.uint8)


def decode(codes):
    v = np.append(VALUES, np.nan)[codes & 0x7F]
    return np.where(codes & 0x80, -v, v)


def quantize(x, tile):
    """(codes rows x ld, scales) of float32 x, laid out as fp8_quantize_b128 writes them."""
    rows, cols = x.shape
    ld = -(-cols // 16) * 16
    step = 128 if tile else 1
    nr, nc = -(-rows // step), -(-cols // 128)
    codes = np.zeros((rows, ld), np.uint8)
    scales = np.zeros((nr, nc), np.float32)
    for c in range(nc):
        part = x[:, 128 * c:128 * c + 128].astype(np.float64)
        a = np.abs(part).max(1)
        if tile:
            a = np.array([a[128 * r:128 * r + 128].max() for r in range(nr)])
        s = np.maximum((a / 448.0).astype(np.float32), np.float32(2.0 ** -126))
        scales[:, c] = s
        full = np.repeat(s, step)[:rows].astype(np.float64)[:, None]
        codes[:, 128 * c:128 * c + part.shape[1]] = to_codes((part / full).astype(np.float32).astype(np.float64))
    return codes, scales if tile else np.ascontiguousarray(scales.T)


def value(codes, scales, tile):
    """Dequantized operand in 64 bits."""
    s = scales if tile else scales.T
    rows = np.arange(codes.shape[0]) // (128 if tile else 1)
    return decode(codes) * s.astype(np.float64)[rows][:, np.arange(codes.shape[1]) // 128]
