"""Plain 64-bit forms and layout decoders of the FP8 (E4M3, one E8M0 scale per 128) operators,
written from the text of include/svdq.h; shared by the FP8 tests."""
import numpy as np


def e4m3_values(codes: np.ndarray) -> np.ndarray:
    """E4M3 bytes -> float64 (0x7F and 0xFF are NaN)."""
    c = np.asarray(codes, np.uint8).astype(np.int64)
    ex, man = (c >> 3) & 15, (c & 7).astype(np.float64)
    v = np.where(ex > 0, np.ldexp(8.0 + man, ex - 10), np.ldexp(man, -9))
    v = np.where((c & 0x7F) == 0x7F, np.nan, v)
    return np.where(c & 0x80, -v, v)


def scale_offsets(rows: int, K: int, padded: bool = False) -> np.ndarray:
    """Byte offset of (row, group); padded: of every row below Rp and group below Gp."""
    gp = (K + 511) // 512 * 4
    r = np.arange((rows + 127) // 128 * 128 if padded else rows)[:, None]
    g = np.arange(gp if padded else K // 128)[None, :]
    return ((r // 128) * (gp // 4) + g // 4) * 512 + (r % 32) * 16 + ((r % 128) // 32) * 4 + g % 4


def scales_of(buf: np.ndarray, rows: int, K: int) -> np.ndarray:
    return np.asarray(buf, np.uint8).reshape(-1)[scale_offsets(rows, K)]


def scale_padding_of(buf: np.ndarray, rows: int, K: int) -> np.ndarray:
    """Every scale byte that belongs to no (row, group)."""
    b = np.asarray(buf, np.uint8).reshape(-1)
    used = np.zeros(b.size, bool)
    used[scale_offsets(rows, K)] = True
    return b[~used]


def scales_to_buffer(sbytes: np.ndarray, K: int) -> np.ndarray:
    rows = sbytes.shape[0]
    buf = np.zeros(scale_offsets(rows, K, padded=True).size, np.uint8)
    buf[scale_offsets(rows, K)] = sbytes
    return buf


def quantize(y: np.ndarray):
    """(codes, scale bytes) of a float64 matrix: smallest e >= -127 with max|y| <= 448 2^e."""
    rows, K = y.shape
    yg = np.asarray(y, np.float64).reshape(rows, K // 128, 128)
    a = np.abs(yg).max(2)
    e = np.full(a.shape, -127, np.int64)
    while True:
        low = a > np.ldexp(448.0, e)
        if not low.any():
            break
        e = np.where(low, e + 1, e)
    grid = e4m3_values(np.arange(127))
    w = np.abs(yg) / np.ldexp(1.0, e)[..., None]
    hi = np.clip(np.searchsorted(grid, w, side="left"), 0, 126)
    lo = np.clip(hi - 1, 0, 126)
    up = (grid[hi] - w < w - grid[lo]) | ((grid[hi] - w == w - grid[lo]) & (hi % 2 == 0))
    code = np.where(up, hi, lo) | np.where(np.signbit(yg), 0x80, 0)
    return code.reshape(rows, K).astype(np.uint8), (e + 127).astype(np.uint8)


def dequantize(codes: np.ndarray, sbytes: np.ndarray) -> np.ndarray:
    return e4m3_values(codes) * np.repeat(np.ldexp(1.0, sbytes.astype(np.int64) - 127), 128, axis=1)


def check_quantized(codes, sbytes, y64, delta, floor=0.0):
    """The codes and scales are those of some y with |y - y64| <= delta |y64| + floor: the scale
    holds the group's maximum and half of it would not; every value is within half an E4M3 step
    (2^-4 of its binade, 2^-10 below the smallest normal, times the scale) of such a y."""
    rows, K = y64.shape
    a = np.abs(y64).reshape(rows, K // 128, 128).max(2)
    e = sbytes.astype(np.int64) - 127
    lim = np.ldexp(448.0, e)
    assert np.all(a * (1 - delta) - floor <= lim), "a group's scale is too small"
    assert np.all((e == -127) | (a * (1 + delta) + floor > lim / 2)), "a group's scale is too large"
    S = np.repeat(np.ldexp(1.0, e), 128, axis=1)
    v = dequantize(codes, sbytes)
    w = np.maximum(np.abs(v), np.abs(y64) * (1 + delta)) / S
    half = np.where(w >= 2.0 ** -6, np.exp2(np.floor(np.log2(np.maximum(w, 2.0 ** -6))) - 4), 2.0 ** -10) * S
    err = np.abs(v - y64)
    bad = err > half + delta * np.abs(y64) + floor
    assert not bad.any(), f"{bad.sum()} values, first at {np.argwhere(bad)[0]}: {v[bad][0]} for {y64[bad][0]}"


def rmsnorm64(h, gamma, eps):
    y = h / np.sqrt(np.mean(h * h, axis=1, keepdims=True) + eps)
    return y if gamma is None else y * np.asarray(gamma, np.float64)


def act64(x, act):
    with np.errstate(over="ignore"):
        if act == "silu":
            return x / (1.0 + np.exp(-x))
        u = np.sqrt(2.0 / np.pi) * (x + 0.044715 * x ** 3)
        return x / (1.0 + np.exp(-2.0 * u))      # 0.5 (1 + tanh u) = 1 / (1 + exp(-2u))
