"""The dense operators' definitions in 64 bits (numpy): 8-bit rows, their
product, and the residual stream's step between two blocks. Written from the
formats and formulas, apart from the kernels; test infrastructure only."""
import numpy as np

BLOCK = 128


def e4m3_table():
    """The values of the codes 0x00 .. 0x7E (0x7F is NaN): sign-free, ascending."""
    codes = np.arange(0x7F)
    e, m = codes >> 3, codes & 7
    return np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (np.maximum(e, 1) - 10.0))


TABLE = e4m3_table()


def e4m3_decode(codes):
    codes = np.asarray(codes, dtype=np.int64)
    size = np.concatenate([TABLE, [np.nan]])[codes & 0x7F]
    return np.where(codes & 0x80, -size, size)


def e4m3_encode(x):
    """To the nearest value, ties to the even code; NaN and infinities to 0x7F."""
    x = np.asarray(x, dtype=np.float64)
    a = np.minimum(np.where(np.isfinite(x), np.abs(x), 0.0), TABLE[-1])
    hi = np.clip(np.searchsorted(TABLE, a), 1, len(TABLE) - 1)
    lo = hi - 1
    up, down = TABLE[hi] - a, a - TABLE[lo]
    code = np.where(up < down, hi, np.where(down < up, lo, np.where(hi % 2 == 0, hi, lo)))
    code = code + 0x80 * np.signbit(x)
    return np.where(np.isfinite(x), code, 0x7F).astype(np.uint8)


def scale_byte(amax):
    """The smallest e with amax <= 448 * 2^(e - 127), from 0 on."""
    for e in range(255):
        if amax <= 448 * 2.0 ** (e - 127):
            return e
    raise ValueError(amax)


def quantize_rows(x):
    """[rows, k] -> codes [rows, k], scales [rows, 4 * ceil(k / 512)] (127 past the last block)."""
    x = np.asarray(x, dtype=np.float64)
    rows, k = x.shape
    codes = np.zeros((rows, k), np.uint8)
    scales = np.full((rows, 4 * -(-k // 512)), 127, np.uint8)
    for r in range(rows):
        for b in range(-(-k // BLOCK)):
            v = x[r, b * BLOCK:(b + 1) * BLOCK]
            fine = np.abs(v[np.isfinite(v)])
            scales[r, b] = scale_byte(fine.max() if fine.size else 0.0)
            codes[r, b * BLOCK:(b + 1) * BLOCK] = e4m3_encode(v / 2.0 ** (float(scales[r, b]) - 127))
    return codes, scales


def dequantize(codes, scales):
    k = codes.shape[1]
    power = np.where(scales == 255, np.nan, 2.0 ** (scales.astype(np.float64) - 127))
    return e4m3_decode(codes) * np.repeat(power, BLOCK, axis=1)[:, :k]


def product(x, w):
    """Dequantized rows: the products' sums, and the sums of their magnitudes (what errors are measured by)."""
    return x @ w.T, np.abs(x) @ np.abs(w).T


def norm(v, eps):
    return v / np.sqrt(np.mean(v * v, axis=-1, keepdims=True) + eps)


def residual_norm(x, block=None, gate=None, residual_scale=1.0, eps=1e-6, post_norm=False, post_weight=None,
                  pre_weight=None):
    """(y, normed, the magnitudes that y is the sum of)"""
    y, size = x, np.abs(x)
    if block is not None:
        b = norm(block, eps) if post_norm else block
        if post_weight is not None:
            b = b * post_weight
        if gate is not None:
            b = b * gate
        y = x + residual_scale * b
        size = size + np.abs(residual_scale * b)
    normed = norm(y, eps)
    return y, normed if pre_weight is None else normed * pre_weight, size
