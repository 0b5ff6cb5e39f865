"""FP8 with a scale for each block of 128, from its definition, in numpy and 64 bits: the
oracle of the tests of adaptive_block_scaled_amd.fp8."""
import numpy as np

BLOCK = 128
# value of every code: sign, 4 exponent bits (bias 7), 3 mantissa bits, NaN at the end
MAGNITUDES = np.array([m * 2.0 ** -9 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
                       for e in range(16) for m in range(8)])
MAGNITUDES[127] = np.nan
VALUES = np.concatenate([MAGNITUDES, -MAGNITUDES])
MIDDLES = (MAGNITUDES[1:127] + MAGNITUDES[:126]) / 2


def blocks(n):
    return -(-n // BLOCK)


def quantize(x, square=False):
    """(codes, scales) of x [rows, K], block by block."""
    x = np.asarray(x, np.float64)
    rows, k = x.shape
    tall = BLOCK if square else 1
    codes = np.zeros((rows, k), np.uint8)
    scales = np.zeros((-(-rows // tall), blocks(k)), np.uint8)
    for i in range(scales.shape[0]):
        for b in range(scales.shape[1]):
            at = np.s_[i * tall:(i + 1) * tall, b * BLOCK:(b + 1) * BLOCK]
            v = x[at]
            if not np.isfinite(v).all():
                codes[at], scales[i, b] = 0x7F, 255
                continue
            top, e = np.abs(v).max(), -127
            if top > 0:
                e = max(-127, int(np.floor(np.log2(top))) - 9)
                while top > 448 * 2.0 ** e:
                    e += 1
            u = np.abs(v) * 2.0 ** -e
            up, down = np.searchsorted(MIDDLES, u, "right"), np.searchsorted(MIDDLES, u, "left")
            codes[at] = np.where(up % 2 == 0, up, down) + 128 * np.signbit(v)
            scales[i, b] = e + 127
    return codes, scales


def values(codes, scales):
    s = np.where(scales == 255, np.nan, 2.0 ** (scales.astype(np.float64) - 127))
    if scales.shape[0] != codes.shape[0]:
        s = s.repeat(BLOCK, 0)[:codes.shape[0]]
    return VALUES[codes] * s.repeat(BLOCK, 1)[:, :codes.shape[1]]
