"""e4m3 with a power-of-two scale for each group of 128 elements (fp64 oracle;
test infrastructure only, see oracle/__init__.py).

  * group: 128 consecutive elements of a row (the last one shorter), or a block
    of 128 x 128 whose rows share the scale;
  * scale: the least 2^e, e >= -127, with amax <= 448 * 2^e (1 when amax is 0),
    stored as the byte e + 127; a group with an infinity or a NaN: byte 255, all
    codes NaN;
  * code: e4m3(x / scale), nearest even.  The quotient is exact in fp64, so the
    rounding decision is the definition's;
  * storage order of the scales: 512-byte atoms of 128 rows x 4 groups.
"""

import numpy as np

from oracle.fp8 import e4m3_decode, e4m3_encode

GROUP = 128


def quantize(x, square):
    """(codes uint8 [rows, cols], scale bytes uint8 [rows, groups])."""
    x = np.asarray(x, dtype=np.float64)
    rows, cols = x.shape
    groups = -(-cols // GROUP)
    codes = np.zeros((rows, cols), dtype=np.uint8)
    scales = np.zeros((rows, groups), dtype=np.uint8)
    step = GROUP if square else 1
    for r in range(0, rows, step):
        for b in range(groups):
            part = x[r:r + step, b * GROUP:(b + 1) * GROUP]
            if not np.isfinite(part).all():
                byte = 255
                code = np.full(part.shape, 0x7F, dtype=np.uint8)
            else:
                amax = np.abs(part).max()
                byte = 127
                if amax > 0:
                    byte = 0
                    while amax > 448.0 * 2.0 ** (byte - 127):
                        byte += 1
                code = e4m3_encode(part * 2.0 ** (127 - byte))
            codes[r:r + step, b * GROUP:(b + 1) * GROUP] = code
            scales[r:r + step, b] = byte
    return codes, scales


def store(scales):
    """Scale bytes [rows, groups] in their storage order (127 beyond the matrix)."""
    rows, groups = scales.shape
    ra, ga = -(-rows // 128), -(-groups // 4)
    out = np.full(ra * ga * 512, 127, dtype=np.uint8)
    for r in range(rows):
        for b in range(groups):
            out[((b // 4) * ra + r // 128) * 512 + 16 * (r % 32) + 4 * (r % 128 // 32) + b % 4] = scales[r, b]
    return out


def decode(codes, scales):
    """Values of a quantized matrix in fp64."""
    v = e4m3_decode(codes)
    s = np.where(scales == 255, np.nan, 2.0 ** (scales.astype(np.float64) - 127))
    return v * np.repeat(s, GROUP, axis=1)[:, :v.shape[1]]
