"""Pins of the block-scaled e4m3 oracle: the scale's defining inequality, the
rounding error's bound, exact values, the storage order's worked bytes."""

import numpy as np
import pytest

from oracle import fp8_block as fb


@pytest.mark.parametrize("square", [0, 1])
def test_scale_is_the_least_power_of_two(square):
    rng = np.random.default_rng(1)
    x = rng.standard_normal((130, 300)) * 2.0 ** rng.uniform(-20, 20, (130, 1))
    x[3] = 0.0
    q, s = fb.quantize(x, square)
    v = fb.decode(q, s)
    for r in range(130):
        for b in range(3):
            g = x[r - r % 128:r - r % 128 + 128, b * 128:(b + 1) * 128] if square else x[r, b * 128:(b + 1) * 128]
            amax, scale = np.abs(g).max(), 2.0 ** (float(s[r, b]) - 127)
            if amax == 0:
                assert s[r, b] == 127
                continue
            assert amax <= 448 * scale and amax > 448 * scale / 2
            # half a step of e4m3: 2^-4 of the value, 2^-10 of the scale among the subnormals
            err = np.abs(v[r, b * 128:(b + 1) * 128] - x[r, b * 128:(b + 1) * 128])
            assert (err <= np.maximum(2.0 ** -4 * np.abs(x[r, b * 128:(b + 1) * 128]), 2.0 ** -10 * scale)).all()


def test_exact_values_and_special_groups():
    x = np.zeros((2, 260))
    x[0, :3] = [448.0, -1.75, 0.015625]
    x[0, 128] = 449.0
    x[0, 256] = np.inf
    x[1, 0] = np.nan
    q, s = fb.quantize(x, 0)
    assert list(s[0]) == [127, 128, 255] and list(s[1]) == [255, 127, 127]
    assert list(fb.decode(q, s)[0, :3]) == [448.0, -1.75, 0.015625]
    assert fb.decode(q, s)[0, 128] == 448.0      # 224.5 rounds to 224, times 2
    assert (q[0, 256:] == 0x7F).all() and (q[1, :128] == 0x7F).all() and (q[1, 128:] == 0).all()


def test_storage_order():
    s = np.arange(200 * 6, dtype=np.int64).reshape(200, 6) % 120
    out = fb.store(s.astype(np.uint8))
    assert out.size == 2 * 2 * 512
    assert out[0] == s[0, 0] and out[3] == s[0, 3]          # four groups of a row lie side by side
    assert out[16] == s[1, 0] and out[4] == s[32, 0]        # then rows 32 apart, then the next row
    assert out[512] == s[128, 0] and out[1024] == s[0, 4]   # next row atom, next four groups
    assert out[1024 + 2] == 127                             # group 6 does not exist
    assert out[512 + 31 * 16 + 12] == 127                   # nor row 255
