"""CPU: the frequencies of rotary positions, by every scaling, against the formulas."""
import math

import numpy as np
import pytest

import block_scaled_fp4_gemv_amd as g


def plain(R, base):
    return base ** (-2.0 * np.arange(R // 2) / R)


@pytest.mark.parametrize("R,base", [(2, 10000.0), (64, 10000.0), (96, 500000.0), (2048, 1e6)])
def test_unscaled_linear_base(R, base):
    f = plain(R, base)
    np.testing.assert_allclose(g.nvfp4_rope_frequencies(R, base), f, rtol=1e-14)
    np.testing.assert_allclose(g.nvfp4_rope_frequencies(R, base, "linear", 4.0), f / 4, rtol=1e-14)
    if R > 2:
        got = np.array(g.nvfp4_rope_frequencies(R, base, "base", 4.0))
        np.testing.assert_allclose(got, plain(R, base * 4.0 ** (R / (R - 2))), rtol=1e-12)
        # the first pair keeps its wave, the last is stretched by the factor
        np.testing.assert_allclose([got[0], got[-1]], [f[0], f[-1] / 4], rtol=1e-12)


def test_bands():
    f, L, low, high, factor = plain(128, 500000.0), 8192.0, 1.0, 4.0, 8.0
    got = np.array(g.nvfp4_rope_frequencies(128, 500000.0, "bands", factor, L, low, high))
    wave = 2 * math.pi / f
    for j in range(64):
        if wave[j] < L / high:
            want = f[j]
        elif wave[j] > L / low:
            want = f[j] / factor
        else:
            smooth = (L / wave[j] - low) / (high - low)
            want = (1 - smooth) * f[j] / factor + smooth * f[j]
        assert abs(got[j] - want) <= 1e-13 * want


def test_ramp():
    R, base, L, low, high, factor = 128, 10000.0, 4096.0, 1.0, 32.0, 16.0
    f = plain(R, base)
    got = np.array(g.nvfp4_rope_frequencies(R, base, "ramp", factor, L, low, high))
    pair = lambda turns: R * math.log(L / (turns * 2 * math.pi)) / (2 * math.log(base))  # noqa: E731
    first, last = max(math.floor(pair(high)), 0), min(math.ceil(pair(low)), R - 1)
    ramp = np.clip((np.arange(64) - first) / (last - first), 0, 1)
    np.testing.assert_allclose(got, f / factor * ramp + f * (1 - ramp), rtol=1e-13)
    assert got[0] == 1.0 and abs(got[-1] * factor / f[-1] - 1) < 1e-13


@pytest.mark.parametrize("args,status", [
    ((0, 1e4), g.NVFP4_ERR_INVALID_SHAPE), ((3, 1e4), g.NVFP4_ERR_INVALID_SHAPE), ((2050, 1e4), g.NVFP4_ERR_INVALID_SHAPE),
    ((64, 1.0), g.NVFP4_ERR_INVALID_SCALE), ((64, math.inf), g.NVFP4_ERR_INVALID_SCALE), ((64, math.nan), g.NVFP4_ERR_INVALID_SCALE),
    ((64, 1e4, 5), g.NVFP4_ERR_INVALID_ROTATION), ((64, 1e4, -1), g.NVFP4_ERR_INVALID_ROTATION),
    ((64, 1e4, "linear", 0.5), g.NVFP4_ERR_INVALID_SCALE), ((64, 1e4, "linear", math.nan), g.NVFP4_ERR_INVALID_SCALE),
    ((2, 1e4, "base", 2.0), g.NVFP4_ERR_INVALID_ROTATION), ((64, 1e4, "bands", 2.0, 0.0, 1.0, 4.0), g.NVFP4_ERR_INVALID_ROTATION),
    ((64, 1e4, "bands", 2.0, 8192.0, 4.0, 4.0), g.NVFP4_ERR_INVALID_ROTATION),
    ((64, 1e4, "ramp", 2.0, 8192.0, 0.0, 4.0), g.NVFP4_ERR_INVALID_ROTATION),
    ((64, 1e4, "ramp", 2.0, 8192.0, 1.0, math.inf), g.NVFP4_ERR_INVALID_ROTATION),
])
def test_refused(args, status):
    with pytest.raises(g.Nvfp4Error) as e:
        g.nvfp4_rope_frequencies(*args)
    assert e.value.status == status


def test_no_room_is_refused():
    assert g.lib().nvfp4_rope_frequencies(None, 64, 1e4, None) == g.NVFP4_ERR_NULL_POINTER
