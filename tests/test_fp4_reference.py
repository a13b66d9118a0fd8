"""Pins of the tests' plain forms (fp4_reference) against independent sources:
torch's E4M3 cast, rational arithmetic, the oracle's decode and its GEMV."""
from fractions import Fraction

import numpy as np
import pytest
import torch

import fp4_reference as ref
import oracle
import synth


def test_tables():
    t2, t8 = oracle.tables()
    assert np.array_equal(ref.E2M1, t2[:8])
    assert np.array_equal(ref.E4M3, t8[:127])
    got = ref.e4m3(np.arange(256))
    want = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(got, want, equal_nan=True)


def test_scale_rounding_is_torchs_cast():
    v = np.random.default_rng(1).uniform(0, 448, 20000).astype(np.float32)
    v = np.concatenate([v, np.exp2(np.random.default_rng(2).uniform(-12, 8.8, 20000)).astype(np.float32)])
    want = torch.from_numpy(v).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(ref.nearest_code(v.astype(np.float64), ref.E4M3), want)


def test_rounding_in_rationals():
    """Codes of float32 values and scales against exact quotients, ties included."""
    rng = np.random.default_rng(3)
    for _ in range(200):
        g = float(np.float32(np.exp2(rng.uniform(-10, 10))))
        x = (rng.standard_normal(16) * np.exp2(rng.uniform(-6, 6))).astype(np.float32).astype(np.float64)
        if rng.random() < 0.5:
            g = 1.0
            x = rng.choice([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0], 16)
            x[0] = 6.0                                        # scale 1: every value is a tie
        codes, scale = ref.quantize(x, g)

        def nearest(q, table):
            exact = [Fraction(float(t)) for t in table]
            d = [abs(q - t) for t in exact]
            best = [i for i, v in enumerate(d) if v == min(d)]
            return best[0] if len(best) == 1 else next(i for i in best if i % 2 == 0)

        G = Fraction(g)
        assert scale[0] == nearest(max(abs(Fraction(float(v))) for v in x) / (6 * G), ref.E4M3)
        if scale[0] == 0:
            assert not codes.any()
            continue
        s = Fraction(float(ref.E4M3[scale[0]]))
        for v, c in zip(x, codes):
            assert c & 7 == nearest(abs(Fraction(float(v))) / (s * G), ref.E2M1)


def test_values_and_blocked_positions_against_the_oracle():
    inp = synth.random_inputs(129, 96, 1, 7)
    v = ref.values(inp.a, inp.sfa_plain)
    b = ref.values(inp.b, inp.sfb_plain)
    assert np.array_equal(np.einsum("lmk,lk->lm", v, b), oracle.gemv(inp, "plain").s_f64)
    assert np.array_equal(ref.from_blocked(inp.sfa_blocked[0], 129, 96), inp.sfa_plain[0])
    mask = ref.blocked_pad_mask(129, 96)
    assert (inp.sfa_blocked[0][mask] == 0x7F).all() and mask.sum() == mask.size - 129 * 6


def test_route_by_hand():
    x = np.array([[0.0, 1.0, 1.0, -np.inf], [np.nan, -np.inf, -np.inf, -np.inf], [np.inf, 0.0, np.inf, 1.0]])
    ids, w = ref.route(x, None, 2, "softmax")
    assert ids.tolist() == [[1, 2], [-1, -1], [0, 2]]
    assert np.allclose(w, [[0.5, 0.5], [0, 0], [0.5, 0.5]])
    ids, w = ref.route(x[:1], np.array([9.0, 0, 0, 99.0]), 2, "sigmoid", renormalize=False, scaling=2.0)
    assert ids.tolist() == [[0, 1]] and np.allclose(w, [[1.0, 2 / (1 + np.exp(-1.0))]])
    # two groups of two: the second group's pair is worth more
    ids, _ = ref.route(np.array([[3.0, 0.0, 2.0, 2.0]]), None, 2, "sigmoid", 2, 1, 2)
    assert ids.tolist() == [[2, 3]]
    ids, _ = ref.route(np.array([[3.0, 0.0, 2.0, 2.0]]), None, 2, "sigmoid", 2, 1, 1)
    assert ids.tolist() == [[0, 1]]


def test_lists_by_hand():
    offsets, order = ref.lists(np.array([[2, 0], [-1, 2], [5, 0]]), 4)
    assert offsets.tolist() == [0, 2, 2, 4, 4] and order.tolist() == [1, 5, 0, 3]


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16, torch.float32])
def test_the_tolerance_rejects(dtype):
    """A term left out, a row taken for another and a wrong rounding all fail."""
    rng = np.random.default_rng(5)
    a, b = rng.standard_normal((64, 512)), rng.standard_normal((32, 512))
    want, size = b @ a.T, np.abs(b) @ np.abs(a).T
    good = torch.from_numpy(want).to(dtype)
    ref.check_product(good, want, size, 512, dtype)
    for bad in (b[:, 16:] @ a[:, 16:].T, np.roll(want, 1, 0), want * (1 + 4 * ref.HALF_STEP[dtype] + 2.0 ** -12)):
        with pytest.raises(AssertionError):
            ref.check_product(torch.from_numpy(bad).to(dtype), want, size, 512, dtype)
