"""Pins of the draft operators' fp64 reference (CPU only): closed forms, brute
force and exact small cases."""

import itertools

import numpy as np
import pytest

from oracle import draft as OD
from oracle import processed_distribution


def test_e2m1_rounds_to_nearest_even():
    v = OD.e2m1_values()
    # the format: one fraction bit, two exponent bits of bias 1
    for c in range(8):
        e, f = c >> 1, c & 1
        assert v[c] == (f / 2 if e == 0 else (1 + f / 2) * 2.0 ** (e - 1)) and v[c + 8] == -v[c]
    for x in np.linspace(-6, 6, 4801):
        d = np.abs(v[:8] - abs(x))
        best = np.flatnonzero(d == d.min())
        code = int(OD.to_e2m1(x)) & 7
        assert code in best and (len(best) == 1 or code % 2 == 0)


def test_scale_is_the_smallest_power_of_two():
    for a in [6.0, 6.0000001, 5.99, 3.0, 3.0000002, 1e-30, 3e38, 1.0, 0.75]:
        s = 2.0 ** (int(OD.scale4_byte(a)) - 127.0)
        assert a / s <= 6 < a / (s / 2)
    assert OD.scale4_byte(0.0) == 127 and OD.scale4_byte(np.inf) == 255
    assert OD.scale4_byte(1e-45) == 1 and OD.scale4_byte(np.nan) == 255


def test_quantize_is_exact_on_its_own_values():
    rng = np.random.default_rng(0)
    code = rng.integers(0, 16, (5, 96)).astype(np.uint8)
    code[:, ::32] = 7                                  # every block reaches 6
    q, s = OD.pack_codes(code), rng.integers(100, 150, (5, 3)).astype(np.uint8)
    q2, s2 = OD.quantize4(OD.dequantize4(q, s))
    assert np.array_equal(s, s2)
    assert np.array_equal(OD.unpack_codes(q2) & 7, code & 7)
    assert np.array_equal(OD.unpack_codes(q), code)


@pytest.mark.parametrize("T,k,p,mp", itertools.product((0.5, 1.0), (0, 2, 3), (1.0, 0.6), (0.0, 0.3, 1.0)))
def test_filtered_by_brute_force(T, k, p, mp):
    rng = np.random.default_rng(int(10 * T) + k)
    for _ in range(20):
        z = rng.normal(size=7) * 2
        z[rng.integers(7)] = z[0]                      # ties
        P, _ = OD.filtered(z, T, k, p, mp)
        w = np.exp((z - z.max()) / T)
        keep = np.ones(7, bool)
        if k:
            keep &= np.array([(z > v).sum() < k for v in z])
        tot = w[keep].sum()
        if p < 1:
            p32 = float(np.float32(p))
            keep &= np.array([w[keep & (z > v)].sum() < p32 * tot for v in z])
        keep &= w >= float(np.float32(mp))
        assert np.array_equal(P > 0, keep)
        assert np.allclose(P, np.where(keep, w, 0) / w[keep].sum(), rtol=1e-14, atol=0)


def test_filtered_without_min_p_is_the_processed_distribution():
    z = np.random.default_rng(3).normal(size=200) * 3
    for T, k, p in ((0.7, 0, 1.0), (1.0, 20, 0.5), (1.3, 0, 0.25)):
        assert np.array_equal(OD.filtered(z, np.float32(T), k, p)[0],
                              processed_distribution(z, float(np.float32(T)), k, p)[0])


def test_greedy_and_rows_without_a_distribution():
    P, _ = OD.filtered([1.0, 3.0, 3.0, -np.inf], 0.0, 1, 0.5, 0.5)
    assert list(P) == [0, 1, 0, 0] and OD.draw(P, 0.999)[0] == 1
    z = [0.0, 1.0]
    for bad in ((-1.0,), (np.nan,), (np.inf,), (1.0, -1), (1.0, 0, 0.0), (1.0, 0, 1.5), (1.0, 0, 1.0, -0.1),
                (1.0, 0, 1.0, 1.1), (1.0, 0, np.nan), (1.0, 0, 1.0, np.nan)):
        assert OD.filtered(z, *bad)[0] is None
    for z in ([np.nan, 0.0], [np.inf, 0.0], [-np.inf, -np.inf]):
        assert OD.filtered(z, 1.0)[0] is None
    assert OD.draw(None, 0.5)[0] == -1 and OD.draw(P, 1.0)[0] == -1 and OD.draw(P, -0.1)[0] == -1
