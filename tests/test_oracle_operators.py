"""Pins of the fp64 reference of the operators around the verification (CPU)."""

from fractions import Fraction

import numpy as np
import pytest

import oracle as O
from oracle import operators as OP


def test_worked_example_from_probabilities():
    # nickwang.xyz, "算完三个 token 的全部概率": A accepted, C rejected, B drawn
    p = np.array([[[.5, .3, .2]] * 4])
    q = np.array([[[.6, .1, .3]] * 3])
    r = OP.verify_probs(p, q, np.array([[0, 2, 1]]), np.array([3]), np.array([[.7, .9, .2]]),
                        np.array([.2]))
    assert r["out_tokens"][0].tolist() == [0, 1, -1, -1] and r["n_emitted"][0] == 2
    assert r["path"][0] == O.PATH_REJECT and r["stop_pos"][0] == 1
    assert np.allclose(r["alpha"][0], [5 / 6, 2 / 3, 1.0], atol=1e-15)
    assert abs(r["residual_mass"][0] - 0.2) < 1e-15


def test_matches_the_logit_oracle_on_its_distributions():
    rng = np.random.default_rng(5)
    B, K, V = 24, 4, 50
    zt, zd = rng.normal(size=(B, K + 1, V)) * 2, rng.normal(size=(B, K, V)) * 2
    tok = rng.integers(0, V, (B, K))
    n = rng.integers(0, K + 1, B)
    u, uf = (rng.random(s).astype(np.float32) for s in ((B, K), B))
    dist = lambda z: np.stack([[O.processed_distribution(r, 1.0)[0] for r in b] for b in z])  # noqa: E731
    a = O.verify(zt, zd, tok, n, u, uf, 1.0, eos_id=7)
    b = OP.verify_probs(dist(zt), dist(zd), tok, n, u, uf, eos_id=7)
    for k in ("out_tokens", "n_emitted", "path", "stop_pos"):
        assert np.array_equal(a[k], b[k]), k
    assert np.allclose(a["residual_mass"], b["residual_mass"], atol=1e-14)


def test_lookup_drafts_preserve_the_target_distribution():
    # q one at x: accept with p(x), else draw from p without x: exactly p
    p = [Fraction(1, 2), Fraction(1, 3), Fraction(1, 6)]
    for x in range(3):
        res = [Fraction(0) if v == x else p[v] for v in range(3)]
        total = sum(res)
        out = [(p[x] if v == x else 0) + (1 - p[x]) * res[v] / total for v in range(3)]
        assert out == p
    pr = np.array([[[.5, .25, .25]] * 2])
    for u, uf, want in ((.4, .9, [0, 2]), (.6, .4, [1, -1]), (.6, .6, [2, -1])):
        r = OP.verify_probs(pr, None, np.array([[0]]), np.array([1]), np.array([[u]]),
                            np.array([uf]))
        assert r["out_tokens"][0].tolist() == want


def test_e4m3_values_and_rounding():
    v = OP.e4m3_values()
    assert v[0x7e] == 448 and v[1] == 2.0 ** -9 and v[0x38] == 1.0 and np.isnan(v[[0x7f, 0xff]]).all()
    codes = np.r_[0:0x7f, 0x80:0xff].astype(np.uint8)
    assert np.array_equal(OP.to_e4m3(v[codes]), codes)
    # ties go to the even fraction: 17 lies between 16 (0x58) and 18 (0x59)
    assert OP.to_e4m3(17.0) == 0x58 and OP.to_e4m3(19.0) == 0x5a
    torch = pytest.importorskip("torch")
    x = np.random.default_rng(3).normal(size=20000) * np.exp(np.random.default_rng(4).normal(size=20000) * 3)
    x = np.clip(x, -448, 448).astype(np.float32)
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(OP.to_e4m3(x), want)


@pytest.mark.parametrize("amax,byte", [(0.0, 127), (448.0, 127), (448.00003, 128), (224.0, 126),
                                       (1.75, 119), (1.7500001, 120), (2.0 ** -130, 1),
                                       (np.inf, 255), (np.nan, 255)])
def test_scale_byte(amax, byte):
    assert OP.scale_byte(amax) == byte
    if 0 < amax < np.inf and byte > 1:
        s = 2.0 ** (byte - 127)
        assert amax / s <= 448 and amax / (s / 2) > 448      # the smallest that fits


def test_quantize_round_trip_is_within_half_a_step():
    rng = np.random.default_rng(9)
    x = rng.normal(size=(5, 384)) * np.exp(rng.normal(size=(5, 384)))
    q, s = OP.quantize(x)
    sv = np.repeat(2.0 ** (s - 127.0), 128, 1)
    err = np.abs(OP.dequantize(q, s) - x)
    # half a step: 2^-4 of a normal value, 2^-10 scales in the subnormals
    assert np.all(err <= np.maximum(np.abs(x) * 2.0 ** -4, sv * 2.0 ** -10) * (1 + 1e-12))


def test_hidden_norm_by_hand():
    h, y, t = OP.hidden_norm([[3.0, 4.0]], [[1.0, 1.0]], np.ones(2), post_weight=np.array([1.0, 2.0]),
                             gate=np.array([[2.0, 1.0]]), scale=0.5, eps=1e-300)
    rms = np.sqrt(12.5)
    assert np.allclose(t, [[3 / rms, 4 / rms]]) and np.allclose(h, 1 + t)
    assert np.allclose((y * y).mean(), 1.0)
