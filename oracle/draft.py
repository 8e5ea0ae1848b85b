"""fp64 reference of the operators of a draft step.

TEST INFRASTRUCTURE ONLY: plain numpy in float64, written from the operators'
definitions, one row at a time where that is the plainest form.

* ``quantize4`` / ``dequantize4``: e2m1 codes with one power-of-two scale for each
  block of 32.
* ``filtered``: a row's distribution after temperature, top-k, top-p and min-p,
  with how near its decisions are to the border.
"""

import numpy as np

from .specverify_oracle import icdf, processed_distribution

BLOCK4 = 32
GRID4 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def e2m1_values():
    """Value of every e2m1 code, sign in bit 3."""
    return np.concatenate([GRID4, -GRID4])


def to_e2m1(x):
    """Codes of the nearest e2m1 value, ties to the even code, for |x| <= 6."""
    x = np.asarray(x, dtype=np.float64)
    a = np.abs(x)
    hi = np.clip(np.searchsorted(GRID4, a), 1, 7)
    lo = hi - 1
    dl, dh = a - GRID4[lo], GRID4[hi] - a
    code = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi).astype(np.uint8)
    return code | (np.signbit(x).astype(np.uint8) << 3)


def pack_codes(code):
    """Two codes to a byte, the first in the low half: [R, D] -> [R, D / 2]."""
    return code[:, 0::2] | (code[:, 1::2] << 4)


def unpack_codes(q):
    out = np.empty((q.shape[0], 2 * q.shape[1]), dtype=np.uint8)
    out[:, 0::2], out[:, 1::2] = q & 15, q >> 4
    return out


def scale4_byte(amax):
    """e8m0 byte of the smallest power of two, at least 2^-126, that brings
    ``amax`` to at most 6; 127 for 0, 255 where it is not finite."""
    amax = np.asarray(amax, dtype=np.float64)
    m, e = np.frexp(amax)                              # amax = m 2^e, m in [0.5, 1)
    byte = np.clip(np.where(m <= 0.75, e - 3, e - 2) + 127, 1, 254)
    byte = np.where(amax == 0, 127, byte)
    return np.where(np.isfinite(amax), byte, 255).astype(np.uint8)


def quantize4(x):
    """Packed codes [R, D / 2] and scale bytes [R, D / 32] of [R, D] values; a
    block with a NaN or an infinity is zero codes with scale byte 255."""
    x = np.asarray(x, dtype=np.float64)
    R, D = x.shape
    v = x.reshape(R, D // BLOCK4, BLOCK4)
    s = scale4_byte(np.abs(v).max(-1))
    bad = s == 255
    with np.errstate(invalid="ignore"):
        q = to_e2m1(np.where(bad[..., None], 0.0, v) * 2.0 ** (127.0 - s)[..., None])
    return pack_codes(q.reshape(R, D)), s


def dequantize4(q, s):
    c = unpack_codes(q)
    R, D = c.shape
    sv = np.where(s == 255, np.nan, 2.0 ** (s.astype(np.float64) - 127))
    return (e2m1_values()[c].reshape(R, D // BLOCK4, BLOCK4) * sv[..., None]).reshape(R, D)


def filtered(z, temperature, top_k=0, top_p=1.0, min_p=0.0):
    """(P, margin) of a row of finite or -inf logits: its distribution and the
    distance of its nearest top-p or min-p decision from the other outcome.  P
    is None for a parameter out of range or a row that has no distribution.
    Parameters are taken as the float32 values that a call holds."""
    z = np.asarray(z, dtype=np.float64)
    temperature, top_p, min_p = (float(np.float32(x)) for x in (temperature, top_p, min_p))
    if not (0 <= temperature < np.inf and top_k >= 0 and 0 < top_p <= 1 and 0 <= min_p <= 1):
        return None, np.inf
    if np.any(np.isnan(z)) or np.any(z == np.inf) or not np.any(z > -np.inf):
        return None, np.inf
    if temperature == 0:
        P = np.zeros(len(z))
        P[int(np.argmax(z))] = 1.0                     # the first of equal ones
        return P, np.inf
    P, info = processed_distribution(z, temperature, top_k, top_p)
    margin = np.inf
    if top_p < 1:
        # equal logits go together: what lies above the threshold, and at or above
        Q, _ = processed_distribution(z, temperature, top_k)
        above, reached = Q[z > info["tau_p"]].sum(), Q[z >= info["tau_p"]].sum()
        margin = min(top_p - above, reached - top_p)
    if min_p > 0:
        with np.errstate(over="ignore"):
            w = np.exp((z - z.max()) / temperature)
        other = w < 1                                  # the largest is always kept
        if other.any():
            margin = min(margin, np.abs(w[other] - min_p).min())
        P = np.where(w >= min_p, P, 0.0)
        P = P / P.sum()
    return P, float(margin)


def draw(P, u):
    """(token, margin) of a distribution, -1 for none or u outside [0, 1)."""
    if P is None or not 0.0 <= u < 1.0:
        return -1, np.inf
    return icdf(P, float(u))
