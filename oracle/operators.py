"""fp64 reference of the operators around the verification step.

TEST INFRASTRUCTURE ONLY: plain numpy in float64, written from the operators'
definitions, one row or request at a time where that is the plainest form.

* ``verify_probs``: the verification from probabilities.  Same rule and readings
  as ``specverify_oracle.verify``; the accept test is decided on the products
  u q < p, which float64 holds exactly for float32 inputs.
* ``quantize`` / ``dequantize``: e4m3 values with one power-of-two scale for each
  run of 128.
* ``hidden_norm``: the norms around a block with its gate and residual scale.
"""

import numpy as np

from .specverify_oracle import (CDF_FLAG_REL, FLAG_CDF, FLAG_EMPTY_RESIDUAL, FLAG_NONE,
                                PATH_BONUS, PATH_EOS, PATH_ERROR, PATH_REJECT, icdf, residual)

BLOCK = 128
E4M3_MAX = 448.0


def _valid(a):
    return bool(np.all(np.isfinite(a)) and np.all(a >= 0))


def verify_probs(target, draft, draft_tokens, draft_len, u, u_final, eos_id=-1):
    """Verification of every request from target [B, K+1, V] and draft
    [B, K, V] probabilities (``draft`` None: one at the drafted token).  Values
    are widened exactly; the keys of the result are those of ``verify``."""
    target = np.asarray(target, dtype=np.float64)
    B, K1, V = target.shape
    K = K1 - 1
    res = {
        "out_tokens": np.full((B, K + 1), -1, dtype=np.int32),
        "n_emitted": np.full(B, -1, dtype=np.int32),
        "alpha": np.full((B, K), np.nan),
        "residual_mass": np.zeros(B),
        "stop_pos": np.full(B, -1, dtype=np.int32),
        "path": np.full(B, PATH_ERROR, dtype=np.int32),
        "flag_kind": np.zeros(B, dtype=np.int32),
        "flag_pos": np.full(B, -1, dtype=np.int32),
        "evaluated": np.ones(B, dtype=bool),
    }
    for b in range(B):
        _one(res, b, target, draft, draft_tokens, draft_len, u, u_final, eos_id, K, V)
    return res


def _draft_row(draft, b, k, x, V):
    if draft is not None:
        return np.asarray(draft[b, k], dtype=np.float64)
    q = np.zeros(V)
    q[x] = 1.0
    return q


def _one(res, b, target, draft, draft_tokens, draft_len, u, u_final, eos_id, K, V):
    n, uf = int(draft_len[b]), float(u_final[b])
    if not 0 <= n <= K or not 0.0 <= uf < 1.0:
        return
    alphas, accepts = [], []
    for k in range(n):
        x, uk = int(draft_tokens[b, k]), float(u[b, k])
        if not 0 <= x < V or not 0.0 <= uk < 1.0:
            return
        p, q = target[b, k, x], _draft_row(draft, b, k, x, V)[x]
        if not _valid(p) or not _valid(q) or not q > 0.0:
            return
        alphas.append(min(1.0, p / q))
        accepts.append(uk * q < p)
    out = np.full(K + 1, -1, dtype=np.int32)
    stop, path = n, PATH_BONUS
    for k in range(n):
        if not accepts[k]:
            stop, path = k, PATH_REJECT
            break
        out[k] = draft_tokens[b, k]
        if out[k] == eos_id:
            stop, path = k, PATH_EOS
            break
    mass, flag = 0.0, FLAG_NONE
    if path != PATH_EOS:
        w = P = target[b, stop]
        if not _valid(P):
            return
        if path == PATH_REJECT:
            Q = _draft_row(draft, b, stop, int(draft_tokens[b, stop]), V)
            if not _valid(Q):
                return
            w = residual(P, Q)
            mass = float(w.sum())
            if mass == 0.0:
                w, flag = P, FLAG_EMPTY_RESIDUAL
        if not w.sum() > 0.0:
            return
        out[stop], margin = icdf(w, uf)
        if flag == FLAG_NONE and margin < CDF_FLAG_REL:
            flag = FLAG_CDF
    res["alpha"][b, :n] = alphas
    res["out_tokens"][b] = out
    res["n_emitted"][b] = stop + 1
    res["residual_mass"][b] = mass
    res["stop_pos"][b] = stop
    res["path"][b] = path
    res["flag_kind"][b] = flag
    if flag != FLAG_NONE:
        res["flag_pos"][b] = stop


def e4m3_values():
    """Value of every e4m3 byte (4 exponent bits of bias 7, 3 fraction bits,
    no infinities, NaN at 0x7f and 0xff)."""
    out = np.empty(256)
    for c in range(256):
        e, f = (c >> 3) & 15, c & 7
        v = f * 2.0 ** -9 if e == 0 else (1 + f / 8) * 2.0 ** (e - 7)
        out[c] = np.nan if c & 0x7f == 0x7f else (-v if c & 0x80 else v)
    return out


def to_e4m3(x):
    """Bytes of the nearest e4m3 value, ties to the even fraction, for finite
    |x| at most 448 (larger magnitudes are not needed)."""
    x = np.asarray(x, dtype=np.float64)
    grid = e4m3_values()[:0x7f]                       # 0 .. 448, ascending
    a = np.abs(x)
    hi = np.clip(np.searchsorted(grid, a), 1, 126)
    lo = hi - 1
    dl, dh = a - grid[lo], grid[hi] - a
    code = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi).astype(np.uint8)
    return code | (np.signbit(x).astype(np.uint8) << 7)


def scale_byte(amax):
    """e8m0 byte of the scale of runs whose largest magnitude is ``amax``."""
    amax = np.asarray(amax, dtype=np.float64)
    m, e = np.frexp(amax)                              # amax = m 2^e, m in [0.5, 1)
    e = np.where(m <= E4M3_MAX / 512, e - 9, e - 8)
    byte = np.clip(e + 127, 1, 254)
    byte = np.where(amax == 0, 127, byte)
    return np.where(np.isfinite(amax), byte, 255).astype(np.uint8)


def quantize(x):
    """Bytes [R, D] and scale bytes [R, D / 128] of [R, D] values; a run with a
    NaN or an infinity is NaN bytes with scale byte 255."""
    x = np.asarray(x, dtype=np.float64)
    R, D = x.shape
    v = x.reshape(R, D // BLOCK, BLOCK)
    s = scale_byte(np.abs(v).max(-1))
    bad = s == 255
    with np.errstate(invalid="ignore"):
        q = to_e4m3(np.where(bad[..., None], 0.0, v) * 2.0 ** (127.0 - s)[..., None])
    q[bad] = 0x7f
    return q.reshape(R, D), s


def dequantize(q, s):
    R, D = q.shape
    sv = np.where(s == 255, np.nan, 2.0 ** (s.astype(np.float64) - 127))
    return (e4m3_values()[q].reshape(R, D // BLOCK, BLOCK) * sv[..., None]).reshape(R, D)


def hidden_norm(x, r, weight, post_weight=None, gate=None, scale=1.0, eps=1e-6):
    """(r', y, t) with r' = r + t, t = scale * gate * N(x; post_weight),
    y = N(r'; weight), all [M, D] float64; gate [G, D], G dividing M."""
    x, r = np.asarray(x, dtype=np.float64), np.asarray(r, dtype=np.float64)
    M, D = x.shape
    if post_weight is not None:
        x = post_weight * x / np.sqrt((x * x).mean(1, keepdims=True) + eps)
    if gate is not None:
        x = x * np.repeat(gate, M // len(gate), 0)
    t = scale * x
    h = r + t
    return h, weight * h / np.sqrt((h * h).mean(1, keepdims=True) + eps), t
