"""A row whose mass from the bracket up is below top-p's share of the total by less than
a step of the whole numbers that masses are summed in: it rounds to the share or above,
so that the bracket holds no threshold, which is not the same as all of it being kept.

The row is built so, from the kernels' own arithmetic: one token of weight 1 and one of
0.3 (`high` together), 4032 tokens a and 8064 tokens b below them that hold as much again
and a hair more (top-p is 1/2), the rest masked.  Which tokens a sample of the row shows
decides the bracket: all of a, and 128 of b, enough not to say on which side of the
threshold they lie.  Min-p ends just below b, so the bracket does too."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import speculative_decoding_sampling_amd as S  # noqa: E402
from test_gpu_draft_filter import DEV, F32  # noqa: E402

pytestmark = pytest.mark.gpu

V = 1000000
UNIT = 2.0 ** 42                                       # of the sums: 62 - ceil(log2 V)
SEGMENT, CHUNK, CHUNKS = 1024, 64, 128                 # tokens, and pieces of the sample


def table_exp(x, bits):
    """exp(x) by a table of 2^bits entries and a polynomial, of degree 3 for 512 entries
    and 4 for 64, as the kernels take it (the argument's remainder in one rounding)."""
    n = 2 ** bits
    step = np.float64(np.log(np.longdouble(2)) / n)
    k = np.rint(x * n / np.log(2.0))
    r = np.float64(np.longdouble(x) - np.longdouble(k) * np.longdouble(step))
    q = 1 / 6 + (r / 24 if bits == 6 else 0)
    q = 1 + r * (0.5 + r * q)
    t = np.float64(np.exp2(np.longdouble(k) / n))
    return np.float64(t + t * (r * q))


def row_of(seed):
    rng = np.random.default_rng(seed)
    # the second token: high takes .5 to .6 of a step above a whole number of them
    while True:
        z2 = np.float32(-1.2 + 0.1 * rng.random())
        high = 1 + table_exp(np.float64(z2), 6)
        part = high * UNIT % 1
        if 0.5 < part < 0.6:
            break
    rest = high + 2 * (1 - part) / 2 / UNIT            # p Z: half way from high to the whole number above
    za = np.float32(np.log(rest / 2 / 4032) - 1e-4)
    zb = np.float32(np.log(rest / 2 / 8064) - 1e-4)
    z = np.full(V, -np.inf, dtype=np.float32)
    z[[5000, 5001]] = 0.0, z2
    chunks = -(-(-(-V // 4)) // 16)
    seen = [c * chunks // CHUNKS * CHUNK for c in range(CHUNKS)]
    shown = rng.permutation(CHUNKS)
    for c in shown[:63]:
        z[seen[c]:seen[c] + CHUNK] = za
    for c in shown[63:65]:
        z[seen[c]:seen[c] + CHUNK] = zb
    free = sorted(set(range(10, V // SEGMENT)) - {at // SEGMENT for at in seen})
    for g in free[:31]:
        z[g * SEGMENT:g * SEGMENT + 256] = zb
    assert (z == za).sum() == 4032 and (z == zb).sum() == 128 + 31 * 256
    mass = (z == za).sum() * table_exp(np.float64(za), 9) + (z == zb).sum() * table_exp(np.float64(zb), 9)
    # and what is missing in ever smaller tokens, each alone in its segment
    g = 40
    while rest - mass > 1e-16:
        zt = np.nextafter(np.float32(np.log(rest - mass)), np.float32(-np.inf))
        z[free[g] * SEGMENT + 7] = zt
        mass += table_exp(np.float64(zt), 9)
        g += 1
    assert zb > np.log(rest - mass + 1e-12) and abs(rest - mass) < 2e-15
    return z, za, zb


@pytest.mark.parametrize("seed", range(8))
def test_a_bracket_that_starts_at_the_share_within_a_step(seed):
    z, za, zb = row_of(seed)
    min_p = float(np.float32(np.exp(np.float64(zb)) * (1 - 1e-5)))
    probs = S.filter_probs(torch.from_numpy(z)[None].to(DEV), 1.0, 0, 0.5, min_p, dtype=F32)[0].cpu().numpy()
    # a lies at the border, on either side of it; b below it by half of the mass
    kept = set(np.unique(z[probs > 0]).tolist())
    sure = {0.0, float(z[5001])}
    assert kept in (sure, sure | {float(za)}), (kept, za, zb)
