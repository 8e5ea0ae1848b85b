"""Float32 probabilities are the value rounded once, bfloat16 ones those rounded again.

w = exp((z - m) / T) is good to 4e-14 (the exponential's truncation) and |x| 2^-51 (the
argument's roundings), below 1e-13 where a probability is a normal float32 (x > -104),
and so are their sum and, with two roundings of 2^-53, the quotient: 2e-13; the
reference's own argument is off by |z / T| 2^-52, below 2e-13 here.  Together below
2^-41 of the value; then half a step, 2^-24 of it or 2^-150 among subnormals."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import speculative_decoding_sampling_amd as S  # noqa: E402
from oracle import draft as OD  # noqa: E402
from test_gpu_draft_filter import BF, DEV, F32, logits  # noqa: E402

pytestmark = pytest.mark.gpu

FILTERS = [(1.0, 0, 1.0, 0.0), (0.7, 0, 1.0, 0.0), (0.25, 0, 1.0, 0.0), (1.3, 0, 0.95, 0.0), (0.9, 300, 1.0, 0.0),
           (0.8, 0, 1.0, 0.01), (1.1, 2000, 0.97, 0.001)]


@pytest.mark.parametrize("V", [5, 1000, 20001, 32768, 32769, 50001, 152064])
@pytest.mark.parametrize("dtype", [F32, BF])
def test_probabilities_are_rounded_once(V, dtype):
    R, worst = 3, 0.0
    for n, f in enumerate(FILTERS):
        print(f"[filter] V={V} {dtype} {f}", flush=True)
        z = logits(R, V, 7 * n + V, dtype)
        z[2, : V // 2] *= 8                            # down to x = -300 and lower
        probs = S.filter_probs(z.to(DEV), *f)
        assert torch.equal(S.filter_probs(z.to(DEV), *f, dtype=BF), probs.to(BF))
        for i in range(R):
            P, margin = OD.filtered(z[i].double().numpy(), *f)
            if margin < 1e-9:
                continue
            off = np.abs(probs[i].double().cpu().numpy() - P)
            assert np.all(off <= P * (2.0 ** -24 + 2.0 ** -41) + 2.0 ** -150), \
                (i, np.max((off - 2.0 ** -150) / np.maximum(P, 2.0 ** -126)) * 2.0 ** 24)
