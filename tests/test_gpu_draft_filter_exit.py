"""Long rows that one wave finishes: few tokens pass min-p and together they hold
less than top-p asks for, so that the row ends by min-p's threshold alone (the
tolerances are those of test_gpu_draft_filter.py)."""

import pytest

torch = pytest.importorskip("torch")

import speculative_decoding_sampling_amd as S  # noqa: E402
from test_gpu_draft_filter import BF, DEV, F32, check, logits  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("V", [33000, 50001, 152064])
@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("n", [1, 20, 64])
def test_min_p_ends_a_row_whose_top_p_is_not_reached(V, dtype, n):
    # n tokens near the largest above a floor that holds 0.2 to 4 times the 1 % that
    # top-p drops
    R, p, mp = 48, 0.99, 0.3
    print(f"[filter] V={V} {dtype} n={n}", flush=True)
    z = logits(R, V, V + n, F32, 0.7, 0)
    floor = z.double().exp().sum(1)
    g = torch.Generator().manual_seed(n)
    top = 1 - torch.rand(R, n, generator=g, dtype=torch.float64)      # logits 0 to 1 below the largest
    top[:, 0] = 1.0
    share = 0.01 * 20.0 ** torch.linspace(-0.5, 0.5, R, dtype=torch.float64)
    mass = (top - 1).exp().sum(1)
    # floor = share (floor + e^m mass)
    m = (floor * (1 - share) / share / mass).log()
    at = torch.randperm(V, generator=g)[:n]
    z[:, at] = (m[:, None] + top - 1).float()
    z = z.to(dtype)
    u = torch.rand(R, generator=g)
    once = None
    for _ in range(5):
        probs, tok = S.filter_probs(z.to(DEV), 1.0, 0, p, mp, u=u.to(DEV))
        assert torch.equal(tok, S.sample_filtered(z.to(DEV), u.to(DEV), 1.0, 0, p, mp))
        assert once is None or torch.equal(once, probs)
        once = probs
    assert check(z, u, 1.0, 0, p, mp, probs, tok) <= 1
    kept = (probs > 0).sum(1).cpu()
    assert int(kept.max()) <= n and bool((kept[-10:] == kept[-10:].max()).all())
