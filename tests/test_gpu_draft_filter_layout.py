"""Outputs whose rows lie between others: strides that are not nested, and one buffer
that holds logits and probabilities of many requests in turn."""

import pytest

torch = pytest.importorskip("torch")

import speculative_decoding_sampling_amd as S  # noqa: E402
from test_gpu_draft_filter import DEV, F32, I32, check, logits  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("V", [1001, 33000])
def test_strides_that_are_not_nested(V):
    # rows of request b at (2 b + 3 l) V: 0, 3, 2, 5, 4, 7
    B, L = 3, 2
    z = logits(B * L, V, V)
    u = torch.rand(B * L, generator=torch.Generator().manual_seed(1))
    buf = torch.full((9 * V,), 7.0, device=DEV)
    tok = torch.full((9,), -7, dtype=I32, device=DEV)
    probs, out = buf.as_strided((B, L, V), (2 * V, 3 * V, 1)), tok.as_strided((B, L), (2, 3))
    f = (0.9, 40, 0.95, 0.0)
    S.filter_probs(z.view(B, L, V).to(DEV), *f, u=u.view(B, L).to(DEV), probs=probs, out_tokens=out)
    assert check(z, u, *f, probs.reshape(B * L, V), out.reshape(B * L)) <= 1
    for i in (1, 6, 8):
        assert bool((buf[i * V:(i + 1) * V] == 7).all()) and int(tok[i]) == -7


@pytest.mark.parametrize("B,L", [(300, 5), (2000, 1)])
def test_one_buffer_for_logits_and_probabilities(B, L):
    V = 600
    buf = torch.zeros(B, L, 2, V, device=DEV)
    z = logits(B * L, V, B)
    buf[:, :, 0] = z.view(B, L, V).to(DEV)
    u = torch.rand(B, L, generator=torch.Generator().manual_seed(B))
    f = (1.1, 0, 0.9, 0.02)
    probs, tok = S.filter_probs(buf[:, :, 0], *f, u=u.to(DEV), probs=buf[:, :, 1])
    assert torch.equal(buf[:, :, 0].cpu(), z.view(B, L, V))
    want = S.filter_probs(z.view(B, L, V).to(DEV), *f, u=u.to(DEV), dtype=F32)
    assert torch.equal(probs, want[0]) and torch.equal(tok, want[1])
    with pytest.raises(S.SpecVerifyError):
        S.filter_probs(buf[:, :, 0], *f, probs=buf.view(-1)[V - 1:V - 1 + B * L * 2 * V - V].as_strided(
            (B, L, V), (2 * L * V, 2 * V, 1)))
