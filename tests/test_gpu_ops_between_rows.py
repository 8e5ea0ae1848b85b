"""Outputs that lie between the rows of their inputs (GPU only): rows padded past
the vocabulary may hold them, the rows themselves may not."""

import pytest

torch = pytest.importorskip("torch")

import speculative_decoding_sampling_amd as S  # noqa: E402
from tests.test_gpu_ops_probs import BF, F32, make  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("V", [2000, 40000])
@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("side", ["target_probs", "draft_probs"])
def test_verify_probs_writes_into_the_padding(V, dtype, side):
    B, K, pad = 3, 2, 64
    w = {k: v.to(DEV).contiguous() for k, v in make(B, K, V, dtype, V).items()}
    want = S.verify_probs(**w)
    rows = w[side]
    wide = torch.zeros(*rows.shape[:2], V + pad, dtype=dtype, device=DEV)
    wide[..., :V] = rows
    words = wide.view(torch.int32)                      # the same memory as 4-byte words
    v4 = V * wide.element_size() // 4
    out = words[1, 1, v4:v4 + B * (K + 1)].view(B, K + 1)
    ne = words[2, 0, v4 + 8:v4 + 8 + B]
    for _ in range(2):
        got = S.verify_probs(**dict(w, **{side: wide[..., :V]}), out_tokens=out, n_emitted=ne)
        assert got["out_tokens"] is out
        assert torch.equal(out, want["out_tokens"]) and torch.equal(ne, want["n_emitted"])
    assert torch.equal(wide[..., :V], rows)
    # one word earlier its first element lies in a row
    bad = words[1, 1, v4 - 1:v4 - 1 + B * (K + 1)].view(B, K + 1)
    with pytest.raises(S.SpecVerifyError):
        S.verify_probs(**dict(w, **{side: wide[..., :V]}), out_tokens=bad)
