"""The operators refuse outputs and workspaces that lie over their inputs or
over each other before anything is enqueued (CPU only: every call here is
refused)."""

import pytest

from tests.test_ops_abi import EINVAL, FAR, FUSED, FUSED_OK, caller, lib  # noqa: F401

DIAG = dict(ap=FAR[12], rm=FAR[13], sp=FAR[14], pa=FAR[15])
FUSED_IN = ("h", "s", "p", "dl", "tok", "n", "u", "uf")
FUSED_OUT = ("tl", "out", "ne", "ws", "ap", "rm", "sp", "pa")


@pytest.mark.parametrize("out", FUSED_OUT)
def test_verify_fp8_lm_head_outputs_over_inputs(lib, out):  # noqa: F811
    call = caller(lib.specv_verify_fp8_lm_head, FUSED, dict(FUSED_OK, **DIAG))
    for name in FUSED_IN:
        assert call(**{out: FUSED_OK[name]}) == EINVAL, name
    # the last bytes of the largest inputs: draft_logits [2][3][1000] bfloat16
    # ends 12000 bytes after its start, hidden [2][4][256] 2048 after its own
    assert call(**{out: FAR[3] + 12000 - 16}) == EINVAL
    assert call(**{out: FAR[0] + 2048 - 16}) == EINVAL


@pytest.mark.parametrize("i", range(1, len(FUSED_OUT)))
def test_verify_fp8_lm_head_outputs_over_each_other(lib, i):  # noqa: F811
    ok = dict(FUSED_OK, **DIAG)
    call = caller(lib.specv_verify_fp8_lm_head, FUSED, ok)
    for other in FUSED_OUT[:i]:
        assert call(**{FUSED_OUT[i]: ok[other]}) == EINVAL, other
