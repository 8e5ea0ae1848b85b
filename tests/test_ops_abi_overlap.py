"""The operators refuse outputs and workspaces that lie over their inputs or
over each other before anything is enqueued (CPU only: every call here is
refused)."""

import pytest

from tests.test_ops_abi import (EINVAL, FAR, FUSED, FUSED_OK, PROBS, PROBS_OK, caller, lib)  # noqa: F401

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


PROBS_OUT = ("out", "ne", "ws", "ap", "rm", "sp", "pa")


@pytest.mark.parametrize("out", PROBS_OUT)
@pytest.mark.parametrize("t,stride", [("t", "tsb"), ("d", "dsb")])
def test_verify_probs_outputs_over_rows(lib, out, t, stride):  # noqa: F811
    call = caller(lib.specv_verify_probs, PROBS, dict(PROBS_OK, **DIAG))
    base, rows = PROBS_OK[t], 4 if t == "t" else 3
    row = 90000 * 4
    last = base + (PROBS_OK[stride] + (rows - 1) * 90000) * 4      # the last row of the last request
    for at in (base, base + row, last, last + row - 16, base - 16 if out == "ws" else base + 16):
        assert call(**{out: at}) == EINVAL, at - base
    # rows far apart: over the last of them, and over one that starts inside
    wide = {stride: 1 << 24, stride[:2] + "k": 1 << 20}
    last = base + ((1 << 24) + (rows - 1) * (1 << 20)) * 4
    for at in (base + (1 << 22), last, last + row - 16):
        assert call(**{out: at}, **wide) == EINVAL, at - base
    # one row for all positions or requests, and half types
    assert call(**{out: base + 4 * PROBS_OK[stride] + 64}, **{stride[:2] + "k": 0}) == EINVAL
    assert call(**{out: base + row - 16}, **{stride: 0}) == EINVAL
    assert call(**{out: base + 2 * (PROBS_OK[stride] + 90000) + 64}, dt=1) == EINVAL
