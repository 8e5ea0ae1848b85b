"""The operators' refusals of launches too large for the hardware and of
verifications whose outputs lie over their inputs, on the CPU: nothing is
enqueued."""

import pytest

from tests.test_ops_abi import (EINVAL, EUNSUPPORTED, FAR, NORM, NORM_OK, PROBS, PROBS_OK, caller,
                                lib)  # noqa: F401


@pytest.mark.parametrize("M,D", [(1 << 22, 8192), (1 << 23, 4096), (1 << 26, 8), (0x7fffffff, 1)])
def test_hidden_norm_of_too_many_rows(lib, M, D):  # noqa: F811
    # 2^32 threads: one workgroup a row
    call = caller(lib.specv_hidden_norm, NORM, NORM_OK)
    assert call(M=M, D=D, ot=1, gate=None) == EUNSUPPORTED
    # one fewer is a size; the null x is then what is wrong
    if M < 0x7fffffff:
        assert call(M=M - 1, D=D, ot=1, gate=None, x=None) == EINVAL


def test_quantize_and_pack_of_too_many_values(lib):  # noqa: F811
    q = lib.specv_fp8_quantize
    assert q(FAR[0], 1, 1 << 20, 32768, FAR[1], FAR[2], None) == EUNSUPPORTED
    assert q(None, 1, (1 << 20) - 1, 32768, FAR[1], FAR[2], None) == EINVAL
    n = lib.specv_fp8_lm_head_packed_weight_bytes
    assert n(4194304, 65536) == 0 and n(4194304, 8192) > 4194304 * 8192
    assert lib.specv_fp8_lm_head_pack_weight(FAR[0], FAR[1], FAR[2], 4194304, 65536, None) == EUNSUPPORTED


@pytest.mark.parametrize("B,V", [(1 << 22, 32768), (1 << 22, 1), (1 << 20, 16 * 1024 * 1024 // 4),
                                 (0x7fffffff, 40000)])
def test_verify_probs_of_too_many_requests(lib, B, V):  # noqa: F811
    assert caller(lib.specv_verify_probs, PROBS, PROBS_OK)(B=B, V=V) == EUNSUPPORTED
    assert lib.specv_verify_probs_workspace_bytes(B, 1, V) == 0


@pytest.mark.parametrize("kw", [
    dict(out="tok"), dict(out="n"), dict(out="u"), dict(out="uf"), dict(ne="n"), dict(ws="u"),
    dict(ap="u"), dict(ne="out"), dict(ws="out"), dict(sp="ne"), dict(pa="out"), dict(rm="uf"),
])
def test_verify_probs_outputs_over_inputs(lib, kw):  # noqa: F811
    over = {k: PROBS_OK[v] for k, v in kw.items()}
    assert caller(lib.specv_verify_probs, PROBS, PROBS_OK)(**over) == EINVAL
