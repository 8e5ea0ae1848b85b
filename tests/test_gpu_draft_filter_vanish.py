"""Draws at u = 0 past tokens that count as nothing one by one but not together: a
weight of at most 1e-290 of the largest is not drawn, however many there are."""

import math

import pytest

torch = pytest.importorskip("torch")

import speculative_decoding_sampling_amd as S  # noqa: E402
from test_gpu_draft_filter import BF, DEV, F32, I32  # noqa: E402

pytestmark = pytest.mark.gpu

NOTHING = 1e-290


def first_with_weight(z, T):
    """Of each row the first id whose weight is above 1e-290, and how near the
    nearest weight is to that, in units of the exponent."""
    x = (z.double() - z.double().max(1, keepdim=True).values) / T
    return (x > math.log(NOTHING)).int().argmax(1).int(), (x - math.log(NOTHING)).abs().min()


@pytest.mark.parametrize("V", [300, 20001, 32768, 36000, 50001, 129279])
@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("f", [(0, 1.0, 0.0), (0, 0.9999, 0.0), (0, 0.3, 0.0), (200, 1.0, 0.0), (3000, 1.0, 0.0),
                               (1024, 0.9, 0.0), (20000, 1.0, 0.0), (0, 1.0, 0.5), (1 << 20, 1.0, 0.0)])
def test_many_tokens_of_no_weight_come_first(V, dtype, f):
    # x = -674 .. -668: weights of 1e-293 to 7e-291, thousands of them before the
    # first token that counts (x = 0, or -600 before it); top-k keeps their ties
    T = 0.125
    depth = torch.tensor([674.0, 671.0, 669.0, 668.0, 667.0, 668.0, 674.0])
    R = len(depth)
    z = (-depth * T)[:, None].expand(R, V).contiguous()
    z[:, V - 7] = 0.0
    z[5, V - 9] = -600 * T
    z[5, V - 5] = -600 * T
    z[6, ::2] = -math.inf
    z[6, V - 7] = 0.0
    z = z.to(dtype)                                    # (bfloat16: x in steps of 4)
    u = torch.zeros(R)
    u[3] = 2.0 ** -149                                 # the smallest that is not 0
    k, p, mp = f
    print(f"[filter] V={V} {dtype} k={k} p={p} mp={mp}", flush=True)
    want, near = first_with_weight(z, T)
    assert float(near) > 0.1
    want[3] = V - 7
    if p < 1.0 or mp > 0.0 or k == 1:
        want[:] = V - 7
    probs, tok = S.filter_probs(z.to(DEV), T, k, p, mp, u=u.to(DEV))
    assert torch.equal(tok, S.sample_filtered(z.to(DEV), u.to(DEV), T, k, p, mp))
    assert tok.cpu().tolist() == want.tolist()
    assert probs.argmax(1).cpu().tolist() == [V - 7] * R and bool((probs.sum(1) == 1).all())


def test_each_request_with_its_own_filters():
    V, T = 40000, 0.125
    k = torch.tensor([0, 0, 500, 0, 600], dtype=I32)
    p = torch.tensor([1.0, 0.999, 1.0, 1.0, 0.9])
    z = torch.full((5, V), -670 * T)
    z[:, 35000] = 0.0
    tok = S.sample_filtered(z.to(DEV), torch.zeros(5, device=DEV), T, k.to(DEV), p.to(DEV), 0.0)
    assert tok.cpu().tolist() == [35000] * 5
