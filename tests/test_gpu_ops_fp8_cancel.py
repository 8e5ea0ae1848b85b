"""Logits that cancel, on the GPU: large products of both signs beside small ones.

Float32 logits hold their contract to the last bit: every product here is an
integer and every sum of them below 2^24, so float32 accumulation is exact.
bfloat16 logits take the 8-bit product, which of each 8 products it adds at
once drops of each what lies below 2^-13 of the largest: 8 * 2^-13 of that
product at most, and so 2^-10 sum |h w| in all, before the rounding to half a
bfloat16 step.  That, and not half a step of the logit, is what the header
promises; float32 accumulation adds nothing, its sums being exact.
"""

import pytest

torch = pytest.importorskip("torch")

import speculative_decoding_sampling_amd as S  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32, E4, E8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn, torch.float8_e8m0fnu


def operands(M, V, D, seed):
    """Integers whose large entries (256 a side) come in pairs that cancel."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    h = torch.randint(1, 5, (M, D), generator=g, device=DEV).float()
    w = torch.randint(-4, 5, (V, D), generator=g, device=DEV).float()
    big = torch.randperm(D // 2, generator=g, device=DEV)[:32] * 2
    sign = torch.randint(0, 2, (V, 32), generator=g, device=DEV).float() * 2 - 1
    h[:, big] = h[:, big + 1] = 256.0
    w[:, big], w[:, big + 1] = 256.0 * sign, -256.0 * sign
    one = lambda t: torch.full((len(t), D // 128), 127, dtype=torch.uint8, device=DEV).view(E8)  # noqa: E731
    return h, w, (h.to(E4), one(h)), (w.to(E4), one(w))


@pytest.mark.parametrize("M,V,D", [(1, 1000, 128), (7, 3001, 640), (33, 33000, 896), (100, 33000, 1152),
                                   (128, 40960, 4096), (300, 20001, 2048)])
def test_logits_that_cancel(M, V, D):
    print(f"[fp8 cancel] M={M} V={V} D={D}", flush=True)
    h, w, hq, wq = operands(M, V, D, M + V)
    # 64 products of 2^16 and D of at most 16: every partial sum is below 2^24
    assert 64 * 2 ** 16 + 16 * D < 2 ** 24
    want, mag = h.double() @ w.double().T, h.double() @ w.abs().double().T
    packed = S.pack_fp8_lm_head(*wq)
    assert torch.equal(S.fp8_lm_head(*hq, packed, dtype=F32).double(), want)
    err = (S.fp8_lm_head(*hq, packed).double() - want).abs()
    tol = 2.0 ** -10 * mag
    assert bool((err <= tol + 2.0 ** -8 * (want.abs() + tol)).all())
    print("  largest error %.1f of a bound of %.1f" % (err.max(), tol.max()), flush=True)
