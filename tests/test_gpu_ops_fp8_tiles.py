"""The 8-bit LM head's tile products, its reads past the caches, extremes of
the scales and work on other streams, on the GPU.

The vocabularies are large enough that every product is chosen (small ones take
the product for few rows, whatever the rows).  Integers make every float32 sum
exact, so the logits must equal a float32 product of the same integers on the
GPU, rounded once; general inputs are held to the bounds of the 64-bit tests.
"""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import speculative_decoding_sampling_amd as S  # noqa: E402
from oracle import operators as OP  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32, E4, E8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn, torch.float8_e8m0fnu


def operands(R, D, top, lo, hi, seed):
    """8-bit integers up to ``top`` with scales 2^lo .. 2^hi, and their values."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    v = torch.randint(-top, top + 1, (R, D), generator=g, device=DEV).float()
    e = torch.randint(lo, hi + 1, (R, D // 128), generator=g, device=DEV)
    q, s = v.to(E4), (e + 127).to(torch.uint8).view(E8)
    return q, s, v * torch.exp2(e.float()).repeat_interleave(128, 1)


def run(M, V, D, dtype, seed=1, **kw):
    h, w = operands(M, D, 8, 0, 2, seed), operands(V, D, 4, -2, 0, seed + 1)
    packed = S.pack_fp8_lm_head(*w[:2])
    return h, w, packed, S.fp8_lm_head(*h[:2], packed, dtype=dtype, **kw)


# rows below, at and past every row block; one to sixteen runs, in whole scale
# words and not; vocabularies of whole and ragged tiles, odd and even
TILES = [
    (17, 151999, 128), (31, 40960, 640), (33, 33000, 384), (45, 100003, 128), (64, 33000, 896),
    (64, 60007, 128), (65, 33000, 896), (65, 100003, 256), (90, 20001, 384), (96, 20002, 1152),
    (97, 33000, 640), (97, 60007, 2048), (120, 100003, 256), (128, 40960, 896), (128, 20001, 384),
    (129, 40960, 640), (200, 20001, 128), (257, 20001, 1024), (257, 33000, 1152), (300, 40960, 256),
    (385, 60007, 384), (520, 20001, 1152),
    (65, 20001, 896), (33, 20001, 2944), (96, 20001, 1536), (50, 30720, 1536), (90, 20001, 4096),
    (130, 20001, 896), (65, 32000, 896), (33, 40003, 1536), (96, 32000, 2048), (50, 50000, 2944),
    (190, 30720, 1152), (250, 20001, 2048),
]


@pytest.mark.parametrize("M,V,D", TILES)
@pytest.mark.parametrize("dtype", [BF, F32])
def test_exact_on_integers(M, V, D, dtype):
    print(f"[fp8 tiles] M={M} V={V} D={D} {dtype}", flush=True)
    h, w, _, got = run(M, V, D, dtype, M + V)
    want = (h[2] @ w[2].T).to(dtype)
    assert torch.equal(got, want), int((got != want).sum())


@pytest.mark.parametrize("M", [1, 17, 33, 70, 100, 128])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_weights_larger_than_the_caches(M, dtype):
    # 287 MB of weights, read once: every product's loads past the caches
    V, D = 70001, 4096
    print(f"[fp8 tiles] M={M} V={V} D={D} {dtype}", flush=True)
    h, w, _, got = run(M, V, D, dtype, M)
    want = (h[2] @ w[2].T).to(dtype)
    assert torch.equal(got, want), int((got != want).sum())


@pytest.mark.parametrize("M,V,D", [(40, 33000, 4096), (90, 20001, 2048), (128, 33000, 1152),
                                   (300, 20000, 2048)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_general_inputs_within_the_accumulation_bound(M, V, D, dtype):
    print(f"[fp8 tiles] general M={M} V={V} D={D} {dtype}", flush=True)
    g = torch.Generator(device=DEV).manual_seed(M)
    rnd = lambda *n: torch.randn(*n, generator=g, device=DEV)  # noqa: E731
    h = S.quantize_fp8(rnd(M, D) * torch.exp(rnd(1, D)))
    w = S.quantize_fp8(rnd(V, D) * torch.exp(rnd(V, 1)) / D ** 0.5)
    got = S.fp8_lm_head(*h, S.pack_fp8_lm_head(*w), dtype=dtype)
    val = lambda q, s: q.float() * s.float().repeat_interleave(128, 1)  # noqa: E731
    a, b = val(*h).double(), val(*w).double()
    want, mag = a @ b.T, a.abs() @ b.abs().T
    tol = (2 * D * 2.0 ** -24 + (2.0 ** -10 if dtype == BF else 0)) * mag
    err = (got.double() - want).abs()
    assert bool((err <= tol + torch.finfo(dtype).eps / 2 * (want.abs() + tol)).all())


@pytest.mark.parametrize("M", [100, 300])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_nan_stays_in_its_row_and_column(M, dtype):
    V, D = 33000, 640
    h, w, _, want = run(M, V, D, dtype, 5)
    hb, hs, wb, ws = (t.view(torch.uint8).clone() for t in (*h[:2], *w[:2]))
    hb[2, 77], hs[70, 4], wb[9, 500], ws[V - 1, 3] = 0x7f, 255, 0xff, 255
    got = S.fp8_lm_head(hb.view(E4), hs.view(E8), S.pack_fp8_lm_head(wb.view(E4), ws.view(E8)),
                        dtype=dtype)
    bad = torch.zeros(M, V, dtype=torch.bool, device=DEV)
    bad[[2, 70]] = True
    bad[:, [9, V - 1]] = True
    assert torch.equal(got.isnan(), bad)
    assert torch.equal(got[~bad], want[~bad])


@pytest.mark.parametrize("M,V", [(5, 20008), (100, 33000), (100, 33001), (300, 20008)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_logits_anywhere_and_what_lies_around_them(M, V, dtype):
    D = 256
    h, w, packed, want = run(M, V, D, dtype, 9)
    for shift in (0, 1, 3, 4, 8):                       # values off a 16-byte border
        big = torch.full(((M + 2) * V + shift,), 77.0, dtype=dtype, device=DEV)
        view = big[V + shift:V + shift + M * V].view(M, V)
        assert S.fp8_lm_head(*h[:2], packed, dtype=dtype, logits=view) is view
        assert torch.equal(view, want)
        assert bool((big[:V + shift] == 77).all()) and bool((big[V + shift + M * V:] == 77).all())


@pytest.mark.parametrize("M,V", [(3, 100), (100, 33000)])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("side", ["hidden", "weight"])
def test_smallest_and_largest_scales(M, V, dtype, side):
    # one operand's scales at the ends of their range, the other's at one.
    # Values below 2^-126 may count as 0: 2^-126 a value of the other operand,
    # and results below it as well.
    D = 384
    h, w = operands(M, D, 8, 0, 0, 11), operands(V, D, 4, 0, 0, 12)
    packed = S.pack_fp8_lm_head(*w[:2])
    plain = h[2].double() @ w[2].double().T
    mag = (h[2] if side == "weight" else w[2]).abs().double().sum(1)
    mag = mag[:, None] if side == "weight" else mag[None, :]
    for byte in (0, 1, 2, 9, 10, 240):
        hs = torch.full((M, D // 128), byte if side == "hidden" else 127, dtype=torch.uint8, device=DEV)
        ws = torch.full((V, D // 128), byte if side == "weight" else 127, dtype=torch.uint8, device=DEV)
        packed = S.pack_fp8_lm_head(w[0], ws.view(E8))
        got = S.fp8_lm_head(h[0], hs.view(E8), packed, dtype=dtype).double()
        want = plain * 2.0 ** (byte - 127)
        slack = 2.0 ** -126 * (mag + 1)
        lim = want.abs() * torch.finfo(dtype).eps / 2 * 1.01 + slack
        assert bool(((got - want).abs() <= lim).all()), byte


def test_scales_cancel_across_operands():
    # huge times tiny: exact, no product leaves the float range
    M, V, D = 70, 33000, 256
    h, w = operands(M, D, 8, 0, 0, 13), operands(V, D, 4, 0, 0, 14)
    want = h[2] @ w[2].T
    for e in (100, -100):
        hs = torch.full((M, 2), 127 + e, dtype=torch.uint8, device=DEV).view(E8)
        ws = torch.full((V, 2), 127 - e, dtype=torch.uint8, device=DEV).view(E8)
        got = S.fp8_lm_head(h[0], hs, S.pack_fp8_lm_head(w[0], ws), dtype=F32)
        assert torch.equal(got, want)


@pytest.mark.parametrize("M", [6, 100])
def test_streams_graphs_and_repeats(M):
    V, D = 33000, 640
    h, w, packed, first = run(M, V, D, BF, 20)
    h2 = operands(M, D, 8, 0, 2, 23)
    second = S.fp8_lm_head(*h2[:2], packed)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(3):
        x = S.fp8_lm_head(*h[:2], packed, stream=s1)
        y = S.fp8_lm_head(*h2[:2], packed, stream=s2)
        torch.cuda.synchronize()
        assert torch.equal(x, first) and torch.equal(y, second)
    q, s = h[0].clone(), h[1].clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        res = S.fp8_lm_head(q, s, packed)
    for src, want in ((h2, second), (h, first), (h2, second), (h, first)):
        q.view(torch.uint8).copy_(src[0].view(torch.uint8))
        s.view(torch.uint8).copy_(src[1].view(torch.uint8))
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(res, want)
        assert torch.equal(S.fp8_lm_head(*h[:2], packed), first)


def test_outputs_on_another_stream_wait_for_their_memory():
    # The output's memory was a tensor that the current stream still reads when
    # the call on another stream is made.
    n, D = 4096, 4096
    x = torch.randn(64, D, device=DEV)
    want = S.quantize_fp8(x)
    slow = torch.randn(n, n, device=DEV)
    s1 = torch.cuda.Stream()
    for call in (lambda: S.quantize_fp8(x, stream=s1),
                 lambda: S.hidden_norm(x, x, slow[0], dtype=E4, stream=s1)):
        torch.cuda.synchronize()
        call()
        torch.cuda.synchronize()
        old = torch.full((64, D), 5, dtype=torch.uint8, device=DEV)
        torch.cuda.synchronize()
        for _ in range(20):
            y = slow @ slow
        kept = old.clone()                              # behind the products
        del old
        got = call()
        torch.cuda.synchronize()
        assert bool((kept == 5).all())
        del y, kept
    got = S.quantize_fp8(x, stream=s1)
    torch.cuda.synchronize()
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(got, want))


def test_tiny_eps():
    # 1 / sqrt(eps) of a subnormal eps is finite: a row of zeros stays zero
    z = torch.zeros(2, 512, device=DEV)
    one = torch.ones(512, device=DEV)
    for eps in (1e-6, 1e-37, 1e-39, 1e-44):
        r, y = S.hidden_norm(z, z, one, post_weight=one, eps=eps, dtype=F32)
        assert not r.any() and not y.any()
    v = torch.full((2, 512), 1e-21, device=DEV)         # squares of 1e-42 beside eps
    r, y = S.hidden_norm(v, z, one, eps=1e-41, dtype=F32)
    # eps and the squares lie on the subnormals' grid of 2^-149: each of the
    # three values is off by at most half of it
    want, half = 1e-21 / (1e-42 + 1e-41) ** 0.5, 2.0 ** -150
    assert bool(((y - want).abs() <= want * (2 * half / 1.1e-41 + 2.0 ** -20)).all())
