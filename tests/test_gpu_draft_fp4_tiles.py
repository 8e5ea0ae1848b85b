"""The 4-bit LM head where its weights fill the card: every tile of up to 128
hidden rows, even and uneven row blocks, against the fp64 reference.

With small integers and scales in a narrow range every float32 sum is exact:
products are multiples of 2^-4 (4-bit states: 0.25 * 2^-2) and below 2^8, so sums
below 2^18 are whole multiples that a float32 holds, and the logits must be equal.
"""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import speculative_decoding_sampling_amd as S  # noqa: E402
from oracle import draft as OD  # noqa: E402
from test_gpu_draft_fp4 import BF, DEV, E2, E8, F32, codes, dev4, states  # noqa: E402

pytestmark = pytest.mark.gpu


def equal_to_the_reference(M, V, D, kind, dtype):
    h, hd = states(kind, M, D, M)
    w = codes(V, D, -2, 0, V)
    got = S.fp4_lm_head(*hd, S.pack_fp4_lm_head(*dev4(*w)), dtype=dtype).cpu()
    want = h @ OD.dequantize4(*w).T
    assert np.abs(want).max() < 2.0 ** 18
    assert torch.equal(got, torch.from_numpy(want).to(dtype)), \
        int((got != torch.from_numpy(want).to(dtype)).sum())


@pytest.mark.parametrize("M,V,D", [
    # one to four 32-row steps a tile and several row blocks, whole or short; runs of one step to many
    (33, 40001, 128), (64, 24576, 256), (65, 24577, 384), (97, 20001, 640), (128, 20008, 1152),
    (129, 20001, 128), (160, 16640, 896), (200, 20001, 512), (257, 20001, 256), (320, 20000, 384),
    (321, 16390, 640), (450, 16640, 128), (1, 131073, 128), (20, 65536, 384), (31, 70001, 256),
])
@pytest.mark.parametrize("kind", [4, 8])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_exact_on_integers(M, V, D, kind, dtype):
    print(f"[fp4] M={M} V={V} D={D} states={kind} {dtype}", flush=True)
    equal_to_the_reference(M, V, D, kind, dtype)


@pytest.mark.parametrize("kind", [4, 8])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_nan_stays_in_its_row_and_column(kind, dtype):
    M, V, D = 200, 20001, 512
    h, (q, s) = states(kind, M, D, 5)
    wq, ws = codes(V, D, -2, 0, 6)
    ws[777, 3] = 255
    s = s.view(torch.uint8).clone()
    s[131, -1] = 255
    got = S.fp4_lm_head(q, s.view(E8), S.pack_fp4_lm_head(*dev4(wq, ws)), dtype=dtype).cpu()
    nan = torch.zeros(M, V, dtype=torch.bool)
    nan[131] = True
    nan[:, 777] = True
    assert torch.equal(got.isnan(), nan)
    ws[777, 3] = 127
    want = torch.from_numpy(h @ OD.dequantize4(wq, ws).T).to(dtype)
    assert torch.equal(got[~nan], want[~nan])


@pytest.mark.parametrize("kind", [4, 8])
@pytest.mark.parametrize("M,V", [(5, 3000), (150, 20001)])
def test_scales_that_start_anywhere(kind, M, V):
    D = 640
    _, (q, s) = states(kind, M, D, 8)
    packed = S.pack_fp4_lm_head(*dev4(*codes(V, D, -2, 0, 7)))
    want = S.fp4_lm_head(q, s, packed)
    for shift in (1, 2, 3):
        room = torch.zeros(s.numel() + shift, dtype=torch.uint8, device=DEV)
        room[shift:] = s.view(torch.uint8).flatten()
        assert torch.equal(S.fp4_lm_head(q, room[shift:].view(s.shape).view(E8), packed), want)


@pytest.mark.parametrize("V", [20000, 20001])
def test_rows_around_the_logits_are_left(V):
    M, D = 150, 256
    _, h = states(4, M, D, 9)
    packed = S.pack_fp4_lm_head(*dev4(*codes(V, D, -2, 0, 10)))
    for dtype in (BF, F32):
        big = torch.full((M + 2, V), 77.0, dtype=dtype, device=DEV)
        S.fp4_lm_head(*h, packed, dtype=dtype, logits=big[1:M + 1])
        assert (big[0] == 77).all() and (big[M + 1] == 77).all()
        assert torch.equal(big[1:M + 1], S.fp4_lm_head(*h, packed, dtype=dtype))


@pytest.mark.parametrize("M", [1, 16, 40, 100, 128, 260])
def test_weights_larger_than_the_caches(M):
    # the rows of a repeated block of weights give the logits of a small call
    n, rep, D = 4096, 34, 4096
    V = n * rep - 31
    wq, ws = dev4(*codes(n, D, -2, 0, 21))
    big = S.pack_fp4_lm_head(wq.view(torch.uint8).repeat(rep, 1)[:V].contiguous().view(E2),
                             ws.view(torch.uint8).repeat(rep, 1)[:V].contiguous().view(E8))
    small = S.pack_fp4_lm_head(wq, ws)
    for kind in (4, 8):
        h, hd = states(kind, M, D, 22)
        want = torch.from_numpy(h @ OD.dequantize4(wq.view(torch.uint8).cpu().numpy(),
                                                   ws.view(torch.uint8).cpu().numpy()).T).to(BF)
        assert np.abs(want.float().numpy()).max() < 2.0 ** 18
        assert torch.equal(S.fp4_lm_head(*hd, small).cpu(), want)
        got = S.fp4_lm_head(*hd, big)
        want = want.to(DEV)
        for i in range(rep):
            k = min(n, V - n * i)
            assert torch.equal(got[:, n * i:n * i + k], want[:, :k]), (kind, i)


def test_streams_graphs_and_repeats():
    M, V, D = 150, 20001, 640
    (_, a), (_, b) = states(4, M, D, 13), states(4, M, D, 14)
    packed = S.pack_fp4_lm_head(*dev4(*codes(V, D, -2, 0, 15)))
    ra, rb = S.fp4_lm_head(*a, packed), S.fp4_lm_head(*b, packed)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        x, y = S.fp4_lm_head(*a, packed, stream=s1), S.fp4_lm_head(*b, packed, stream=s2)
        torch.cuda.synchronize()
        assert torch.equal(x, ra) and torch.equal(y, rb)
    st = [t.clone() for t in a]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        res = S.fp4_lm_head(*st, packed)
    for src, want in ((b, rb), (a, ra), (b, rb)):
        for t, v in zip(st, src):
            t.view(torch.uint8).copy_(v.view(torch.uint8))
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(res, want)
        assert torch.equal(S.fp4_lm_head(*a, packed), ra)
