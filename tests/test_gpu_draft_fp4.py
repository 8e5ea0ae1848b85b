"""The LM head on 4-bit floats on the GPU against the fp64 reference.

Quantising is exact arithmetic but for the one rounding to a code: codes must
be equal.  With small integers and scales in a narrow range every float32 sum
of the product is exact, so the logits must be equal too (bfloat16: the exact
sum rounded to nearest even).  On general inputs the float32 accumulation of D
products is off by at most D roundings, each at most 2 u of the sum of
magnitudes should the matrix core truncate (u = 2^-24): 2 D u sum |h w|.  The
mixed product, behind bfloat16 logits of 8-bit states only, drops of each 8
products it adds what lies below 2^-13 of the largest: at most 8 * 2^-13 of it,
2^-10 sum |h w| more.  Each result is then rounded, by half a step of the output
type.
"""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import speculative_decoding_sampling_amd as S  # noqa: E402
from oracle import draft as OD  # noqa: E402
from oracle import operators as OP  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32, E4, E8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn, torch.float8_e8m0fnu
E2 = torch.float4_e2m1fn_x2


def bytes_of(t):
    return t.view(torch.uint8).cpu().numpy()


def dev4(q, s):
    return torch.from_numpy(q).to(DEV).view(E2), torch.from_numpy(s).to(DEV).view(E8)


def dev8(q, s):
    return torch.from_numpy(q).to(DEV).view(E4), torch.from_numpy(s).to(DEV).view(E8)


def codes(R, D, lo, hi, seed):
    """Random codes and scales 2^lo .. 2^hi."""
    rng = np.random.default_rng(seed)
    return OD.pack_codes(rng.integers(0, 16, (R, D)).astype(np.uint8)), \
        rng.integers(127 + lo, 128 + hi, (R, D // 32)).astype(np.uint8)


def integers8(R, D, top, lo, hi, seed):
    """Small integers as e4m3 bytes and scales 2^lo .. 2^hi."""
    rng = np.random.default_rng(seed)
    q = OP.to_e4m3(rng.integers(-top, top + 1, (R, D)).astype(np.float64))
    q[q == 0x80] = 0
    return q, rng.integers(127 + lo, 128 + hi, (R, D // 128)).astype(np.uint8)


def states(kind, M, D, seed):
    """(values, device pair) of exactly held hidden states."""
    if kind == 4:
        q = codes(M, D, 0, 2, seed)
        return OD.dequantize4(*q), dev4(*q)
    q = integers8(M, D, 8, 0, 2, seed)
    return OP.dequantize(*q), dev8(*q)


@pytest.mark.parametrize("R,D,dtype", [(1, 32, F32), (3, 96, BF), (5, 4096, F32), (257, 224, BF),
                                       (2, 65536, BF), (1, 4064, F32)])
def test_quantize_codes_are_exact(R, D, dtype):
    rng = np.random.default_rng(R + D)
    x = rng.normal(size=(R, D)) * np.exp(3 * rng.normal(size=(R, 1))) * np.exp(rng.normal(size=(R, D)))
    x[0, :32] = 0
    x = torch.from_numpy(x).to(dtype)
    q, s = S.quantize_fp4(x.to(DEV))
    assert q.shape == (R, D // 2) and s.shape == (R, D // 32)
    wq, ws = OD.quantize4(x.double().numpy())
    assert np.array_equal(bytes_of(s), ws) and np.array_equal(bytes_of(q), wq)


def test_quantize_every_float_near_the_grid():
    v = OD.GRID4
    mid = (v[1:] + v[:-1]) / 2
    x = np.concatenate([v, mid, np.nextafter(mid.astype(np.float32), np.float32(0)),
                        np.nextafter(mid.astype(np.float32), np.float32(1e9))]).astype(np.float32)
    x = np.concatenate([x, -x])
    rows = []
    for i in range(0, len(x), 31):
        row = np.zeros(32, np.float32)
        part = x[i:i + 31]
        row[:len(part)] = part
        row[31] = 6.0                                   # the scale is one
        rows.append(row)
    x = np.stack(rows)
    for f in (1.0, 2.0 ** 20, 2.0 ** -100, 2.0 ** -126):
        q, s = S.quantize_fp4(torch.from_numpy(x * np.float32(f)).to(DEV))
        wq, ws = OD.quantize4((x * np.float32(f)).astype(np.float64))
        assert np.array_equal(bytes_of(s), ws) and np.array_equal(bytes_of(q), wq), f


def test_quantize_borders_of_the_scale_and_extremes():
    top = [6.0, np.nextafter(np.float32(6), np.float32(7)), 3.0, 3.4e38, 1e-38, 1e-45, 2.0 ** -124,
           2.0 ** -126, np.inf, np.nan, -np.inf, -6.5]
    x = np.zeros((len(top), 64), np.float32)
    for i, t in enumerate(top):
        x[i, 3], x[i, 40] = t, 1.0
    q, s = S.quantize_fp4(torch.from_numpy(x).to(DEV))
    wq, ws = OD.quantize4(x.astype(np.float64))
    assert np.array_equal(bytes_of(s), ws), (bytes_of(s)[:, 0], ws[:, 0])
    assert np.array_equal(bytes_of(q), wq)


SIZES = [
    # M, V, D: row tiles (1 .. past several blocks), vocabulary tails, odd runs
    (1, 1, 128), (1, 32, 256), (2, 33, 384), (5, 1000, 640), (6, 4097, 4096), (16, 300, 1152),
    (31, 257, 512), (32, 256, 512), (33, 255, 512), (64, 511, 1024), (65, 513, 896), (96, 1000, 128),
    (100, 2000, 1152), (127, 640, 512), (128, 640, 640), (129, 640, 768), (160, 999, 2048),
    (161, 777, 384), (320, 1025, 1024), (321, 640, 256), (577, 1300, 512), (1100, 520, 384),
]


@pytest.mark.parametrize("M,V,D", SIZES)
@pytest.mark.parametrize("kind", [4, 8])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_exact_on_integers(M, V, D, kind, dtype):
    print(f"[fp4] M={M} V={V} D={D} states={kind} {dtype}", flush=True)
    h, hd = states(kind, M, D, 1)
    w = codes(V, D, -2, 0, 2)
    got = S.fp4_lm_head(*hd, S.pack_fp4_lm_head(*dev4(*w)), dtype=dtype)
    want = h @ OD.dequantize4(*w).T
    # products are multiples of 2^-4 (4-bit: 0.25 * 2^-2) below 2^8: sums below 2^19 are exact
    assert np.abs(want).max() < 2.0 ** 18
    assert torch.equal(got.cpu(), torch.from_numpy(want).to(dtype)), \
        int((got.cpu() != torch.from_numpy(want).to(dtype)).sum())


@pytest.mark.parametrize("M,V,D", [(5, 2000, 4096), (40, 700, 1152), (130, 900, 2048), (330, 600, 4096),
                                   (3, 64, 65536), (70, 300, 16384)])
@pytest.mark.parametrize("kind", [4, 8])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_general_inputs_within_the_accumulation_bound(M, V, D, kind, dtype):
    print(f"[fp4] general M={M} V={V} D={D} states={kind} {dtype}", flush=True)
    rng = np.random.default_rng(M)
    x = rng.normal(size=(M, D)) * np.exp(rng.normal(size=(1, D)))
    hq = OD.quantize4(x) if kind == 4 else OP.quantize(x)
    h = OD.dequantize4(*hq) if kind == 4 else OP.dequantize(*hq)
    wq = OD.quantize4(rng.normal(size=(V, D)) * np.exp(rng.normal(size=(V, 1))) / np.sqrt(D))
    w = OD.dequantize4(*wq)
    got = S.fp4_lm_head(*(dev4 if kind == 4 else dev8)(*hq), S.pack_fp4_lm_head(*dev4(*wq)), dtype=dtype)
    want = h @ w.T
    mixed = kind == 8 and dtype == BF
    tol = (2 * D * 2.0 ** -24 + (2.0 ** -10 if mixed else 0)) * (np.abs(h) @ np.abs(w).T)
    err = np.abs(got.double().cpu().numpy() - want)
    bound = tol + torch.finfo(dtype).eps / 2 * (np.abs(want) + tol)
    assert np.all(err <= bound)
    print("  max error / bound %.2e, error / rms %.2e" % (np.max(err / bound),
                                                          np.sqrt((err ** 2).mean() / (want ** 2).mean())))


@pytest.mark.parametrize("kind", [4, 8])
def test_blocks_of_very_different_scales(kind):
    # one block of each row carries all of it, its scale alone decides the size
    M, V, D = 40, 96, 1152
    step = 32 if kind == 4 else 128
    nb = D // step
    h, hd = states(kind, M, D, 3)
    hq, hs = (bytes_of(t).copy() for t in hd)
    per = hq.shape[1] // nb
    for m in range(M):
        hq[m].reshape(nb, per)[np.arange(nb) != m % nb] = 0
        hs[m] = 127 + (m - 20) * 2
    wq, ws = codes(V, D, 0, 0, 4)
    ws[:] = 127 + (np.arange(V) % 41 - 20)[:, None]
    h = (OD.dequantize4 if kind == 4 else OP.dequantize)(hq, hs)
    want = h @ OD.dequantize4(wq, ws).T
    for rep in (1, 5):                                  # both row-tile families
        d = (dev4 if kind == 4 else dev8)(np.tile(hq, (rep, 1)), np.tile(hs, (rep, 1)))
        for dtype in (F32, BF):
            got = S.fp4_lm_head(*d, S.pack_fp4_lm_head(*dev4(wq, ws)), dtype=dtype)
            assert torch.equal(got.cpu(), torch.from_numpy(np.tile(want, (rep, 1))).to(dtype))


def test_each_block_has_its_own_scale():
    # one column at a time: the scale of its block, and no other, is applied
    D = 512
    wq, ws = codes(64, D, -20, 20, 5)
    w = OD.dequantize4(wq, ws)
    packed = S.pack_fp4_lm_head(*dev4(wq, ws))
    rng = np.random.default_rng(6)
    cols = np.concatenate([np.arange(0, D, 16), rng.integers(0, D, 64)])
    code = np.zeros((len(cols), D), np.uint8)
    code[np.arange(len(cols)), cols] = 2                # 1.0
    hs = rng.integers(107, 147, (len(cols), D // 32)).astype(np.uint8)
    hq = OD.pack_codes(code)
    got = S.fp4_lm_head(*dev4(hq, hs), packed, dtype=F32)
    assert np.array_equal(got.double().cpu().numpy(), OD.dequantize4(hq, hs) @ w.T)
    q8 = np.where(code == 2, OP.to_e4m3(1.0), 0).astype(np.uint8)
    s8 = rng.integers(107, 147, (len(cols), D // 128)).astype(np.uint8)
    for dtype in (F32, BF):
        got = S.fp4_lm_head(*dev8(q8, s8), packed, dtype=dtype)
        assert torch.equal(got.cpu(), torch.from_numpy(OP.dequantize(q8, s8) @ w.T).to(dtype))


@pytest.mark.parametrize("kind", [4, 8])
def test_large_products_that_cancel(kind):
    # +a -a with a small rest far below: float32 sums of exact products keep it
    D, V = 256, 33
    rng = np.random.default_rng(7)
    code = np.zeros((V, D), np.uint8)
    code[:, 0], code[:, 1] = 7, 15                      # 6, -6
    code[:, 40] = rng.integers(1, 8, V)
    ws = np.full((V, D // 32), 127, np.uint8)
    ws[:, 1] = 127 - 12
    wq = OD.pack_codes(code)
    if kind == 4:
        hc = np.zeros((2, D), np.uint8)
        hc[:, [0, 1, 40]] = 7
        hq, hs = OD.pack_codes(hc), np.full((2, D // 32), 127, np.uint8)
        h, d = OD.dequantize4(hq, hs), dev4(hq, hs)
    else:
        hq = np.zeros((2, D), np.uint8)
        hq[:, [0, 1, 40]] = OP.to_e4m3(448.0)
        hs = np.full((2, D // 128), 127, np.uint8)
        h, d = OP.dequantize(hq, hs), dev8(hq, hs)
    got = S.fp4_lm_head(*d, S.pack_fp4_lm_head(*dev4(wq, ws)), dtype=F32)
    assert np.array_equal(got.double().cpu().numpy(), h @ OD.dequantize4(wq, ws).T)


@pytest.mark.parametrize("M", [7, 200])
@pytest.mark.parametrize("kind", [4, 8])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_nan_stays_in_its_row_and_column(M, kind, dtype):
    V, D = 300, 512
    h, hd = states(kind, M, D, 5)
    hq, hs = (bytes_of(t).copy() for t in hd)
    wq, ws = codes(V, D, -2, 0, 6)
    want = S.fp4_lm_head(*hd, S.pack_fp4_lm_head(*dev4(wq, ws)), dtype=dtype).cpu()
    rows_bad, cols_bad = {4}, {9, 299}
    hs[4, 1] = ws[9, 15] = ws[299, 3] = 255
    wq[299, 48:64] = 0                                  # a NaN block as the quantiser writes it
    if kind == 8:
        hq[2, 77] = 0x7f
        rows_bad.add(2)
    else:
        hq[4, 16:32] = 0
    got = S.fp4_lm_head(*(dev4 if kind == 4 else dev8)(hq, hs), S.pack_fp4_lm_head(*dev4(wq, ws)),
                        dtype=dtype).cpu()
    rows = [m for m in range(M) if m not in rows_bad]
    cols = [v for v in range(V) if v not in cols_bad]
    for m in rows_bad:
        assert got[m].isnan().all()
    for v in cols_bad:
        assert got[:, v].isnan().all()
    assert torch.equal(got[rows][:, cols], want[rows][:, cols])


def test_pack_from_values_and_layout():
    rng = np.random.default_rng(8)
    V, D = 70, 640
    w = torch.from_numpy(rng.normal(size=(V, D))).to(BF).to(DEV)
    q, s = S.quantize_fp4(w)
    a, b = S.pack_fp4_lm_head(w), S.pack_fp4_lm_head(q, s)
    assert torch.equal(a.data, b.data) and (a.V, a.D) == (V, D)
    p, qn, sn = a.data.cpu().numpy(), bytes_of(q), bytes_of(s)
    pieces = p[:96 * D // 2].reshape(3, 10, 64, 16)
    for g, st, l in ((0, 0, 0), (1, 3, 40), (2, 9, 5), (2, 1, 6), (2, 1, 37)):
        v, k = 32 * g + l % 32, 64 * st + 32 * (l // 32)
        assert np.array_equal(pieces[g, st, l], qn[v, k // 2:k // 2 + 16] if v < V else np.zeros(16))
    words = p[96 * D // 2:].reshape(3, 3, 64, 4)
    assert words[1, 2, 2, 0] == sn[34, 16] and words[1, 2, 34, 1] == sn[34, 19]
    assert words[1, 2, 2, 2] == 127 and words[2, 0, 3, 2] == sn[67, 4] and words[2, 1, 35, 0] == sn[67, 9]
    assert (words[2, :, 6:32] == 127).all()


@pytest.mark.parametrize("M,V", [(6, 3000), (200, 3000), (6, 3001), (200, 3001)])
@pytest.mark.parametrize("kind", [4, 8])
def test_rows_around_the_logits_are_left(M, V, kind):
    D = 256
    _, h = states(kind, M, D, 9)
    packed = S.pack_fp4_lm_head(*dev4(*codes(V, D, -2, 0, 10)))
    for dtype in (BF, F32):
        big = torch.full((M + 2, V), 77.0, dtype=dtype, device=DEV)
        S.fp4_lm_head(*h, packed, dtype=dtype, logits=big[1:M + 1])
        assert (big[0] == 77).all() and (big[M + 1] == 77).all()
        assert torch.equal(big[1:M + 1], S.fp4_lm_head(*h, packed, dtype=dtype))


def test_logits_past_32_bits():
    # more than 2^31 logits: the rows at the end are those of a small call
    M, V, D = 560, 4000003, 128
    _, h = states(4, M, D, 12)
    wq, ws = dev4(*codes(4099, D, -2, 0, 11))
    n = (V + 4098) // 4099
    big = S.pack_fp4_lm_head(wq.view(torch.uint8).repeat(n, 1)[:V].contiguous().view(E2),
                             ws.view(torch.uint8).repeat(n, 1)[:V].contiguous().view(E8))
    out = S.fp4_lm_head(*h, big)
    ref = S.fp4_lm_head(*h, S.pack_fp4_lm_head(wq, ws))
    for m in (0, 300, M - 1):
        for v0 in (0, 4099 * 500, 4099 * 975):
            k = min(4099, V - v0)
            assert torch.equal(out[m, v0:v0 + k], ref[m, :k])


def test_streams_graphs_and_repeats():
    for M, kind in ((6, 8), (150, 4)):
        (_, a), (_, b) = states(kind, M, 640, 13), states(kind, M, 640, 14)
        packed = S.pack_fp4_lm_head(*dev4(*codes(2000, 640, -2, 0, 15)))
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


def test_python_refusals():
    (_, h4), (_, h8) = states(4, 4, 256, 1), states(8, 4, 256, 1)
    w = dev4(*codes(50, 256, 0, 0, 2))
    packed = S.pack_fp4_lm_head(*w)
    with pytest.raises(ValueError):
        S.quantize_fp4(torch.zeros(4, 200, device=DEV))
    with pytest.raises(TypeError):
        S.quantize_fp4(torch.zeros(4, 256, device=DEV, dtype=torch.float16))
    with pytest.raises(TypeError):
        S.fp4_lm_head(h4[0].view(torch.uint8), h4[1], packed)
    with pytest.raises(ValueError):
        S.fp4_lm_head(h4[0], h8[1], packed)
    with pytest.raises(ValueError):
        S.fp4_lm_head(h8[0], h4[1], packed)
    with pytest.raises(ValueError):
        S.fp4_lm_head(h4[0][:, :64].contiguous(), h4[1][:, :4].contiguous(), packed)
    with pytest.raises(TypeError):
        S.fp4_lm_head(*h4, w[0])
    with pytest.raises(TypeError):
        S.fp4_lm_head(*h4, packed, dtype=torch.float16)
    with pytest.raises(S.SpecVerifyError):
        S.fp4_lm_head(h4[0][:0], h4[1][:0], packed)
    with pytest.raises(S.SpecVerifyError):
        S.pack_fp4_lm_head(w[0][:, :48].contiguous(), w[1][:, :3].contiguous())     # D = 96
