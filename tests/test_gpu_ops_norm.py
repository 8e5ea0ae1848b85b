"""The norms around a block on the GPU against the fp64 reference.

Error bound, u = 2^-24.  A row's factor f comes from a sum of D squares: each
thread adds at most 64 of them, a wave 6 levels, a workgroup 16 values, then a
division, an addition, a square root and a division: its relative error is at
most n u with n = (64 + 6 + 16) / 2 + 4 < 50.  t = f g w x adds 4 roundings
and r' = r + t one of r': |dr'| <= 55 u |t| + u |r'| =: e.  In y = w h f2 the
factor f2 has relative error 50 u + |e|_2 / |r'|_2, and three roundings follow:
|dy| <= |w f2| e + |y| (54 u + |e|_2 / |r'|_2).  Each result is then rounded
once more, by half a step of its type.
"""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import speculative_decoding_sampling_amd as S  # noqa: E402
from oracle import operators as OP  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32, E4 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
U = 2.0 ** -24
EPS = 1e-6


def make(M, D, xt, rt, wt, post, gate_rows, seed, big=1.0):
    g = torch.Generator().manual_seed(seed)
    ch = 1 + 20 * (torch.rand(D, generator=g) < 0.02).float()
    x = (torch.randn(M, D, generator=g) * ch * big).to(xt)
    r = (torch.randn(M, D, generator=g) * 3 * ch).to(rt)
    w = (1 + 0.3 * torch.randn(D, generator=g)).to(wt)
    pw = (1 + 0.3 * torch.randn(D, generator=g)).to(wt) if post else None
    gate = torch.sigmoid(torch.randn(gate_rows, D, generator=g)).to(wt) if gate_rows else None
    return x, r, w, pw, gate


def up(t):
    return None if t is None else t.to(DEV)


def half_step(t, v):
    return torch.finfo(t).eps / 2 * np.abs(v) + 1e-40


def check(x, r, w, pw, gate, scale, dtype, got, eps=EPS):
    d = lambda t: None if t is None else t.double().numpy()  # noqa: E731
    h, y, t = OP.hidden_norm(d(x), d(r), d(w), d(pw), d(gate), scale, eps)
    e = 55 * U * np.abs(t) + U * np.abs(h)
    hn = np.sqrt((h * h).sum(1, keepdims=True)) + 1e-300
    en = np.sqrt((e * e).sum(1, keepdims=True))
    f2 = 1 / np.sqrt((h * h).mean(1, keepdims=True) + eps)
    ey = np.abs(d(w) * f2) * e + np.abs(y) * (54 * U + en / hn) + 1e-40
    res = got[0].double().cpu().numpy()
    assert np.all(np.abs(res - h) <= e * 1.01 + half_step(r.dtype, h)), "residual"
    if dtype != E4:
        out = got[1].double().cpu().numpy()
        assert np.all(np.abs(out - y) <= ey * 1.01 + half_step(dtype, y)), "y"
        return
    M, D = y.shape
    q = got[1].view(torch.uint8).cpu().numpy()
    s = got[2].view(torch.uint8).cpu().numpy()
    amax = np.abs(y).reshape(M, -1, 128).max(-1)
    ea = ey.reshape(M, -1, 128).max(-1)
    lo, hi = OP.scale_byte(np.maximum(amax - ea, 0)), OP.scale_byte(amax + ea)
    assert np.all((s == lo) | (s == hi)), "scale"
    sv = np.repeat(2.0 ** (s - 127.0), 128, 1)
    # half a step: 2^-4 of a normal value, 2^-10 scales among the subnormals
    tol = np.maximum((np.abs(y) + ey) * 2.0 ** -4, sv * 2.0 ** -10) + ey * 1.01
    assert np.all(np.abs(OP.dequantize(q, s) - y) <= tol), "8 bits"


@pytest.mark.parametrize("M,D,xt,rt,wt,post,gate_rows,scale,dtype", [
    (1, 1, F32, F32, F32, True, 1, 1.0, F32),
    (1, 4096, BF, BF, BF, False, 0, 1.0, BF),
    (3, 7, BF, F32, F32, True, 3, 0.5, BF),
    (5, 100, BF, BF, F32, True, 1, -0.7, F32),
    (2, 127, F32, BF, BF, True, 2, 1.3, BF),
    (2, 128, BF, BF, BF, True, 2, 1.3, E4),
    (37, 2047, F32, F32, F32, True, 1, 0.5, F32),
    (6, 1152, F32, BF, BF, True, 3, 0.25, E4),
    (20, 4096, BF, F32, BF, True, 4, 0.25, E4),
    (4, 8192, BF, BF, F32, True, 1, 1.0, BF),
    (3, 8200, BF, BF, BF, False, 3, 1.0, BF),          # two groups a thread
    (2, 16384, F32, F32, F32, True, 0, 1.0, E4),
    (2, 16392, BF, F32, BF, True, 1, 1.0, F32),        # more: the residual read late
    (2, 33333, BF, BF, BF, True, 2, 1.0, BF),
    (2, 65536, F32, F32, BF, True, 1, 2.0, E4),        # the widest
    (300, 384, BF, BF, BF, True, 100, 1.0, E4),
])
def test_matches_the_reference(M, D, xt, rt, wt, post, gate_rows, scale, dtype):
    print(f"[norm] M={M} D={D} {xt} {rt} {wt} post={post} gate={gate_rows} -> {dtype}", flush=True)
    x, r, w, pw, gate = make(M, D, xt, rt, wt, post, gate_rows, seed=M + D)
    got = S.hidden_norm(up(x), up(r), up(w), post_weight=up(pw), gate=up(gate), scale=scale, eps=EPS,
                        dtype=dtype)
    assert got[0].dtype == rt and got[1].dtype == dtype
    check(x, r, w, pw, gate, scale, dtype, got)


def test_zero_rows_large_and_small_values():
    for f in (0.0, 1e-15, 1e12):
        x, r, w, pw, gate = make(4, 256, F32, F32, F32, True, 1, 5)
        x, r = x * f, r * f
        got = S.hidden_norm(up(x), up(r), up(w), post_weight=up(pw), gate=up(gate))
        check(x, r, w, pw, gate, 1.0, BF, got)
    z = torch.zeros(2, 256, device=DEV)
    h, q, s = S.hidden_norm(z, z, torch.ones(256, device=DEV), dtype=E4)
    assert not q.view(torch.uint8).any() and (s.view(torch.uint8) == 127).all() and not h.any()


def test_in_place_and_unaligned():
    x, r, w, pw, gate = make(6, 512, BF, BF, BF, True, 2, 6)
    ra, xa = up(r), up(x)
    got = S.hidden_norm(xa, ra, up(w), post_weight=up(pw), gate=up(gate), residual_out=ra, out=xa)
    assert got[0] is ra and got[1] is xa
    check(x, r, w, pw, gate, 1.0, BF, got)
    # arrays that start off 16 bytes: element loads, the same values
    off = lambda t: torch.cat([t.flatten()[:1], t.flatten()]).to(DEV)[1:].view(t.shape)  # noqa: E731
    b = S.hidden_norm(off(x), off(r), off(w), post_weight=off(pw), gate=off(gate))
    assert torch.equal(got[0], b[0]) and torch.equal(got[1], b[1])
    q1 = S.hidden_norm(up(x), up(r), up(w), post_weight=up(pw), gate=up(gate), dtype=E4)
    q2 = S.hidden_norm(off(x), off(r), off(w), post_weight=off(pw), gate=off(gate), dtype=E4)
    for a, c in zip(q1, q2):
        assert torch.equal(a.view(torch.uint8), c.view(torch.uint8))


def test_bad_values_stay_in_their_row():
    x, r, w, pw, gate = make(8, 384, BF, F32, BF, True, 0, 7)
    good = S.hidden_norm(up(x), up(r), up(w), post_weight=up(pw), dtype=E4)
    x[2, 5], r[4, 300], r[6, 0] = float("nan"), float("inf"), float("nan")
    got = S.hidden_norm(up(x), up(r), up(w), post_weight=up(pw), dtype=E4)
    q, s = got[1].view(torch.uint8).cpu(), got[2].view(torch.uint8).cpu()
    for row, run in ((2, 0), (4, 2), (6, 0)):
        assert s[row, run] == 255 and (q[row, 128 * run:128 * run + 128] == 0x7f).all()
    ok = [0, 1, 3, 5, 7]
    assert torch.equal(q[ok], good[1].view(torch.uint8).cpu()[ok])
    y = S.hidden_norm(up(x), up(r), up(w), post_weight=up(pw))[1].cpu()
    assert y[2, 5].isnan() and y[4, 300].isnan() and y[6].isnan().all() and not y[ok].isnan().any()


def test_rows_around_the_outputs_are_left():
    x, r, w, pw, gate = make(3, 256, BF, BF, BF, True, 0, 8)
    ro = torch.full((5, 256), 9.0, dtype=BF, device=DEV)
    q = torch.zeros(5, 256, dtype=torch.uint8, device=DEV) + 3
    s = torch.zeros(5, 2, dtype=torch.uint8, device=DEV) + 5
    S.hidden_norm(up(x), up(r), up(w), post_weight=up(pw), dtype=E4, residual_out=ro[1:4],
                  out=q.view(E4)[1:4], out_scale=s.view(torch.float8_e8m0fnu)[1:4])
    for t, v in ((ro, 9), (q, 3), (s, 5)):
        assert (t[0] == v).all() and (t[4] == v).all()


def test_streams_graphs_and_shapes():
    x, r, w, pw, gate = make(12, 640, BF, F32, F32, True, 4, 9)
    a = dict(post_weight=up(pw), gate=up(gate), scale=0.3, dtype=E4)
    want = S.hidden_norm(up(x), up(r), up(w), **a)
    s1 = torch.cuda.Stream()
    xs, rs, ws = up(x).view(4, 3, 640), up(r).view(4, 3, 640), up(w)
    torch.cuda.synchronize()
    got = S.hidden_norm(xs, rs, ws, stream=s1, **a)
    s1.synchronize()
    assert got[1].shape == (4, 3, 640) and got[2].shape == (4, 3, 5)
    for p, q in zip(want, got):
        assert torch.equal(p.view(torch.uint8).flatten(), q.view(torch.uint8).flatten())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        res = S.hidden_norm(xs, rs, ws, **a)
    for k in range(4):
        if k % 2:
            xs.neg_()
            rs.neg_()                               # odd: negative values, the same magnitudes
        g.replay()
        torch.cuda.synchronize()
        eager = S.hidden_norm(xs, rs, ws, **a)
        for p, q in zip(res, eager):
            assert torch.equal(p.view(torch.uint8), q.view(torch.uint8))


def test_python_refusals():
    x = torch.zeros(4, 200, device=DEV)
    w = torch.ones(200, device=DEV)
    with pytest.raises(ValueError):
        S.hidden_norm(x, x, w, dtype=E4)                       # D not a multiple of 128
    with pytest.raises(ValueError):
        S.hidden_norm(x, x[:2], w)
    with pytest.raises(ValueError):
        S.hidden_norm(x, x, w, gate=torch.ones(3, 200, device=DEV))
    with pytest.raises(TypeError):
        S.hidden_norm(x.half(), x, w)
    with pytest.raises(TypeError):
        S.hidden_norm(x, x, w, gate=torch.ones(200, device=DEV, dtype=BF))
    with pytest.raises(TypeError):
        S.hidden_norm(x, x, w, dtype=torch.float16)
    with pytest.raises(ValueError):
        S.hidden_norm(x.T, x.T, torch.ones(4, device=DEV))     # not contiguous
    for kw in (dict(eps=0.0), dict(scale=float("inf")), dict(out=x)):
        with pytest.raises((S.SpecVerifyError, TypeError)):
            S.hidden_norm(x, x, w, **kw)
    with pytest.raises(S.SpecVerifyError):
        S.hidden_norm(x[:0], x[:0], w)                         # no rows
