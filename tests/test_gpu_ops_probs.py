"""Verification from probabilities on the GPU against the fp64 reference.

The accept test is exact on both sides and the draws sum in float64, so tokens
and counts must be equal except where the draw lies within 1e-10 of an edge of
its token's interval.  accept_prob is a float64 quotient rounded to float32
(half a step, 2^-24 of a value at most 1); a residual mass is a float64 sum of
at most 2^22 terms of total at most 1, in another order than the reference's:
2^22 * 2^-53 bounds both sides' error, 1e-9.
"""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import oracle as O  # noqa: E402
import speculative_decoding_sampling_amd as S  # noqa: E402
from oracle import operators as OP  # noqa: E402
from tests.parity import compare, to_numpy  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32


def make(B, K, V, dtype, seed, pad=0, onehot=False, ragged=False, sharp=2.0, kill=0.0):
    """Random probabilities; ``kill`` zeroes that share of both (a filter's)."""
    g = torch.Generator().manual_seed(seed)
    z = torch.randn(B, K + 1, V + pad, generator=g) * sharp
    zd = z[:, :K] + 0.7 * torch.randn(B, K, V + pad, generator=g)
    if kill:
        z = z.masked_fill(torch.rand(z.shape, generator=g) < kill, -1e9)
        zd = zd.masked_fill(torch.rand(zd.shape, generator=g) < kill, -1e9)
        z[..., 0], zd[..., 0] = 0.0, 0.0
    p = torch.zeros_like(z, dtype=dtype)
    q = torch.zeros_like(zd, dtype=dtype)
    p[..., :V] = torch.softmax(z[..., :V], -1).to(dtype)
    q[..., :V] = torch.softmax(zd[..., :V], -1).to(dtype)
    p[..., V:] = 7.0                                   # past the vocabulary: never read
    q[..., V:] = float("nan")
    tok = torch.empty(B, K, dtype=torch.int32)
    if K:
        e = torch.empty(B, K, V).exponential_(generator=g)
        tok = (q[..., :V].float() / e).argmax(-1).int()
    n = torch.randint(0, K + 1, (B,), generator=g, dtype=torch.int32) if ragged else \
        torch.full((B,), K, dtype=torch.int32)
    return dict(target_probs=p[..., :V], draft_probs=None if onehot else q[..., :V],
                draft_tokens=tok, draft_len=n, u=torch.rand(B, K, generator=g),
                u_final=torch.rand(B, generator=g))


def on_gpu(w):
    def up(t):
        if t is None:
            return None
        if t.is_contiguous() or t.dim() < 3:
            return t.to(DEV)
        base = torch.empty_strided(t.shape, t.stride(), dtype=t.dtype, device=DEV)
        return base.copy_(t)
    return {k: up(v) for k, v in w.items()}


def reference(w, eos):
    d = w["draft_probs"]
    r = OP.verify_probs(w["target_probs"].double().numpy(), None if d is None else d.double().numpy(),
                        w["draft_tokens"].numpy(), w["draft_len"].numpy(), w["u"].numpy(),
                        w["u_final"].numpy(), eos)
    B, K = w["draft_tokens"].shape
    r["topp_margin_rows"] = np.full((B, 2 * K + 1), np.inf)
    return r


def check(w, eos=-1, **kw):
    K = w["draft_tokens"].shape[1]
    got = S.verify_probs(**on_gpu(w), eos_id=eos, debug=True, **kw)
    torch.cuda.synchronize()
    got, ref = to_numpy(got), reference(w, eos)
    rep = compare(got, ref, K, alpha_tol=2.0 ** -24, mass_tol=1e-9)
    assert not rep["mismatches"], rep["mismatches"][:4]
    err = ref["n_emitted"] < 0
    assert np.all(got["accept_prob"][err] == -1) and np.all(got["residual_mass"][err] == 0)
    assert np.array_equal(got["path"], ref["path"])
    used = np.arange(K) < w["draft_len"].numpy()[:, None]
    assert np.all(got["accept_prob"][~used] == -1)
    return got, ref


@pytest.mark.parametrize("B,K,V,dtype,pad,onehot,ragged", [
    (1, 0, 1, F32, 0, False, False),            # one token
    (3, 1, 2, BF, 0, False, False),
    (9, 4, 63, F32, 0, False, True),            # inside one chunk
    (7, 3, 1024, BF, 0, False, True),           # exactly one chunk
    (7, 3, 1025, F32, 0, True, True),           # one past it
    (5, 4, 5000, BF, 1, False, True),           # odd stride: element loads
    (4, 64, 300, F32, 0, False, True),          # the most drafts
    (4, 64, 300, F32, 0, True, False),
    (6, 5, 32000, F32, 0, False, False),
    (2, 2, 32768, BF, 0, False, False),         # the largest one-kernel vocabulary
    (2, 2, 32769, BF, 0, False, False),         # the smallest two-kernel one
    (8, 4, 50001, F32, 3, False, True),
    (4, 4, 128256, F32, 0, False, True),
    (3, 8, 129279, BF, 1, True, True),
    (2, 1, 1 << 20, F32, 0, False, False),      # many record batches
])
def test_matches_the_reference(B, K, V, dtype, pad, onehot, ragged):
    print(f"[probs] B={B} K={K} V={V} {dtype} pad={pad} onehot={onehot}", flush=True)
    w = make(B, K, V, dtype, seed=V + K, pad=pad, onehot=onehot, ragged=ragged,
             sharp=2.0 if V < 10000 else 4.0)
    check(w, eos=1 if V > 1 and K else -1)


def test_every_path_is_met():
    w = make(400, 4, 200, F32, 11, ragged=True)
    w["draft_tokens"][::5, 1] = 3                # some accepted EOS
    got, ref = check(w, eos=3)
    assert set(ref["path"].tolist()) == {O.PATH_REJECT, O.PATH_BONUS, O.PATH_EOS}


def test_filtered_rows_with_zeros():
    check(make(64, 4, 3000, F32, 12, kill=0.98, ragged=True))
    check(make(64, 4, 40000, BF, 13, kill=0.999, ragged=True))


def test_largest_vocabulary():
    V = 4194304
    w = make(1, 1, V, BF, 14, sharp=6.0)
    for uf in (0.0, 0.5, 1 - 2.0 ** -24):
        w["u_final"][0] = uf
        check(w)


def test_draws_at_the_ends_and_on_edges():
    # dyadic weights: every sum is exact, so edges are exact ties
    V = 4096
    p = torch.zeros(6, 1, V)
    p[:, 0, [5, 1500, 4095]] = torch.tensor([0.25, 0.5, 0.25])
    for uf, y in ((0.0, 5), (0.25, 1500), (0.75, 4095), (0.2499999, 5), (1 - 2.0 ** -24, 4095)):
        r = S.verify_probs(p.to(DEV), None, torch.zeros(6, 0, dtype=torch.int32, device=DEV),
                           torch.zeros(6, dtype=torch.int32, device=DEV), torch.zeros(6, 0, device=DEV),
                           torch.full((6,), uf, device=DEV))
        assert (r["out_tokens"] == y).all(), (uf, r["out_tokens"])


def test_accept_ties_are_exact():
    # u q == p exactly rejects (strict), the next float below accepts
    p = torch.tensor([[[0.25, 0.75], [0.5, 0.5]]])
    q = torch.tensor([[[0.5, 0.5]]])
    u = torch.tensor([[0.5]])
    w = dict(target_probs=p, draft_probs=q, draft_tokens=torch.zeros(1, 1, dtype=torch.int32),
             draft_len=torch.ones(1, dtype=torch.int32), u=u, u_final=torch.tensor([0.1]))
    got, _ = check(w)
    assert got["path"][0] == O.PATH_REJECT and got["out_tokens"][0, 0] == 1
    w["u"] = torch.nextafter(u, torch.zeros(1))
    got, _ = check(w)
    assert got["path"][0] == O.PATH_BONUS and got["out_tokens"][0, 0] == 0


@pytest.mark.parametrize("V", [2000, 50000, 200000])
def test_empty_residual_redraws_from_p(V):
    # p below q everywhere (the rows sum to less than one): nothing to correct with
    p = torch.full((3, 2, V), 2.0 ** -12)
    q = torch.full((3, 1, V), 2.0 ** -11)
    w = dict(target_probs=p, draft_probs=q, draft_tokens=torch.full((3, 1), 7, dtype=torch.int32),
             draft_len=torch.ones(3, dtype=torch.int32), u=torch.full((3, 1), 0.9),
             u_final=torch.tensor([0.0, 0.5, 0.99]))
    got = to_numpy(S.verify_probs(**on_gpu(w), debug=True))
    # every sum is exact but the last draw's t: the token is that of u_final
    assert got["out_tokens"][:, 0].tolist() == [0, V // 2, int(np.float32(0.99) * float(V))]
    assert np.all(got["path"] == O.PATH_REJECT) and np.all(got["residual_mass"] == 0)


def test_request_errors_leave_the_others():
    V, K, B = 3000, 3, 16
    for dtype in (F32, BF):
        w = make(B, K, V, dtype, 21)
        w["draft_len"][0] = K + 1
        w["draft_len"][1] = -1
        w["draft_tokens"][2, 1] = V
        w["draft_tokens"][3, 2] = -1
        w["u"][4, 0] = 1.0
        w["u"][5, 1] = float("nan")
        w["u_final"][6] = -0.25
        w["draft_probs"][7, 0, w["draft_tokens"][7, 0]] = 0.0          # q(x) = 0
        w["target_probs"][8, 1, w["draft_tokens"][8, 1]] = float("nan")
        w["target_probs"][9, 0, w["draft_tokens"][9, 0]] = -0.5
        w["draft_len"][10:14] = 0
        w["target_probs"][10, 0, 2999] = float("inf")                  # rows the draw reads
        w["target_probs"][11, 0, 1000] = float("nan")
        w["target_probs"][12, 0, 17] = -1e-30
        w["target_probs"][13, 0] = 0.0
        w["u"][14] = 0.0                                               # accepts the rest
        w["target_probs"][14, 0, 5] = float("nan")                     # a row it does not draw from
        if w["draft_tokens"][14, 0] == 5:
            w["draft_tokens"][14, 0] = 6
        got, ref = check(w)
        assert np.all(got["n_emitted"][:14] == -1) and np.all(got["n_emitted"][14:] > 0)


def test_invalid_draft_row_of_a_rejection():
    w = make(4, 1, 40000, F32, 22)
    w["u"][:] = 1 - 2.0 ** -24
    w["target_probs"][:, 0] *= 0.5                       # p < q at most tokens: rejects
    bad = (w["draft_tokens"][1, 0].item() + 77) % 40000
    w["draft_probs"][1, 0, bad] = float("nan")
    got, ref = check(w)
    assert ref["path"][0] == O.PATH_REJECT and got["n_emitted"][1] == -1


def test_tokens_past_draft_len_are_not_looked_at():
    w = make(8, 4, 2000, F32, 23)
    w["draft_len"][:] = 2
    w["draft_tokens"][:, 2:] = 1 << 30
    w["u"][:, 2:] = float("nan")
    check(w)


def test_broadcast_and_transposed_rows():
    # one target row for every position (stride 0), draft rows laid out [K, B, V]
    B, K, V = 6, 3, 5000
    w = make(B, K, V, F32, 24)
    t = w["target_probs"][:, :1].contiguous()
    w["target_probs"] = t.expand(B, K + 1, V)
    w["draft_probs"] = w["draft_probs"].transpose(0, 1).contiguous().transpose(0, 1)
    g = {k: v.to(DEV) for k, v in w.items() if k not in ("target_probs", "draft_probs")}
    g["target_probs"] = t.to(DEV).expand(B, K + 1, V)
    g["draft_probs"] = w["draft_probs"].transpose(0, 1).contiguous().to(DEV).transpose(0, 1)
    assert g["target_probs"].stride(1) == 0 and g["draft_probs"].stride(0) == V
    got = to_numpy(S.verify_probs(**g, debug=True))
    rep = compare(got, reference(w, -1), K, alpha_tol=2.0 ** -24, mass_tol=1e-9)
    assert not rep["mismatches"], rep["mismatches"][:3]


def test_offsets_past_32_bits():
    # rows that start past 2^31 elements
    B, K, V = 3, 1, 4096
    w = make(B, K, V, BF, 25)
    far = (1 << 31) // 2 + 12345 * 8
    base = torch.zeros(far * 2 + (K + 1) * V, dtype=BF, device=DEV)
    t = torch.as_strided(base, (B, K + 1, V), (far, V, 1))
    t.copy_(w["target_probs"])
    g = on_gpu(w)
    g["target_probs"] = t
    got = to_numpy(S.verify_probs(**g, debug=True))
    rep = compare(got, reference(w, -1), K, alpha_tol=2.0 ** -24, mass_tol=1e-9)
    assert not rep["mismatches"], rep["mismatches"][:3]


def test_rows_around_the_outputs_are_left():
    w = make(5, 3, 40000, F32, 26)
    out = torch.full((7, 4), 99, dtype=torch.int32, device=DEV)
    ne = torch.full((7,), 99, dtype=torch.int32, device=DEV)
    S.verify_probs(**on_gpu(w), out_tokens=out[1:6], n_emitted=ne[1:6])
    assert (out[0] == 99).all() and (out[6] == 99).all() and ne[0] == 99 and ne[6] == 99


@pytest.mark.parametrize("V", [2000, 40000])
def test_streams_graphs_and_repeats(V):
    w1, w2 = make(8, 4, V, F32, 27), make(8, 4, V, F32, 28)
    a, b = on_gpu(w1), on_gpu(w2)
    ra, rb = (to_numpy(S.verify_probs(**x)) for x in (a, b))
    # two streams at once, each with its own workspace
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):
        x, y = S.verify_probs(**a, stream=s1), S.verify_probs(**b, stream=s2)
        torch.cuda.synchronize()
        for k in ra:
            assert np.array_equal(x[k].cpu().numpy(), ra[k]) and np.array_equal(y[k].cpu().numpy(), rb[k])
    # captured once, replayed on other inputs, eager calls between the replays
    static = {k: v.clone() for k, v in a.items()}
    S.verify_probs(**static)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        res = S.verify_probs(**static)
    for src, want in ((b, rb), (a, ra), (b, rb), (a, ra)):
        for k in static:
            static[k].copy_(src[k])
        g.replay()
        torch.cuda.synchronize()
        for k in want:
            assert np.array_equal(res[k].cpu().numpy(), want[k]), k
        S.verify_probs(**src)


def test_python_refusals():
    big = on_gpu(make(2, 2, 70000, F32, 30))
    w = on_gpu(make(2, 2, 100, F32, 30))
    with pytest.raises(TypeError):
        S.verify_probs(**dict(w, target_probs=w["target_probs"].half()))
    with pytest.raises(TypeError):
        S.verify_probs(**dict(w, draft_probs=w["draft_probs"].to(BF)))
    with pytest.raises(ValueError):
        S.verify_probs(**dict(w, target_probs=w["target_probs"].transpose(1, 2).contiguous().transpose(1, 2)))
    with pytest.raises(ValueError):
        S.verify_probs(**dict(w, draft_tokens=w["draft_tokens"][:, :1]))
    with pytest.raises(S.SpecVerifyError):
        S.verify_probs(**w, eos_id=100)
    with pytest.raises(S.SpecVerifyError) as e:
        S.verify_probs(**big, workspace=torch.empty(8, dtype=torch.uint8, device=DEV))
    assert e.value.status == 2
    empty = torch.empty(0, 3, 100, device=DEV)
    with pytest.raises(S.SpecVerifyError):
        S.verify_probs(empty, None, torch.empty(0, 2, dtype=torch.int32, device=DEV),
                       torch.empty(0, dtype=torch.int32, device=DEV), torch.empty(0, 2, device=DEV),
                       torch.empty(0, device=DEV))
