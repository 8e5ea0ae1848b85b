"""Filtered distributions and draws on rows that mislead a sample of them, overflow
a list or tie in the thousands, against the fp64 reference (the tolerances are
those of test_gpu_draft_filter.py)."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import speculative_decoding_sampling_amd as S  # noqa: E402
from test_gpu_draft_filter import BF, DEV, F32, I32, both, check, logits  # noqa: E402

pytestmark = pytest.mark.gpu

FILTERS = [(1.0, 0, 0.9, 0.0), (0.7, 50, 0.95, 0.0), (1.0, 3000, 0.8, 0.0), (1.0, 20000, 1.0, 0.0),
           (1.5, 0, 0.99, 0.001), (1.0, 5000, 0.999, 0.01), (0.3, 0, 0.02, 0.0)]


def shaped(kind, V, R, seed):
    """[R, V] logits of a shape that an even sample of the row does not show."""
    z = logits(R, V, seed, F32, 2.0, 0)
    if kind == "ascending":
        return z.sort(dim=1).values
    if kind == "descending":
        return z.sort(dim=1, descending=True).values
    if kind == "last":                              # the mass in the last few ids
        z -= 20.0
        z[:, -37:] += 25.0
    if kind == "first":
        z -= 20.0
        z[:, :37] += 25.0
    if kind == "run":                               # in one run of 9000 that starts anywhere
        z -= 30.0
        z[:, V // 3 + 1:V // 3 + 9001] += 30.0
    if kind == "comb":                              # at every 64th id
        z -= 30.0
        z[:, 5::64] += 30.0
    if kind == "one":                               # one token has nearly all
        z[:, V // 2 + 3] = 40.0
    return z


@pytest.mark.parametrize("kind", ["ascending", "descending", "last", "first", "run", "comb", "one"])
@pytest.mark.parametrize("V,dtype", [(32768, F32), (33000, F32), (50001, BF), (152064, F32), (200003, BF)])
def test_shaped_rows(kind, V, dtype):
    R, near = 3, 0
    for n, (T, k, p, mp) in enumerate(FILTERS):
        print(f"[filter] {kind} V={V} {dtype} T={T} k={k} p={p} mp={mp}", flush=True)
        z = shaped(kind, V, R, 31 * n + V).to(dtype)
        u = torch.rand(R, generator=torch.Generator().manual_seed(n))
        probs, tok = both(z, u, T, k, p, mp)
        near += check(z, u, T, k, p, mp, probs, tok)
    assert near <= 1 + len(FILTERS) * R // 20


@pytest.mark.parametrize("V", [30000, 50001, 129279])
@pytest.mark.parametrize("dtype", [F32, BF])
def test_ties_by_the_thousand(V, dtype):
    u = torch.tensor([0.0, 0.37, 0.99])
    flat = torch.zeros(3, V)
    steps = torch.zeros(3, V)                       # three values: 5 %, 60 %, the rest
    steps[:, ::20] = 2.0
    steps[:, 1::5] = 1.0
    steps[:, 2::5] = 1.0
    steps[:, 3::5] = 1.0
    coarse = logits(3, V, V).mul(2).round().div(2)  # half steps
    for z in (flat, steps, coarse):
        z = z.to(dtype)
        for f in ((1.0, 10, 1.0, 0.0), (1.0, 0, 0.5, 0.0), (0.8, V // 2, 0.9, 0.0), (1.0, V - 1, 1.0, 0.0),
                  (2.0, 0, 0.97, 0.1)):
            print(f"[filter] ties V={V} {dtype} {f}", flush=True)
            probs, tok = both(z, u, *f)
            assert check(z, u, *f, probs, tok) <= 1


def test_a_row_that_is_nearly_all_masked():
    V = 60000
    u = torch.tensor([0.0, 0.5, 0.999, 0.2])
    for value in (-np.inf, float(torch.finfo(F32).min)):
        z = torch.full((4, V), value)
        z[0, V - 1] = 1.0
        z[1, 0] = -3.0
        z[2, [5, 40000, 59999]] = torch.tensor([1.0, 2.0, 1.5])
        for f in ((1.0, 50, 0.9, 0.0), (1.0, 0, 0.9, 0.0), (1.0, 0, 1.0, 0.1), (0.0, 0, 1.0, 0.0),
                  (1.0, 1000, 1.0, 0.0), (1.0, 0, 1.0, 0.0)):
            probs, tok = both(z, u, *f)
            assert check(z, u, *f, probs, tok) == 0


def test_the_same_row_again_and_again():
    for V in (5000, 50000):
        z = logits(1, V, V)
        u = torch.rand(6, generator=torch.Generator().manual_seed(V))
        args = (0.8, 40, 0.95, 0.01)
        once = z.expand(6, V)
        assert once.stride(0) == 0
        whole = once.contiguous()
        got = S.filter_probs(once.to(DEV), *args, u=u.to(DEV))
        spread = S.filter_probs(z.to(DEV).expand(6, V), *args, u=u.to(DEV))
        assert all(map(torch.equal, got, spread))
        assert check(whole, u, *args, *got) == 0


def test_more_rows_than_a_grid_has_columns():
    R, V = 70001, 5
    z = logits(R, V, 3, F32, 2.0, 0)
    u = torch.rand(R, generator=torch.Generator().manual_seed(4))
    probs, tok = both(z, u, 0.9, 3, 0.9, 0.01)
    at = torch.tensor([0, 1, 65535, 65536, 70000])
    assert check(z[at], u[at], 0.9, 3, 0.9, 0.01, probs[at.to(DEV)], tok[at.to(DEV)]) == 0
    part = S.sample_filtered(z[60000:].to(DEV), u[60000:].to(DEV), 0.9, 3, 0.9, 0.01)
    assert torch.equal(part, tok[60000:])


def test_two_graphs_with_their_own_filters():
    V, B, L = 50001, 3, 2
    z = logits(B * L, V, 8).view(B, L, V).to(DEV)
    u = torch.rand(B, L, device=DEV)
    a = (0.9, 50, 0.95, 0.0)
    b = (torch.tensor([1.0, 0.0, 0.7], device=DEV), torch.tensor([0, 5, 4000], dtype=I32, device=DEV),
         torch.tensor([0.9, 1.0, 0.9], device=DEV), 0.0)
    want = [S.filter_probs(z, *f, u=u, dtype=BF) for f in (a, b)]
    torch.cuda.synchronize()
    graphs = []
    for f in (a, b):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            res = S.filter_probs(z, *f, u=u, dtype=BF)
        graphs.append((g, res))
    for i in (0, 1, 1, 0, 1, 0, 0):
        graphs[i][0].replay()
        eager = S.sample_filtered(z, u, *a)
        torch.cuda.synchronize()
        assert all(map(torch.equal, graphs[i][1], want[i])) and torch.equal(eager, want[0][1])
    rows = z.view(B * L, V).cpu()
    for f, (probs, tok) in zip((a, b), want):
        f = tuple(x.cpu() if isinstance(x, torch.Tensor) else x for x in f)
        assert check(rows, u.view(-1).cpu(), *f, probs.view(B * L, V), tok.view(-1), L=L) <= 1


def test_largest_vocabulary_of_float32():
    V = 4194304
    z = logits(2, V, 6, F32, 2.0, 40)
    u = torch.tensor([0.3, 0.99999])
    T, p = torch.tensor([1.0, 0.8]), torch.tensor([1.0, 0.9])
    for k in (0, 40):
        probs, tok = both(z, u, T, k, p, 0.0)
        assert check(z, u, T, k, p, 0.0, probs, tok) <= 1


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("n", [63, 64, 65, 300, 511, 512, 513, 900])
def test_lists_of_every_length(n, dtype):
    # n equal logits around the threshold, a few above them, the rest far below
    u = torch.tensor([0.0, 0.4, 0.9999])
    for V in (1200, 20001, 32768, 40000):
        z = logits(3, V, n + V, F32, 1.0, 0) - 6.0
        at = torch.randperm(V, generator=torch.Generator().manual_seed(n))[:n + 5]
        z[:, at] = 4.0
        z[:, at[:5]] = torch.tensor([5.0, 5.5, 6.0, 6.5, 7.0])
        z = z.to(dtype)
        for f in ((1.0, 50, 1.0, 0.0), (1.0, 50, 0.6, 0.0), (1.0, n + 5, 0.9, 0.0), (1.0, 0, 0.8, 0.0),
                  (0.7, 3, 0.9, 0.0), (1.0, n + 4, 1.0, 0.5)):
            probs, tok = both(z, u, *f)
            assert check(z, u, *f, probs, tok) <= 1
