"""Verification from probabilities at vocabularies of two kernels (GPU only):
around the number of chunk sums that the draw keeps in registers, exact edges
between chunks and batches of them, and rows whose residual is empty."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import oracle as O  # noqa: E402
import speculative_decoding_sampling_amd as S  # noqa: E402
from tests.test_gpu_ops_probs import BF, F32, check, make  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("V", [65536, 65537, 262143, 262144, 262145])
@pytest.mark.parametrize("dtype", [F32, BF])
def test_around_the_held_sums(V, dtype):
    print(f"[probs] V={V} {dtype}", flush=True)
    check(make(3, 2, V, dtype, seed=V, ragged=True, sharp=4.0), eos=1)


@pytest.mark.parametrize("V", [50000, 200000, 262144, 300001])
def test_exact_edges(V):
    # dyadic weights at the ends of chunks (1024 ids) and of batches of 64 of them
    ids = [0, 1023, 1024, 40000, V - 1]
    if V > 65536:
        ids = [1023, 65535, 65536, 131072, V - 1]
    w = torch.tensor([0.125, 0.25, 0.25, 0.125, 0.25])
    p = torch.zeros(1, 1, V)
    p[0, 0, ids] = w
    p = p.to(DEV)
    e = torch.cumsum(w, 0).tolist()
    none = torch.zeros(1, 0, dtype=torch.int32, device=DEV)
    for k in range(5):
        for uf, y in ((e[k] - 2.0 ** -24, ids[k]), (e[k - 1] if k else 0.0, ids[k])):
            r = S.verify_probs(p, None, none, torch.zeros(1, dtype=torch.int32, device=DEV),
                               none.float(), torch.full((1,), uf, device=DEV))
            assert r["out_tokens"].item() == y, (k, uf)


@pytest.mark.parametrize("V", [262144, 300000])
def test_empty_residual(V):
    p = torch.full((2, 2, V), 2.0 ** -12)
    q = torch.full((2, 1, V), 2.0 ** -11)
    uf = torch.tensor([0.25, 0.99])
    r = S.verify_probs(p.to(DEV), q.to(DEV), torch.full((2, 1), 7, dtype=torch.int32, device=DEV),
                       torch.ones(2, dtype=torch.int32, device=DEV), torch.full((2, 1), 0.9, device=DEV),
                       uf.to(DEV), debug=True)
    assert r["out_tokens"][:, 0].tolist() == [V // 4, int(np.float32(0.99) * float(V))]
    assert (r["path"] == O.PATH_REJECT).all() and not r["residual_mass"].any()


@pytest.mark.parametrize("V", [262144, 300000])
def test_a_bad_entry_anywhere_is_an_error(V):
    w = make(4, 1, V, F32, 5)
    w["draft_len"][:] = 0                               # bonus rows: the whole row is read
    t = w["target_probs"]
    t[0, 0, V - 1], t[1, 0, 65536], t[2, 0, 1023] = float("nan"), -0.5, float("inf")
    up = lambda x: None if x is None else x.to(DEV)  # noqa: E731
    r = S.verify_probs(**{k: up(v) for k, v in w.items()}, debug=True)
    assert r["n_emitted"].tolist() == [-1, -1, -1, 1]
    assert (r["out_tokens"][:3] == -1).all() and r["path"].tolist()[:3] == [O.PATH_ERROR] * 3
