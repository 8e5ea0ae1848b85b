"""A token without weight is never drawn (GPU only).

The running sums of the draw are float64 and each lane's is added in an order
of its own, so neighbouring ones differ by a rounding wherever weights of very
different sizes meet.  Whatever that does to a draw next to an edge, the token
has weight: one that a filter removed has not, nor a lookup's rejected draft.
The draws here lie on edges, where either neighbour is right.
"""

import pytest

torch = pytest.importorskip("torch")

import oracle as O  # noqa: E402
import speculative_decoding_sampling_amd as S  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32
E = 2.0 ** -54


def rows(V, weights, dtype=F32):
    p = torch.zeros(1, 1, V)
    for v, w in weights.items():
        p[0, 0, v] = w
    return p.to(dtype).to(DEV)


def bonus(p, uf=0.5):
    B = len(p)
    none = torch.zeros(B, 0, dtype=torch.int32, device=DEV)
    r = S.verify_probs(p, None, none, torch.zeros(B, dtype=torch.int32, device=DEV), none.float(),
                       torch.full((B,), uf, device=DEV))
    assert (r["n_emitted"] == 1).all()
    return r["out_tokens"][:, 0].long()


# a lane, a chunk or a batch of chunks without weight stands before the one that
# is drawn, whose first entries have none either
EDGES = [
    (128, {0: E, 16: E, 32: 0.5, 70: 0.5}),
    (128, {0: 0.5, 85: 0.5, 16: E, 32: E, 48: E, 96: 2 * E}),
    (5 * 1024 + 100, {0: E, 1024: E, 2048: 0.5, 4096 + 6: 0.5}),
    (40000, {0: E, 16: E, 32: 0.5, 70: 0.5}),
    (40000, {0: E, 1024: E, 2048: 0.5, 4096 + 70: 0.5}),
    (400000, {0: E, 65536: E, 2 * 65536: 0.5, 4 * 65536 + 70: 0.5}),
    (400000, {0: E, 65536: E, 2 * 65536: 0.5, 4 * 65536 + 2048 + 70: 0.5}),
]


@pytest.mark.parametrize("V,weights", EDGES)
@pytest.mark.parametrize("dtype", [F32, BF])
def test_edges_behind_entries_without_weight(V, weights, dtype):
    y = bonus(rows(V, weights, dtype)).item()
    assert weights.get(y) == 0.5, y


@pytest.mark.parametrize("V", [128, 40000])
def test_a_lookups_rejected_draft_is_not_drawn(V):
    # p(64) = 2^-60 rejects the draft, whose residual weight is max(p - 1, 0) = 0
    p = rows(V, {0: E, 16: E, 32: 0.5, 64: 2.0 ** -60, 70: 0.5}).expand(1, 2, V)
    r = S.verify_probs(p, None, torch.full((1, 1), 64, dtype=torch.int32, device=DEV),
                       torch.ones(1, dtype=torch.int32, device=DEV), torch.full((1, 1), 0.5, device=DEV),
                       torch.full((1,), 0.5, device=DEV), debug=True)
    assert r["path"].item() == O.PATH_REJECT and r["out_tokens"][0, 0].item() in (32, 70)


@pytest.mark.parametrize("V", [128, 40000])
def test_a_token_that_the_draft_covers_is_not_drawn(V):
    # equal target and draft probabilities leave token 64 no residual
    p = rows(V, {0: E, 16: E, 32: 0.5, 64: 0.25, 70: 0.5, 100: 2.0 ** -3}).expand(1, 2, V)
    q = rows(V, {64: 0.25, 100: 0.5})
    r = S.verify_probs(p, q, torch.full((1, 1), 100, dtype=torch.int32, device=DEV),
                       torch.ones(1, dtype=torch.int32, device=DEV), torch.full((1, 1), 0.5, device=DEV),
                       torch.full((1,), 0.5, device=DEV), debug=True)
    assert r["path"].item() == O.PATH_REJECT and r["out_tokens"][0, 0].item() in (32, 70)


@pytest.mark.parametrize("V", [1000, 40000])
def test_sparse_rows_of_weights_of_all_sizes(V):
    g = torch.Generator().manual_seed(V)
    B = 2048
    size = torch.tensor([0.5, 2.0 ** -52, 2.0 ** -53, E])
    p = torch.zeros(B, 1, V)
    for b in range(B):
        n = int(torch.randint(3, 9, (1,), generator=g))
        p[b, 0, torch.randperm(V, generator=g)[:n]] = size[torch.randint(0, 4, (n,), generator=g)]
    p[:, 0, V // 2] = 0.5
    y = bonus(p.to(DEV)).cpu()
    assert (p[torch.arange(B), 0, y] > 0).all()
