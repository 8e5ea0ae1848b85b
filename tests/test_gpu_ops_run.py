"""The operators together, as a decode loop uses them (GPU only).

One round: the norms before the LM head give 8-bit hidden states, the 8-bit LM
head and the verification run on them, the round's statistics and the next
draft lengths follow.  The same round from the bfloat16 hidden states takes
the bfloat16 LM head, and the same decisions come from the softmax of the same
logits through the verification from probabilities.
"""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import oracle as O  # noqa: E402
import speculative_decoding_sampling_amd as S  # noqa: E402
from oracle import operators as OP  # noqa: E402
from speculative_decoding_sampling_amd import binding  # noqa: E402
from tests.parity import compare, to_numpy  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32, E4 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


def test_rounds_of_a_decode_loop():
    B, K, V, D = 6, 4, 3000, 512
    g = torch.Generator(device=DEV).manual_seed(3)
    rnd = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    wt = rnd(V, D) * 2 / D ** 0.5
    packed, packed_bf = S.pack_fp8_lm_head(wt), binding.pack_lm_head_weight(wt.to(BF))
    weight, post, gate = (1 + 0.1 * rnd(D)).to(BF), (1 + 0.1 * rnd(D)).to(BF), torch.sigmoid(rnd(B, D)).to(BF)
    residual = rnd(B, K + 1, D)
    monitor = S.DraftLengthMonitor(B, 8, K, DEV)
    n = torch.full((B,), K, dtype=torch.int32, device=DEV)
    for step in range(4):
        x = rnd(B, K + 1, D).to(BF)
        before = residual.clone()
        args = dict(post_weight=post, gate=gate, scale=0.5)
        r1, q, s = S.hidden_norm(x, residual, weight, dtype=E4, **args)
        r2, y = S.hidden_norm(x, residual, weight, **args)
        assert torch.equal(r1, r2) and torch.equal(before, residual)
        h_ref, y_ref, _ = OP.hidden_norm(x.double().cpu().numpy().reshape(-1, D),
                                         residual.double().cpu().numpy().reshape(-1, D),
                                         weight.double().cpu().numpy(), post.double().cpu().numpy(),
                                         gate.double().cpu().numpy(), 0.5)
        assert np.allclose(y.double().cpu().numpy().reshape(-1, D), y_ref, rtol=2.0 ** -8, atol=1e-6)
        logits = S.fp8_lm_head(q, s, packed)
        dl = (logits[:, :K].float() + 0.3 * rnd(B, K, V)).to(BF).contiguous()
        tok = S.sample(dl.reshape(B * K, V), torch.rand(B * K, generator=g, device=DEV)).view(B, K)
        d = dict(draft_logits=dl, draft_tokens=tok, draft_len=n,
                 u=torch.rand(B, K, generator=g, device=DEV), u_final=torch.rand(B, generator=g, device=DEV))
        res = S.verify_fp8_lm_head(q, s, packed, **d, debug=True)
        assert torch.equal(res["target_logits"], logits)
        up = lambda t: t.view(torch.int16).cpu().numpy().view(np.uint16)  # noqa: E731
        ora = O.verify(up(logits), up(dl), tok.cpu().numpy(), n.cpu().numpy(), d["u"].cpu().numpy(),
                       d["u_final"].cpu().numpy(), 1.0, 0, 1.0, -1, "bf16")
        rep = compare(to_numpy({k: v for k, v in res.items() if k != "target_logits"}), ora, K)
        assert not rep["mismatches"], rep["mismatches"][:3]
        # from probabilities: float32 softmax of the same logits
        tp, dp = torch.softmax(logits.float(), -1), torch.softmax(dl.float(), -1)
        pr = S.verify_probs(tp, dp, tok, n, d["u"], d["u_final"], debug=True)
        po = OP.verify_probs(tp.double().cpu().numpy(), dp.double().cpu().numpy(), tok.cpu().numpy(),
                             n.cpu().numpy(), d["u"].cpu().numpy(), d["u_final"].cpu().numpy())
        po["topp_margin_rows"] = np.full((B, 2 * K + 1), np.inf)
        rep = compare(to_numpy(pr), po, K)
        assert not rep["mismatches"], rep["mismatches"][:3]
        assert (pr["accept_prob"] - res["accept_prob"]).abs().max() < 1e-4
        acc, _, totals = S.round_stats(tok, n, res["out_tokens"], res["n_emitted"])
        assert totals[1] == 0 and totals[0] == B
        n, _ = monitor.update(tok, n, res["out_tokens"], res["n_emitted"])
        # the bfloat16 LM head takes the bfloat16 hidden states of the same call
        ref = binding.verify_lm_head(y, packed_bf, **dict(d, draft_len=torch.zeros_like(n)))
        dev = (ref["target_logits"].float() - logits.float()).norm() / logits.float().norm()
        assert dev < 0.1                     # 8-bit operands: a few percent apart
        residual = r1


@pytest.mark.parametrize("B,V", [(4, 40000), (2, 1000), (40, 9000)])   # path 3 twice, path 0
def test_a_round_in_a_graph(B, V):
    K, D = 3, 256
    assert (binding.path_kind(B, K, V) == 3) == (B < 40)
    g = torch.Generator(device=DEV).manual_seed(4)
    rnd = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    packed = S.pack_fp8_lm_head((rnd(V, D) * 3 / D ** 0.5).to(BF))
    weight = (1 + 0.1 * rnd(D)).to(BF)
    x, r = rnd(B, K + 1, D).to(BF), rnd(B, K + 1, D).to(BF)
    dl, tok = (rnd(B, K, V) * 2).to(BF), torch.randint(0, V, (B, K), generator=g, device=DEV, dtype=torch.int32)
    n = torch.full((B,), K, dtype=torch.int32, device=DEV)
    u, uf = torch.rand(B, K, generator=g, device=DEV), torch.rand(B, generator=g, device=DEV)

    def step():
        _, q, s = S.hidden_norm(x, r, weight, dtype=E4)
        res = S.verify_fp8_lm_head(q, s, packed, dl, tok, n, u, uf)
        # the graph's own allocations between the calls take back freed memory
        fill = [torch.full((1 << k,), 0x5a, dtype=torch.uint8, device=DEV) for k in range(10, 22)]
        pr = S.verify_probs(torch.softmax(res["target_logits"].float(), -1), None, tok, n, u, uf)
        return res, pr, fill[0]

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        res, pr, _ = step()
    for k in range(4):
        x.copy_(rnd(B, K + 1, D))
        uf.copy_(torch.rand(B, generator=g, device=DEV))
        graph.replay()
        torch.cuda.synchronize()
        eres, epr, _ = step()
        torch.cuda.synchronize()
        for a, b in ((res, eres), (pr, epr)):
            for key in a:
                assert torch.equal(a[key], b[key]), (k, key)
