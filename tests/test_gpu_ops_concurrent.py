"""The operators called from two threads on two streams at once, on inputs of
unusual strides and dimensions, and with workspaces of the caller's (GPU only).
Every result must equal that of the same call made alone."""

import threading

import pytest

torch = pytest.importorskip("torch")

import speculative_decoding_sampling_amd as S  # noqa: E402
from speculative_decoding_sampling_amd import binding, ops  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32, E4 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


def bits(t):
    return t if t.dtype in (torch.int32, torch.float64) else t.contiguous().view(torch.uint8)


def same(a, b):
    return all(torch.equal(bits(x), bits(y)) for x, y in zip(a, b))


def round_inputs(B, K, V, D, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    x, r = rnd(B, K + 1, D).to(BF), rnd(B, K + 1, D)
    w = (1 + 0.1 * rnd(D)).to(BF)
    packed = S.pack_fp8_lm_head(rnd(V, D) * 2 / D ** 0.5)
    d = dict(draft_logits=(2 * rnd(B, K, V)).to(BF),
             draft_tokens=torch.randint(0, V, (B, K), generator=g, device=DEV, dtype=torch.int32),
             draft_len=torch.randint(0, K + 1, (B,), generator=g, device=DEV, dtype=torch.int32),
             u=torch.rand(B, K, generator=g, device=DEV),
             u_final=torch.rand(B, generator=g, device=DEV))
    return x, r, w, packed, d


def one_round(x, r, w, packed, d, stream=None, **kw):
    r1, q, s = S.hidden_norm(x, r, w, post_weight=w, scale=0.5, dtype=E4, stream=stream)
    v = S.verify_fp8_lm_head(q, s, packed, **d, debug=True, stream=stream, **kw)
    if stream is not None:
        torch.cuda.current_stream().wait_stream(stream)
    p = {k: t for k, t in d.items() if k != "draft_logits"}
    probs = S.verify_probs(torch.softmax(v["target_logits"].float(), -1),
                           torch.softmax(d["draft_logits"].float(), -1), **p, debug=True)
    torch.cuda.current_stream().synchronize()
    return [r1, q, s, *v.values(), *probs.values()]


@pytest.mark.parametrize("B,K,V,D", [(3, 2, 3000, 256), (24, 4, 40000, 384)])
def test_two_threads(B, K, V, D):
    ins = [round_inputs(B, K, V, D, 40 + i) for i in range(2)]
    want = [one_round(*i) for i in ins]
    bad = []

    def work(i, stream):
        try:
            with torch.cuda.stream(stream):
                for _ in range(8):
                    if not same(one_round(*ins[i]), want[i]):
                        bad.append(i)
        except Exception as e:                                  # noqa: BLE001
            bad.append(e)

    ts = [threading.Thread(target=work, args=(i, torch.cuda.Stream())) for i in range(2)]
    torch.cuda.synchronize()
    for t in ts:
        t.start()
    for t in ts:
        t.join()
    assert not bad, bad


@pytest.mark.parametrize("B,K,V,D", [(3, 2, 3000, 256), (24, 4, 40000, 384)])
def test_given_stream_and_workspace(B, K, V, D):
    ins = round_inputs(B, K, V, D, 50)
    want = one_round(*ins)
    n = ops.load_ops_library().specv_verify_fp8_lm_head_workspace_bytes(B, K, V, D, 0, 1.0)
    ws = torch.randint(0, 256, (n + 512,), device=DEV, dtype=torch.uint8)
    s1 = torch.cuda.Stream()
    for _ in range(3):
        assert same(one_round(*ins, stream=s1), want)
        assert same(one_round(*ins, workspace=ws), want)
    # the bytes behind the workspace are not its own
    ws[n:] = 7
    assert same(one_round(*ins, workspace=ws[:n]), want) and bool((ws[n:] == 7).all())


@pytest.mark.parametrize("V", [5000, 50000])
def test_probabilities_of_any_stride(V):
    B, K = 5, 3
    g = torch.Generator(device=DEV).manual_seed(V)
    rows = torch.softmax(torch.randn(K + 1, V, generator=g, device=DEV) * 2, -1)
    dr = torch.softmax(torch.randn(1, V, generator=g, device=DEV) * 2, -1)
    d = dict(draft_tokens=torch.multinomial(dr.expand(B, V), K, generator=g).int(),
             draft_len=torch.full((B,), K, dtype=torch.int32, device=DEV),
             u=torch.rand(B, K, generator=g, device=DEV), u_final=torch.rand(B, generator=g, device=DEV))
    t, q = rows.expand(B, K + 1, V), dr.expand(B, K, V)           # strides of zero
    want = list(S.verify_probs(t.contiguous(), q.contiguous(), **d, debug=True).values())
    assert same(S.verify_probs(t, q, **d, debug=True).values(), want)
    kt = t.transpose(0, 1).contiguous().transpose(0, 1)           # position-major storage
    kq = q.transpose(0, 1).contiguous().transpose(0, 1)
    assert same(S.verify_probs(kt, kq, **d, debug=True).values(), want)
    wide = torch.full((B, K + 1, V + 7), float("nan"), device=DEV)  # rows that start anywhere
    wide[:, :, 3:V + 3] = t
    assert same(S.verify_probs(wide[:, :, 3:V + 3], q, **d, debug=True).values(), want)


def test_one_row_and_many_dimensions():
    g = torch.Generator(device=DEV).manual_seed(60)
    x = torch.randn(2, 3, 1, 4, 256, generator=g, device=DEV)
    w = torch.rand(256, generator=g, device=DEV)
    packed = S.pack_fp8_lm_head(torch.randn(300, 256, generator=g, device=DEV))
    r, q, s = S.hidden_norm(x, x, w, dtype=E4)
    z = S.fp8_lm_head(q, s, packed, dtype=F32)
    assert z.shape == (2, 3, 1, 4, 300) and s.shape == (2, 3, 1, 4, 2)
    r1, q1, s1 = S.hidden_norm(x[1, 2, 0, 3], x[1, 2, 0, 3], w, dtype=E4)
    z1 = S.fp8_lm_head(q1, s1, packed, dtype=F32)
    assert same([r1, q1, s1, z1], [r[1, 2, 0, 3], q[1, 2, 0, 3], s[1, 2, 0, 3], z[1, 2, 0, 3]])


def test_path_of_the_small_batch_follows_other_work():
    # the one-kernel verification polls words of its workspace: memory that held
    # anything before must not be taken for its own
    B, K, V, D = 2, 2, 3000, 256
    assert binding.path_kind(B, K, V) == 3
    ins = round_inputs(B, K, V, D, 70)
    want = one_round(*ins)
    for fill in (0, 255, 1):
        n = ops.load_ops_library().specv_verify_fp8_lm_head_workspace_bytes(B, K, V, D, 0, 1.0)
        ws = torch.full((n,), fill, device=DEV, dtype=torch.uint8)
        for _ in range(3):
            assert same(one_round(*ins, workspace=ws), want)


def test_outputs_in_inference_mode():
    x, w = torch.randn(4, 256, device=DEV), torch.ones(256, device=DEV)
    want = S.hidden_norm(x, x, w)
    with torch.inference_mode():
        got = S.hidden_norm(x, x, w)
        assert all(t.is_inference() for t in got) and same(got, want)
    p = x.clone().requires_grad_(True)                            # no gradients are recorded
    assert not any(t.requires_grad for t in S.hidden_norm(p, p, w))
