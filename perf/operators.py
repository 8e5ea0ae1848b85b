"""Cases, plain forms and calls of the operators around the verification step.

Three operators, each measured over the sizes a serving loop meets:

``norm``   the norms around the target's last block with its gate and residual
           scale: r' = r + scale * gate * N(x; post_weight), y = N(r'; weight),
           with N(v; w) = w * v / sqrt(mean(v^2) + eps); y leaves as bfloat16,
           float32 or 8-bit floats with one power-of-two scale for each 128.
``head``   the LM head on 8-bit floats, logits = (hq * hs) (wq * ws)^T, with a
           power-of-two scale for each run of 128 along the hidden size.
``probs``  verification of drafted tokens against given target and draft
           probabilities and given uniforms.

``run`` is the plain form in elementary torch operations, or the library's own
calls where ``own`` is true.
"""

import math

import torch

own = False

DEV = "cuda"
BLOCK = 128
E4M3_MAX = 448.0
EPS = 1e-6


def listed():
    return [
        # one request, one position: a decode step without drafts
        dict(name="norm_1x4096_bf16", op="norm", B=1, L=1, D=4096, x="bf16", r="bf16", w="bf16",
             post=False, gate="none", scale=1.0, y="bf16"),
        # odd sizes in full precision: a ragged batch of a small draft model
        dict(name="norm_37x2047_f32", op="norm", B=37, L=1, D=2047, x="f32", r="f32", w="f32",
             post=True, gate="all", scale=0.5, y="f32"),
        # 64 requests with 4 drafts each: the rows an 8-bit LM head takes
        dict(name="norm_64x5x4096_fp8", op="norm", B=64, L=5, D=4096, x="bf16", r="f32", w="bf16",
             post=True, gate="request", scale=0.25, y="fp8"),
        # a large batch of a wide model, residual stream in bfloat16
        dict(name="norm_256x9x8192_bf16", op="norm", B=256, L=9, D=8192, x="bf16", r="bf16",
             w="f32", post=True, gate="all", scale=1.0, y="bf16"),
        # one request with 5 drafts at a 32000-token vocabulary
        dict(name="head_6x32000x4096", op="head", M=6, V=32000, D=4096, out="bf16", quant=False),
        # odd rows, vocabulary and number of scale blocks, float32 logits
        dict(name="head_37x20001x1152_f32", op="head", M=37, V=20001, D=1152, out="f32",
             quant=False),
        # 64 requests with 4 drafts, hidden states still in bfloat16
        dict(name="head_320x128256x4096_q", op="head", M=320, V=128256, D=4096, out="bf16",
             quant=True),
        # a large batch: 128 requests with 8 drafts
        dict(name="head_1152x152064x4096", op="head", M=1152, V=152064, D=4096, out="bf16",
             quant=False),
        # one request with 5 drafts
        dict(name="probs_1x5x32000_f32", op="probs", B=1, K=5, V=32000, p="f32", onehot=False,
             eos=-1, pad=0, debug=False),
        # 64 requests with 4 drafts, with the diagnostics a monitor reads
        dict(name="probs_64x4x128256_f32", op="probs", B=64, K=4, V=128256, p="f32",
             onehot=False, eos=-1, pad=0, debug=True),
        # ragged draft lengths, an EOS id, rows padded past the vocabulary
        dict(name="probs_64x8x129279_bf16", op="probs", B=64, K=8, V=129279, p="bf16",
             onehot=False, eos=1, pad=1, debug=False),
        # drafts from a lookup (no draft distribution), a large batch
        dict(name="probs_256x8x152064_f32", op="probs", B=256, K=8, V=152064, p="f32",
             onehot=True, eos=-1, pad=0, debug=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "head", "probs"])
    if op == "norm":
        B, L = _log(rng, 1, 256), rng.randint(1, 9)
        y = rng.choice(["bf16", "f32", "fp8", "fp8"])
        D = _log(rng, 1, 64) * BLOCK if y == "fp8" else _log(rng, 64, 8192)
        return dict(op="norm", B=B, L=L, D=D, x=rng.choice(["bf16", "f32"]),
                    r=rng.choice(["bf16", "f32"]), w=rng.choice(["bf16", "f32"]),
                    post=rng.random() < 0.6, gate=rng.choice(["none", "all", "request", "row"]),
                    scale=round(rng.uniform(0.05, 1.5), 3), y=y)
    if op == "head":
        return dict(op="head", M=_log(rng, 1, 1152), V=_log(rng, 1000, 152064),
                    D=_log(rng, 1, 32) * BLOCK, out=rng.choice(["bf16", "f32"]),
                    quant=rng.random() < 0.4)
    return dict(op="probs", B=_log(rng, 1, 256), K=rng.randint(0, 8), V=_log(rng, 500, 152064),
                p=rng.choice(["f32", "bf16"]), onehot=rng.random() < 0.3,
                eos=rng.choice([-1, 1]), pad=rng.choice([0, 0, 1, 7]),
                debug=rng.random() < 0.4)


def _dtype(name):
    return {"bf16": torch.bfloat16, "f32": torch.float32, "fp8": torch.float8_e4m3fn}[name]


def _quantize(x):
    """8-bit values and the power-of-two scale of each 128 of a float32 [R, D]
    tensor: the smallest scale that brings the block's largest magnitude to at
    most 448 (1 for a block of zeros)."""
    R, D = x.shape
    v = x.reshape(R, D // BLOCK, BLOCK)
    amax = v.abs().amax(-1)
    m, e = torch.frexp(amax)                           # amax = m 2^e, m in [0.5, 1)
    e = torch.where(m <= E4M3_MAX / 512, e - 9, e - 8)
    e = torch.where(amax > 0, e, torch.zeros_like(e))
    s = torch.ldexp(torch.ones_like(amax), e)
    q = (v / s[..., None]).to(torch.float8_e4m3fn).reshape(R, D)
    return q, s.to(torch.float8_e8m0fnu)


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    c = dict(case)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=DEV)

    def uniform(*shape):
        return torch.rand(*shape, generator=g, device=DEV)

    if c["op"] == "norm":
        B, L, D = c["B"], c["L"], c["D"]
        wt = _dtype(c["w"])
        big = 1 + 20 * (uniform(D) < 0.01).float()     # a few channels are much larger
        c["x_in"] = (normal(B, L, D) * big * 2).to(_dtype(c["x"]))
        c["r_in"] = (normal(B, L, D) * big * 4).to(_dtype(c["r"]))
        c["weight"] = (1 + 0.2 * normal(D)).to(wt)
        c["post_weight"] = (1 + 0.2 * normal(D)).to(wt) if c["post"] else None
        rows = {"none": 0, "all": 1, "request": B, "row": B * L}[c["gate"]]
        c["gate_in"] = torch.sigmoid(normal(rows, D)).to(wt) if rows else None
        return c

    if c["op"] == "head":
        M, V, D = c["M"], c["V"], c["D"]
        big = 1 + 10 * (uniform(D) < 0.01).float()
        h = (normal(M, D) * big).bfloat16()
        c["hidden"] = h if c["quant"] else _quantize(h.float())
        wq = torch.empty(V, D, dtype=torch.float8_e4m3fn, device=DEV)
        ws = torch.empty(V, D // BLOCK, dtype=torch.float8_e8m0fnu, device=DEV)
        for v0 in range(0, V, 16384):
            n = min(16384, V - v0)
            w = normal(n, D) * torch.exp(0.5 * normal(n, 1)) * (1.5 / math.sqrt(D))
            q, s = _quantize(w)
            wq[v0:v0 + n] = q
            ws.view(torch.uint8)[v0:v0 + n] = s.view(torch.uint8)
        c["wq"], c["ws"] = wq, ws
        if own:
            # the weight in the kernel's load order, laid out once at model load
            from speculative_decoding_sampling_amd import pack_fp8_lm_head
            c["packed"] = pack_fp8_lm_head(wq, ws)
        return c

    B, K, V = c["B"], c["K"], c["V"]
    Vp, dt = V + c["pad"], _dtype(c["p"])
    z = torch.empty(B, K + 1, Vp, device=DEV).normal_(generator=g).mul_(3)
    tp = torch.zeros(B, K + 1, Vp, dtype=dt, device=DEV)
    tp[..., :V] = torch.softmax(z[..., :V], -1).to(dt)
    zd = z[:, :K]
    zd.add_(torch.empty(B, K, Vp, device=DEV).normal_(generator=g).mul_(0.5))
    dp = torch.zeros(B, K, Vp, dtype=dt, device=DEV)
    dp[..., :V] = torch.softmax(zd[..., :V], -1).to(dt)
    # drafted tokens: draws from the draft rows (the largest of q / exponential)
    e = torch.empty(B, K, V, device=DEV).exponential_(generator=g)
    x = (dp[..., :V].float() / e).argmax(-1) if K else torch.zeros(B, 0, dtype=torch.long,
                                                                     device=DEV)
    del z, zd, e
    c["target"] = tp[..., :V]
    c["draft"] = None if c["onehot"] else dp[..., :V]
    if c["onehot"] and K:
        # a lookup proposes likely tokens: the target's own best for two in three
        best = tp[:, :K, :V].float().argmax(-1)
        x = torch.where(uniform(B, K) < 0.67, best, x)
    if c["eos"] >= 0 and K:
        x[::7, K // 2] = c["eos"]
        if c["draft"] is not None:
            # a drafted token has a positive draft probability
            low = 2.0 ** -20
            cur = c["draft"][::7, K // 2, c["eos"]]
            c["draft"][::7, K // 2, c["eos"]] = torch.clamp(cur.float(), min=low).to(dt)
    c["tokens"] = x.to(torch.int32)
    c["len"] = torch.randint(0, K + 1, (B,), generator=g, device=DEV, dtype=torch.int32) \
        if c["eos"] >= 0 else torch.full((B,), K, dtype=torch.int32, device=DEV)
    c["u"], c["u_final"] = uniform(B, K), uniform(B)
    return c


# ------------------------------------------------------------- plain forms

def _norm_plain(c):
    x, r = c["x_in"].float(), c["r_in"].float()
    B, L, D = x.shape
    if c["post_weight"] is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * c["post_weight"].float()
    if c["gate_in"] is not None:
        gate = c["gate_in"].float()
        x = (x.reshape(gate.shape[0], -1, D) * gate[:, None]).reshape(B, L, D)
    h = r + c["scale"] * x
    y = h * torch.rsqrt((h * h).mean(-1, keepdim=True) + EPS) * c["weight"].float()
    res = h.to(c["r_in"].dtype)
    if c["y"] == "fp8":
        q, s = _quantize(y.reshape(B * L, D))
        return res, q.reshape(B, L, D), s.reshape(B, L, D // BLOCK)
    return res, y.to(_dtype(c["y"]))


def _dequantize(q, s):
    R, D = q.shape
    return (q.float().reshape(R, D // BLOCK, BLOCK) * s.float()[..., None]).reshape(R, D)


def _head_plain(c):
    hq, hs = _quantize(c["hidden"].float()) if c["quant"] else c["hidden"]
    return (_dequantize(hq, hs) @ _dequantize(c["wq"], c["ws"]).T).to(_dtype(c["out"]))


def _probs_plain(c):
    tp, dp, K, V = c["target"], c["draft"], c["K"], c["V"]
    B = tp.shape[0]
    n, u, uf = c["len"].long(), c["u"].double(), c["u_final"].double()
    x = c["tokens"].long()
    k = torch.arange(K, device=tp.device)
    used = k < n[:, None]
    px = torch.gather(tp[:, :K], 2, x[..., None])[..., 0].double()
    qx = torch.gather(dp, 2, x[..., None])[..., 0].double() if dp is not None \
        else torch.ones_like(px)
    accept = u * qx < px
    eos = used & accept & (x == c["eos"])
    stops = torch.cat([(used & ~accept) | eos, torch.ones_like(used[:, :1]) if K else
                       torch.ones(B, 1, dtype=torch.bool, device=tp.device)], 1)
    stop = torch.minimum(stops.int().argmax(1), n)
    at = torch.clamp(stop, max=max(K - 1, 0))[:, None]
    is_eos = (torch.gather(eos, 1, at)[:, 0] & (stop < n)) if K else torch.zeros_like(n).bool()
    reject = (stop < n) & ~is_eos
    b = torch.arange(B, device=tp.device)
    p = tp[b, stop].double()
    w = p
    if K:
        if dp is not None:
            q = dp[b, at[:, 0]].double()
        else:
            q = torch.zeros_like(p).scatter_(1, torch.gather(x, 1, at), 1.0)
        res = torch.where(reject[:, None], torch.clamp(p - q, min=0), torch.zeros_like(p))
        mass = res.sum(1)
        w = torch.where((mass > 0)[:, None], res, p)
    else:
        mass = torch.zeros(B, dtype=torch.float64, device=tp.device)
    cum = torch.cumsum(w, 1)
    t = uf * cum[:, -1]
    y = (cum <= t[:, None]).sum(1)
    last = V - 1 - (w.flip(1) > 0).int().argmax(1)
    y = torch.where(y < V, y, last)
    pos = torch.arange(K + 1, device=tp.device)
    xs = torch.cat([x, torch.zeros(B, 1, dtype=torch.long, device=tp.device)], 1)
    keep = (pos < stop[:, None]) | ((pos == stop[:, None]) & is_eos[:, None])
    out = torch.where(keep, xs, torch.full_like(xs, -1))
    out = torch.where((pos == stop[:, None]) & ~is_eos[:, None], y[:, None], out)
    got = [out.int(), (stop + 1).int()]
    if c["debug"]:
        alpha = torch.where(used, torch.clamp(px / qx, max=1), torch.full_like(px, -1)).float()
        got += [alpha, mass]
    return tuple(got)


def _run_own(c):
    import speculative_decoding_sampling_amd as S
    if c["op"] == "norm":
        return S.hidden_norm(c["x_in"], c["r_in"], c["weight"], post_weight=c["post_weight"],
                             gate=c["gate_in"], scale=c["scale"], eps=EPS, dtype=_dtype(c["y"]))
    if c["op"] == "head":
        hq, hs = S.quantize_fp8(c["hidden"]) if c["quant"] else c["hidden"]
        return S.fp8_lm_head(hq, hs, c["packed"], dtype=_dtype(c["out"]))
    r = S.verify_probs(c["target"], c["draft"], c["tokens"], c["len"], c["u"], c["u_final"],
                       c["eos"], debug=c["debug"])
    got = [r["out_tokens"], r["n_emitted"]]
    return tuple(got + [r["accept_prob"], r["residual_mass"]] if c["debug"] else got)


def run(state):
    if own:
        return _run_own(state)
    return {"norm": _norm_plain, "head": _head_plain, "probs": _probs_plain}[state["op"]](state)


def work(case):
    c = case
    size = {"bf16": 2, "f32": 4}
    if c["op"] == "norm":
        M, D = c["B"] * c["L"], c["D"]
        gate = {"none": 0, "all": 1, "request": c["B"], "row": M}[c["gate"]]
        out = D + D // BLOCK if c["y"] == "fp8" else D * size[c["y"]]
        return {"bytes": M * D * (size[c["x"]] + 2 * size[c["r"]]) + M * out +
                (1 + c["post"] + gate) * D * size[c["w"]],
                "flops": M * D * (4 + 4 * c["post"] + 3)}
    if c["op"] == "head":
        M, V, D = c["M"], c["V"], c["D"]
        h = 2 * M * D if c["quant"] else M * (D + D // BLOCK)
        return {"bytes": h + V * (D + D // BLOCK) + M * V * size[c["out"]],
                "flops": 2 * M * V * D}
    B, K, V, s = c["B"], c["K"], c["V"], size[c["p"]]
    # one target row of each request, and the draft row of a rejected position;
    # the entries of the drafted tokens
    rows = B if c["onehot"] or K == 0 else 2 * B
    return {"bytes": rows * V * s + B * K * (2 * s + 8) + B * (K + 4) * 4,
            "flops": 3 * rows * V}


# ------------------------------------------- the definitions in 64 bits

def exact(case, seed):
    c = prepare(case, seed)
    if c["op"] == "norm":
        D = c["D"]
        x = c["x_in"].double().reshape(-1, D)
        r = c["r_in"].double().reshape(-1, D)
        M = x.shape[0]
        if c["post_weight"] is not None:
            x = c["post_weight"].double() * x / (x.square().sum(1, keepdim=True) / D + EPS).sqrt()
        if c["gate_in"] is not None:
            x = x * c["gate_in"].double().repeat_interleave(M // c["gate_in"].shape[0], 0)
        h = r + c["scale"] * x
        y = c["weight"].double() * h / (h.square().sum(1, keepdim=True) / D + EPS).sqrt()
        shape = (c["B"], c["L"], D)
        if c["y"] != "fp8":
            return h.reshape(shape), y.reshape(shape)
        blocks = y.reshape(M, D // BLOCK, BLOCK)
        amax = blocks.abs().max(-1).values
        s = torch.exp2(torch.ceil(torch.log2(amax / E4M3_MAX)))
        s = torch.where(amax > 0, s, torch.ones_like(s))
        return (h.reshape(shape), (blocks / s[..., None]).reshape(shape),
                s.reshape(c["B"], c["L"], -1))
    if c["op"] == "head":
        hq, hs = _quantize(c["hidden"].float()) if c["quant"] else c["hidden"]
        h = hq.double() * hs.float().double().repeat_interleave(BLOCK, 1)
        out = []
        for v0 in range(0, c["V"], 16384):
            w = c["wq"][v0:v0 + 16384].float().double()
            w *= c["ws"][v0:v0 + 16384].float().double().repeat_interleave(BLOCK, 1)
            out.append(torch.mm(h, w.t()))
        return torch.cat(out, 1)
    if not c["debug"]:
        return None
    # the tokens are decisions; the diagnostics are numbers
    B, K = c["B"], c["K"]
    alpha = torch.full((B, K), -1.0, dtype=torch.float64)
    mass = torch.zeros(B, dtype=torch.float64)
    for b in range(B):
        stopped = False
        for k in range(int(c["len"][b])):
            v = int(c["tokens"][b, k])
            p = c["target"][b, k].double()
            q = torch.zeros_like(p)
            if c["draft"] is None:
                q[v] = 1.0
            else:
                q = c["draft"][b, k].double()
            a = min(1.0, float(p[v]) / float(q[v]))
            alpha[b, k] = a
            if stopped:
                continue
            if float(c["u"][b, k]) * float(q[v]) < float(p[v]):
                stopped = v == c["eos"]
            else:
                mass[b] = torch.relu(p - q).sum()
                stopped = True
    return None, None, alpha.to(DEV), mass.to(DEV)
