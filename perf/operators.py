"""The operators around the expert layer, as cases that can be timed and compared.

What runs between the residual stream and the experts of one MoE block, in order: the
residual's addition with its root-mean-square norm and an 8-bit output (``moe_add_rmsnorm``),
the router's product (``moe_gate_logits``), the choice of experts (``moe_route_groups``), and
the dense projections into and out of the experts' width, in 8-bit integers
(``moe_int8_linear`` from bf16 tokens, ``moe_int8_matmul`` from tokens the norm has quantised).

``own`` False computes each in its plain form (elementary torch operations), True calls the
package.  ``exact`` is each operator's definition in 64 bits.
"""
import math

import torch

own = False

LOWEST = -3.4028234663852886e38   # the lowest finite float: masks an expert, as -inf does
EPS = 1e-6
BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64


def listed():
    return [
        # One token of a decode step through the norm in front of the experts (MXFP8 output).
        dict(name="norm_decode_1", op="norm", T=1, H=7168, q8="mxfp8", residual=True),
        # The same norm for an 8K prefill chunk.
        dict(name="norm_chunk_8192", op="norm", T=8192, H=7168, q8="mxfp8", residual=True),
        # One token's projection from the hidden width into the experts' width.
        dict(name="int8_decode_1", op="int8", M=1, N=3584, K=7168, out="bf16"),
        # A decode batch: the norm gives 8-bit tokens with a scale each, the projection takes them.
        dict(name="norm_int8_256", op="normed", M=256, N=3584, K=7168),
        # A ragged batch, odd output width, float32 output (sums that go on in float32).
        dict(name="int8_ragged_1000", op="int8", M=1000, N=2051, K=1040, out="f32"),
        # An 8K prefill chunk's projection.
        dict(name="int8_chunk_8192", op="int8", M=8192, N=3584, K=7168, out="bf16"),
        # Router logits of a small decode batch, of a large one, of an 8K chunk.
        dict(name="gate_decode_8", op="gate", T=8, H=7168, E=896),
        dict(name="gate_batch_256", op="gate", T=256, H=7168, E=896),
        dict(name="gate_chunk_8192", op="gate", T=8192, H=7168, E=896),
        # Group-limited sigmoid routing with a balance bias: a decode batch and an 8K chunk.
        dict(name="route_decode_8", op="route", T=8, E=896, K=16, G=8, KG=4, score="sigmoid",
             group="top2", bias=True, renorm=True, masked=0.0),
        dict(name="route_chunk_8192", op="route", T=8192, E=896, K=16, G=8, KG=4,
             score="sigmoid", group="top2", bias=True, renorm=True, masked=0.0),
        # Softmax routing over few experts, some of them masked, weights not renormalised.
        dict(name="route_softmax_4096", op="route", T=4096, E=128, K=8, G=1, KG=1,
             score="softmax", group="max", bias=False, renorm=False, masked=0.05),
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], spread evenly over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "int8", "normed", "gate", "route"])
    if op == "norm":
        return dict(op=op, T=_spread(rng, 1, 8192), H=32 * _spread(rng, 4, 224),
                    q8=rng.choice(["mxfp8", "int8", "none"]), residual=rng.random() < 0.8)
    if op in ("int8", "normed"):
        c = dict(op=op, M=_spread(rng, 1, 8192), N=_spread(rng, 64, 3584),
                 K=16 * _spread(rng, 8, 448))
        if op == "int8":
            c["out"] = rng.choice(["bf16", "f32"])
        return c
    if op == "gate":
        return dict(op=op, T=_spread(rng, 1, 8192), H=8 * _spread(rng, 16, 896),
                    E=_spread(rng, 8, 896))
    G = rng.choice([1, 1, 2, 4, 8, 16])
    per = max(1, _spread(rng, 8, 896) // G)
    KG = rng.randint(1, G)
    return dict(op=op, T=_spread(rng, 1, 8192), E=G * per, K=rng.randint(1, min(32, KG * per)),
                G=G, KG=KG, score=rng.choice(["sigmoid", "softmax"]),
                group=rng.choice(["top2", "max"]), bias=rng.random() < 0.5,
                renorm=rng.random() < 0.5, masked=rng.choice([0.0, 0.0, 0.05, 0.5]))


def work(case):
    op = case["op"]
    if op == "norm":
        T, H = case["T"], case["H"]
        q = {"mxfp8": H + H // 32, "int8": H + 4, "none": 0}[case["q8"]]
        rows = 2 * H * (4 if case["residual"] else 2) + q   # x, residual, sum, y; 8-bit output
        return {"bytes": T * rows + 2 * H, "flops": 6 * T * H}
    if op in ("int8", "normed"):
        M, N, K = case["M"], case["N"], case["K"]
        b = 2 * M * K + N * K + 4 * N + (4 if case.get("out") == "f32" else 2) * M * N
        if op == "normed":
            b += 4 * M * K + 2 * K    # the residual read, the sum written, the norm's weight
        return {"bytes": b, "flops": 2 * M * N * K}
    if op == "gate":
        T, H, E = case["T"], case["H"], case["E"]
        return {"bytes": 2 * T * H + 2 * E * H + 4 * T * E, "flops": 2 * T * H * E}
    T, E, K = case["T"], case["E"], case["K"]
    return {"bytes": 4 * T * E + 8 * T * K + (4 * E if case["bias"] else 0), "flops": 10 * T * E}


def _tokens(T, H, g, dev):
    """Hidden states: normal, with a few channels much larger than the others."""
    x = torch.randn(T, H, generator=g, device=dev)
    big = torch.randint(0, H, (max(1, H // 512),), generator=g, device=dev)
    x[:, big] *= 8.0
    return x.to(BF16)


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    op, s = case["op"], dict(case)
    if op in ("norm", "normed"):
        T, H = (case["T"], case["H"]) if op == "norm" else (case["M"], case["K"])
        q8 = case["q8"] if op == "norm" else "int8"
        s["x"] = _tokens(T, H, g, dev)
        s["r"] = 2.0 * _tokens(T, H, g, dev) if case.get("residual", True) else None
        s["w"] = (1.0 + 0.1 * torch.randn(H, generator=g, device=dev)).to(BF16)
        s["h"] = torch.empty_like(s["x"]) if s["r"] is not None else None
        s["y"] = torch.empty_like(s["x"]) if op == "norm" else None
        if q8 == "mxfp8":
            s["xq"] = torch.empty(T, H, dtype=torch.uint8, device=dev)
            s["xs"] = torch.empty(T, H // 32, dtype=torch.uint8, device=dev)
        elif q8 == "int8":
            s["xq"] = torch.empty(T, H, dtype=torch.int8, device=dev)
            s["xs"] = torch.empty(T, dtype=F32, device=dev)
    if op in ("int8", "normed"):
        M, N, K = case["M"], case["N"], case["K"]
        if op == "int8":
            s["x"] = _tokens(M, K, g, dev)
        wf = 0.02 * torch.randn(N, K, generator=g, device=dev)
        s["w_s"] = wf.abs().amax(1) / 127.0
        s["wq"] = torch.round(wf / s["w_s"][:, None]).to(torch.int8)
        s["out"] = torch.empty(M, N, dtype=F32 if case.get("out") == "f32" else BF16, device=dev)
        if own:
            import mxfp8_mxfp4_experts_amd as m
            s["workspace"] = torch.empty(m.moe_int8_workspace_size(M, N, K), dtype=torch.uint8,
                                         device=dev)
    if op == "gate":
        T, H, E = case["T"], case["H"], case["E"]
        s["x"] = _tokens(T, H, g, dev)
        s["w"] = (torch.randn(E, H, generator=g, device=dev) / math.sqrt(H)).to(BF16)
        s["logits"] = torch.empty(T, E, dtype=F32, device=dev)
        if own:
            import mxfp8_mxfp4_experts_amd as m
            s["workspace"] = torch.empty(m.moe_gate_workspace_size(T, E, H), dtype=torch.uint8,
                                         device=dev)
    if op == "route":
        T, E, K = case["T"], case["E"], case["K"]
        s["logits"] = 1.5 * torch.randn(T, E, generator=g, device=dev)
        s["b"] = 0.1 * torch.randn(E, generator=g, device=dev) if case["bias"] else None
        if case["masked"]:
            # Experts that may not take a token: half of them by -inf, half by the lowest float;
            # and some tokens (padding) that no expert may take.
            hide = torch.rand(T, E, generator=g, device=dev) < case["masked"]
            hide |= torch.rand(T, 1, generator=g, device=dev) < case["masked"] / 10
            low = torch.where(torch.rand(T, E, generator=g, device=dev) < 0.5,
                              torch.tensor(LOWEST, device=dev), torch.tensor(-math.inf, device=dev))
            s["logits"] = torch.where(hide, low, s["logits"])
        s["idx"] = torch.empty(T, K, dtype=torch.int32, device=dev)
        s["wt"] = torch.empty(T, K, dtype=F32, device=dev)
    return s


def run(s):
    return _package(s) if own else _plain(s)


# ---------------------------------------------------------------------------
# The calls that a user of the package makes.

def _package(s):
    import mxfp8_mxfp4_experts_amd as m

    op = s["op"]
    if op == "norm":
        q8 = {"mxfp8": m.Q8_MXFP8, "int8": m.Q8_INT8, "none": m.Q8_NONE}[s["q8"]]
        m.moe_add_rmsnorm(s["x"], s["w"], EPS, residual=s["r"], q8=q8, residual_out=s["h"],
                          y=s["y"], xq=s.get("xq"), xs=s.get("xs"))
        out = {"h": s["h"], "y": s["y"]}
        if s["q8"] == "mxfp8":
            out["xq"] = s["xq"].view(torch.float8_e4m3fn)
            out["xs"] = s["xs"].view(torch.float8_e8m0fnu)
        elif s["q8"] == "int8":
            out["xq"], out["xs"] = s["xq"].to(BF16), s["xs"]
        return out
    if op == "normed":
        m.moe_add_rmsnorm(s["x"], s["w"], EPS, residual=s["r"], q8=m.Q8_INT8,
                          residual_out=s["h"], want_y=False, xq=s["xq"], xs=s["xs"])
        m.moe_int8_matmul(s["xq"], s["xs"], s["wq"], s["w_s"], out=s["out"],
                          workspace=s["workspace"])
        return {"h": s["h"], "out": s["out"]}
    if op == "int8":
        return m.moe_int8_linear(s["x"], s["wq"], s["w_s"], out=s["out"],
                                 workspace=s["workspace"])
    if op == "gate":
        return m.moe_gate_logits(s["x"], s["w"], out=s["logits"], workspace=s["workspace"])
    idx, wt = m.moe_route_groups(
        s["logits"], s["b"], s["K"], n_group=s["G"], topk_group=s["KG"],
        score=m.SCORE_SOFTMAX if s["score"] == "softmax" else m.SCORE_SIGMOID,
        group_score=m.GROUP_TOP2 if s["group"] == "top2" else m.GROUP_MAX,
        renormalise=s["renorm"], routed_scaling=1.0, topk_idx=s["idx"], topk_w=s["wt"])
    return {"idx": idx, "w": wt}


# ---------------------------------------------------------------------------
# The plain forms.

def _norm(x, r, w):
    """The float32 sum and its norm (rounded by the caller)."""
    h = x.float() if r is None else x.float() + r.float()
    y = h * torch.rsqrt(h.square().mean(1, keepdim=True) + EPS) * w.float()
    return h, y


def _mxfp8(y):
    """E4M3 values and E8M0 scales: per 32 elements the smallest 2^e with absmax <= 448 * 2^e."""
    g = y.view(y.shape[0], -1, 32)
    amax = g.abs().amax(2)
    m, p = torch.frexp(amax)                       # amax = m * 2^p, m in [0.5, 1)
    e = (p - 9 + (m > 0.875)).clamp(-127, 127)     # 448 = 0.875 * 2^9
    e = torch.where(amax < 2.0 ** -126, torch.full_like(e, -127), e)
    q = torch.ldexp(g, -e[..., None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
    return q.view(y.shape), (e + 127).to(torch.uint8).view(torch.float8_e8m0fnu)


def _int8(y):
    """Whole numbers of [-127, 127] (in float32) and a scale for each row."""
    # A tensor divides; a Python number would become a product with its rounded reciprocal, and
    # codes that fall between two whole numbers would go another way.
    s = (y.abs().amax(1) / torch.full((1,), 127.0, device=y.device)).clamp_min(2.0 ** -126)
    return torch.round(y * (1.0 / s)[:, None]).clamp(-127.0, 127.0), s


def _scores(logits, score, masked):
    """Each expert's score: evaluated in float64 and rounded once to float32, as routing defines
    it (the choice of experts compares these values, so both sides need the same ones)."""
    d = logits.double()
    if score == "sigmoid":
        return (1.0 / (1.0 + torch.exp(-d))).float()
    d = torch.where(masked, -math.inf, d)
    top = d.amax(1, keepdim=True)
    e = torch.exp(d - torch.where(top == -math.inf, torch.zeros_like(top), top))
    return (e / e.sum(1, keepdim=True).clamp_min(1e-300)).float()


def _route(s):
    logits, T, E, K, G, KG = s["logits"], s["T"], s["E"], s["K"], s["G"], s["KG"]
    masked = logits <= LOWEST
    score = _scores(logits, s["score"], masked)
    key = score if s["b"] is None else score + s["b"]
    key = torch.where(masked, -math.inf, key)
    if G > 1:
        best = key.view(T, G, E // G).sort(2, descending=True)[0]
        top = best[..., 0]
        if s["group"] == "top2" and E // G > 1:
            top = top + torch.where(best[..., 1] == -math.inf, 0.0, best[..., 1])
        rank = top.sort(dim=1, descending=True, stable=True)[1]
        keep = torch.zeros(T, G, dtype=torch.bool, device=key.device)
        keep.scatter_(1, rank[:, :KG], True)
        key = torch.where(keep.repeat_interleave(E // G, 1), key, -math.inf)
    val, idx = key.sort(dim=1, descending=True, stable=True)
    val, idx = val[:, :K], idx[:, :K]
    none = val == -math.inf
    w = torch.where(none, 0.0, score.gather(1, idx)).double()
    if s["renorm"]:
        total = w.sum(1, keepdim=True)
        w = torch.where(total > 0, w / total, 0.0)
    return {"idx": torch.where(none, -1, idx).to(torch.int32), "w": w.float()}


def _plain(s):
    op = s["op"]
    if op == "norm":
        h, y = _norm(s["x"], s["r"], s["w"])
        out = {"h": h.to(BF16) if s["r"] is not None else None, "y": y.to(BF16)}
        if s["q8"] == "mxfp8":
            out["xq"], out["xs"] = _mxfp8(y)
        elif s["q8"] == "int8":
            q, out["xs"] = _int8(y)
            out["xq"] = q.to(BF16)
        return out
    if op == "gate":
        return s["x"].float() @ s["w"].float().t()
    if op == "route":
        return _route(s)
    h = None
    if op == "normed":
        h, y = _norm(s["x"], s["r"], s["w"])
        h = h.to(BF16)
    else:
        y = s["x"].float()
    q, sx = _int8(y)
    out = ((q @ s["wq"].float().t()) * sx[:, None] * s["w_s"]).to(s["out"].dtype)
    return out if h is None else {"h": h, "out": out}


# ---------------------------------------------------------------------------
# The definitions in 64 bits.

def _norm64(s):
    h = s["x"].double() + (s["r"].double() if s["r"] is not None else 0.0)
    return h, h / torch.sqrt((h * h).sum(1, keepdim=True) / h.shape[1] + EPS) * s["w"].double()


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "norm":
        h, y = _norm64(s)
        out = {"h": h if s["r"] is not None else None, "y": y}
        if case["q8"] == "mxfp8":
            # What the 8 bits stand for: the values over their block's scale, before rounding.
            g = y.view(y.shape[0], -1, 32)
            e = torch.ceil(torch.log2(g.abs().amax(2) / 448.0)).clamp(-127, 127)
            out["xq"] = (g / torch.exp2(e)[..., None]).reshape(y.shape)
            out["xs"] = torch.exp2(e)
        elif case["q8"] == "int8":
            scale = y.abs().amax(1) / 127.0
            out["xq"], out["xs"] = y / scale[:, None], scale
        return out
    if op == "gate":
        return s["x"].double() @ s["w"].double().t()
    if op in ("int8", "normed"):
        h, y = _norm64(s) if op == "normed" else (None, s["x"].double())
        scale = y.abs().amax(1, keepdim=True) / 127.0
        q = torch.round(y / scale)
        out = (q @ s["wq"].double().t()) * scale * s["w_s"].double()
        return out if h is None else {"h": h, "out": out}
    # Routing, token by token of the definition but for all tokens at once: sums and comparisons
    # of the scores that float32 holds.
    logits, T, E, K, G, KG = s["logits"].double(), case["T"], case["E"], case["K"], case["G"], case["KG"]
    out_of_play = logits <= LOWEST
    if case["score"] == "sigmoid":
        score = torch.special.expit(logits)
    else:
        score = torch.softmax(torch.where(out_of_play, -math.inf, logits), 1).nan_to_num(0.0)
    score = score.to(F32)
    key = score + s["b"] if s["b"] is not None else score.clone()
    key[out_of_play] = -math.inf
    if G > 1:
        n = 2 if case["group"] == "top2" and E // G > 1 else 1
        best = key.view(T, G, -1).topk(n, 2)[0]
        worth = best[..., 0] + (best[..., 1].nan_to_num(neginf=0.0) if n == 2 else 0.0)
        # ranks with ties to the lower group: how many groups come before this one
        at = torch.arange(G, device=key.device)
        before = (worth[:, None, :] > worth[:, :, None]) | (
            (worth[:, None, :] == worth[:, :, None]) & (at[None, None, :] < at[None, :, None]))
        key[(before.sum(2) >= KG).repeat_interleave(E // G, 1)] = -math.inf
    order = torch.argsort(key, dim=1, descending=True, stable=True)[:, :K]
    gone = torch.isneginf(key.gather(1, order))
    w = score.double().gather(1, order).masked_fill(gone, 0.0)
    if case["renorm"]:
        w = (w / w.sum(1, keepdim=True)).nan_to_num(0.0)
    return {"idx": order.masked_fill(gone, -1).to(torch.int32), "w": w}
