"""Block-scaled FP8 products and the way of tokens into expert order and back, as cases that
can be timed and compared.

Two families around the grouping of tokens by expert (``moe_permute``): matrix products of
E4M3 codes with a float scale for each block of 128 (``moe_fp8_linear``, from bf16 tokens, and
``moe_quant_fp8`` with ``moe_fp8_grouped``, every expert's rows times that expert's weight);
and rows of tokens sorted by expert (``moe_sort_tokens``), brought back with the routing
weights applied (``moe_unsort_tokens``), and the gradients of both (``moe_unsort_tokens``
without weights, ``moe_unsort_tokens_grad``).

``own`` False computes each in its plain form (elementary torch operations), True calls the
package.  ``exact`` is each operator's definition in 64 bits.
"""
import math

import torch

own = False

BLOCK = 128                       # elements of K, and output columns, that share a scale
E4M3_MAX = 448.0
BF16, F32, F64, FP8 = torch.bfloat16, torch.float32, torch.float64, torch.float8_e4m3fn
TYPES = {"bf16": BF16, "f32": F32}


def listed():
    return [
        # One token of a decode step through a dense projection.
        dict(name="linear_decode_1", op="linear", M=1, N=3584, K=7168),
        # A large decode batch.
        dict(name="linear_batch_256", op="linear", M=256, N=3584, K=7168),
        # A ragged batch: odd output width, K not whole blocks.
        dict(name="linear_ragged_1000", op="linear", M=1000, N=2051, K=1040),
        # An 8K prefill chunk's projection.
        dict(name="linear_chunk_8192", op="linear", M=8192, N=3584, K=7168),
        # Gate and up of one GPU's experts, a decode step: few rows per expert.
        dict(name="grouped_decode_8", op="grouped", T=8, top_k=8, E=28, E_local=28, N=7168, K=3584,
             gather=True, skew=0.0),
        # Rows that are in expert order already (the down product), half the experts elsewhere,
        # some experts much busier than others, odd widths.
        dict(name="grouped_ragged_700", op="grouped", T=700, top_k=3, E=66, E_local=33, N=1027,
             K=1296, gather=False, skew=1.2),
        # A prefill chunk's tokens through one GPU's experts.
        dict(name="grouped_chunk_2048", op="grouped", T=2048, top_k=8, E=28, E_local=28, N=3584,
             K=3584, gather=True, skew=0.0),
        # A decode batch's tokens grouped and copied into expert order.
        dict(name="sort_decode_8", op="sort", T=8, top_k=16, E=896, E_local=896, H=7168,
             type="bf16", train=False),
        # The same of a prefill chunk.
        dict(name="sort_chunk_4096", op="sort", T=4096, top_k=8, E=28, E_local=28, H=3584,
             type="bf16", train=False),
        # A training step's share of an expert-parallel group: half the routes go elsewhere;
        # float rows of odd width, and the tokens' gradient.
        dict(name="sort_train_ragged", op="sort", T=1000, top_k=3, E=64, E_local=32, H=1037,
             type="f32", train=True),
        # A prefill chunk's rows back into token order, the routing weights applied.
        dict(name="unsort_chunk_8192", op="unsort", T=8192, top_k=8, E=28, E_local=28, H=3584,
             type="bf16", train=False),
        # A training step: the same, and the gradients of the rows and of the weights.
        dict(name="unsort_train_4096", op="unsort", T=4096, top_k=8, E=56, E_local=28, H=3584,
             type="bf16", train=True),
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], spread evenly over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["linear", "linear", "grouped", "grouped", "sort", "unsort"])
    if op == "linear":
        return dict(op=op, M=_spread(rng, 1, 8192), N=_spread(rng, 64, 3584),
                    K=16 * _spread(rng, 8, 448))
    # Experts here, and in all: as many, or two or four times as many.
    E_local = _spread(rng, 4, 64)
    E = E_local * rng.choice([1, 1, 2, 4])
    top_k = min(E, rng.randint(1, 8 if op == "grouped" else 16))
    if op == "grouped":
        # No more weights than the largest listed case has.
        K = 16 * _spread(rng, 8, 224)
        N = min(_spread(rng, 64, 3584), 28 * 7168 * 3584 // (E_local * K))
        return dict(op=op, T=_spread(rng, 1, 2048), top_k=top_k, E=E, E_local=E_local, N=N, K=K,
                    gather=rng.random() < 0.5, skew=rng.choice([0.0, 0.0, 1.2]))
    H = rng.choice([_spread(rng, 8, 3584), 8 * _spread(rng, 1, 448)])
    kind = rng.choice(["bf16", "f32"])
    # No more than the largest listed case moves.
    most = 8192 * 8 * 3584 // (2 if kind == "f32" else 1) // 2
    return dict(op=op, T=_spread(rng, 1, max(1, min(8192, most // (top_k * H)))), top_k=top_k, E=E,
                E_local=E_local, H=H, type=kind, train=rng.random() < 0.5)


def _blocks(n):
    return (n + BLOCK - 1) // BLOCK


def work(case):
    op = case["op"]
    if op == "linear":
        M, N, K = case["M"], case["N"], case["K"]
        return {"bytes": 2 * M * K + N * K + 4 * _blocks(N) * _blocks(K) + 2 * M * N,
                "flops": 2 * M * N * K}
    # The routes that stay here, and the experts that get any, as expected.
    T, k = case["T"], case["top_k"]
    share = case["E_local"] / case["E"]
    R = T * k * share
    if op == "grouped":
        N, K = case["N"], case["K"]
        touched = case["E_local"] * (1.0 - (1.0 - k / case["E"]) ** T)
        rows = T if case["gather"] else R
        b = 2 * rows * K + touched * (N * K + 4 * _blocks(N) * _blocks(K)) + 2 * R * N
        return {"bytes": int(b), "flops": int(2 * R * N * K)}
    row = case["H"] * (2 if case["type"] == "bf16" else 4)
    if op == "sort":
        b = 4 * T * k * 3 + T * row + R * row           # ids, sorted routes, rows of routes
        if case["train"]:
            b += R * row + T * row
        return {"bytes": int(b), "flops": int(R * case["H"]) if case["train"] else 0}
    b = 8 * T * k + R * row + T * row
    f = 2 * R * case["H"]
    if case["train"]:
        b += T * row + R * row + R * row + 4 * T * k
        f += 3 * R * case["H"]
    return {"bytes": int(b), "flops": int(f)}


# ---------------------------------------------------------------------------
# Inputs.

def _tokens(T, H, g, dev):
    """Hidden states: normal, with a few channels much larger than the others."""
    x = torch.randn(T, H, generator=g, device=dev)
    big = torch.randint(0, H, (max(1, H // 512),), generator=g, device=dev)
    x[:, big] *= 8.0
    return x


def _weight(E, N, K, g, dev):
    """A weight's E4M3 codes [E, N, K] and scales [E, N / 128, K / 128], block by block as a
    checkpoint's converter makes them."""
    codes = torch.empty(E, N, K, dtype=FP8, device=dev)
    scales = torch.empty(E, _blocks(N), _blocks(K), dtype=F32, device=dev)
    for e in range(E):
        w = torch.zeros(_blocks(N) * BLOCK, _blocks(K) * BLOCK, device=dev)
        w[:N, :K] = 0.02 * torch.randn(N, K, generator=g, device=dev)
        b = w.view(_blocks(N), BLOCK, _blocks(K), BLOCK)
        s = b.abs().amax((1, 3)) / E4M3_MAX
        codes[e] = (b / s[:, None, :, None]).view(w.shape)[:N, :K].to(FP8)
        scales[e] = s
    return codes, scales


def _route(case, g, dev):
    """Top-k ids of distinct experts per token, and weights that add up to one."""
    T, E, k = case["T"], case["E"], case["top_k"]
    # The larger of E random keys per token; with a skew some experts' keys are larger.
    key = -torch.log(-torch.log(torch.rand(T, E, generator=g, device=dev).clamp(1e-7, 1 - 1e-7)))
    if case.get("skew"):
        rank = torch.randperm(E, generator=g, device=dev) + 1
        key = key - case["skew"] * torch.log(rank.float())
    idx = key.sort(1, descending=True)[1][:, :k].to(torch.int32).contiguous()
    w = torch.sigmoid(torch.randn(T, k, generator=g, device=dev))
    return idx, (w / w.sum(1, keepdim=True)).contiguous()


def _window(case):
    """The first expert that is held here."""
    return (case["E"] - case["E_local"]) // 2


def _group(case, idx):
    """Expert offsets, the kept routes in expert order and every route's place among them."""
    R, E_local = idx.numel(), case["E_local"]
    local = idx.reshape(-1).long() - _window(case)
    kept = (idx.reshape(-1) >= 0) & (local >= 0) & (local < E_local)
    key = torch.where(kept, local, E_local)
    order = torch.sort(key, stable=True)[1]
    end = torch.cumsum((key[:, None] == torch.arange(E_local, device=idx.device)).sum(0), 0)
    offsets = torch.cat([torch.zeros(1, dtype=end.dtype, device=idx.device), end])
    at = torch.arange(R, device=idx.device)
    here = at < end[-1]
    sorted_route = torch.where(here, order, -1)
    route_row = torch.empty_like(order)
    route_row[order] = torch.where(here, at, -1)
    return (offsets.to(torch.int32), sorted_route.to(torch.int32), route_row.to(torch.int32))


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    op, s = case["op"], dict(case)
    if op == "linear":
        M, N, K = case["M"], case["N"], case["K"]
        s["x"] = _tokens(M, K, g, dev).to(BF16)
        w, w_s = _weight(1, N, K, g, dev)
        s["w"], s["w_s"] = w[0], w_s[0]
        s["out"] = torch.empty(M, N, dtype=BF16, device=dev)
        if own:
            import mxfp8_mxfp4_experts_amd as m
            s["workspace"] = torch.empty(m.moe_fp8_workspace_size(M, N, K), dtype=torch.uint8,
                                         device=dev)
        return s
    idx, wt = _route(case, g, dev)
    R = idx.numel()
    if op == "sort":
        # The grouping is part of the sort.
        s["idx"] = idx
        s["offsets"] = torch.empty(case["E_local"] + 1, dtype=torch.int32, device=dev)
        s["sorted_route"] = torch.empty(R, dtype=torch.int32, device=dev)
        s["route_row"] = torch.empty(R, dtype=torch.int32, device=dev)
        if own:
            import mxfp8_mxfp4_experts_amd as m
            s["workspace"] = torch.empty(m.moe_workspace_size(case["T"], case["top_k"],
                                                              case["E_local"], 128, 128),
                                         dtype=torch.uint8, device=dev)
    else:
        s["offsets"], s["sorted_route"], s["route_row"] = _group(case, idx)
    if op == "grouped":
        N, K = case["N"], case["K"]
        rows = case["T"] if case["gather"] else R
        s["x"] = _tokens(rows, K, g, dev).to(BF16)
        s["w"], s["w_s"] = _weight(case["E_local"], N, K, g, dev)
        s["xq"] = torch.empty(rows, K, dtype=torch.uint8, device=dev)
        s["xs"] = torch.empty(_blocks(K), rows, dtype=F32, device=dev)
        # Rows behind the last expert's are not written: zeros stay.
        s["out"] = torch.zeros(R, N, dtype=BF16, device=dev)
        return s
    T, H, kind = case["T"], case["H"], TYPES[case["type"]]
    if op == "sort":
        s["x"] = _tokens(T, H, g, dev).to(kind)
        s["rows"] = torch.zeros(R, H, dtype=kind, device=dev)
        if case["train"]:
            s["drows"] = torch.randn(R, H, generator=g, device=dev).to(kind)
            s["dx"] = torch.empty(T, H, dtype=kind, device=dev)
        return s
    s["wt"] = wt
    s["rows"] = _tokens(R, H, g, dev).to(kind)
    s["out"] = torch.empty(T, H, dtype=kind, device=dev)
    if case["train"]:
        s["dout"] = torch.randn(T, H, generator=g, device=dev).to(kind)
        s["drows"] = torch.zeros(R, H, dtype=kind, device=dev)
        s["dw"] = torch.empty(T, case["top_k"], dtype=F32, device=dev)
    return s


def run(s):
    return _package(s) if own else _plain(s)


# ---------------------------------------------------------------------------
# The calls that a user of the package makes.

def _package(s):
    import mxfp8_mxfp4_experts_amd as m

    op = s["op"]
    if op == "linear":
        return m.moe_fp8_linear(s["x"], s["w"], s["w_s"], out=s["out"], workspace=s["workspace"])
    if op == "grouped":
        m.moe_quant_fp8(s["x"], xq=s["xq"], xs=s["xs"])
        return m.moe_fp8_grouped(s["xq"], s["xs"], s["w"], s["w_s"], s["offsets"],
                                 sorted_route=s["sorted_route"] if s["gather"] else None,
                                 top_k=s["top_k"], out=s["out"])
    if op == "sort":
        m.moe_permute(s["idx"], _window(s), s["E_local"], s["workspace"], s["offsets"],
                      s["sorted_route"], s["route_row"])
        out = {"offsets": s["offsets"], "sorted_route": s["sorted_route"],
               "route_row": s["route_row"],
               "rows": m.moe_sort_tokens(s["x"], s["route_row"], s["top_k"], rows=s["rows"])}
        if s["train"]:
            out["dx"] = m.moe_unsort_tokens(s["drows"], s["route_row"], None, s["top_k"],
                                            out=s["dx"])
        return out
    out = {"out": m.moe_unsort_tokens(s["rows"], s["route_row"], s["wt"], s["top_k"],
                                      out=s["out"])}
    if s["train"]:
        out["drows"], out["dw"] = m.moe_unsort_tokens_grad(s["dout"], s["rows"], s["route_row"],
                                                           s["wt"], drows=s["drows"], dw=s["dw"])
    return out


# ---------------------------------------------------------------------------
# The plain forms.

def _quantised(x):
    """What the tokens' codes stand for: codes times scale, in float32."""
    T, K = x.shape
    f = torch.zeros(T, _blocks(K) * BLOCK, device=x.device)
    f[:, :K] = x
    f = f.view(T, _blocks(K), BLOCK)
    # A tensor divides; a Python number would become a product with its rounded reciprocal.
    top = torch.full((1,), E4M3_MAX, device=x.device)
    scale = (f.abs().amax(2, keepdim=True) / top).clamp_min(2.0 ** -126)
    q = (f * (1.0 / scale)).clamp(-E4M3_MAX, E4M3_MAX).to(FP8).float()
    return (q * scale).view(T, -1)[:, :K]


def _dequantised(w, w_s):
    N, K = w.shape
    s = w_s.repeat_interleave(BLOCK, 0)[:N].repeat_interleave(BLOCK, 1)[:, :K]
    return w.float() * s


def _plain(s):
    op = s["op"]
    if op == "linear":
        return (_quantised(s["x"]) @ _dequantised(s["w"], s["w_s"]).t()).to(BF16)
    k = s["top_k"]
    if op == "grouped":
        x = _quantised(s["x"])
        out = torch.zeros_like(s["out"])
        at = s["offsets"].tolist()
        for e in range(s["E_local"]):
            if at[e + 1] > at[e]:
                rows = (x[(s["sorted_route"][at[e]:at[e + 1]] // k).long()] if s["gather"]
                        else x[at[e]:at[e + 1]])
                out[at[e]:at[e + 1]] = (rows @ _dequantised(s["w"][e], s["w_s"][e]).t()).to(BF16)
        return out
    if op == "sort":
        offsets, sorted_route, row = _group(s, s["idx"])
        here = (sorted_route >= 0)[:, None]
        rows = torch.where(here, s["x"][(sorted_route.clamp_min(0) // k).long()], 0)
        out = {"offsets": offsets, "sorted_route": sorted_route, "route_row": row, "rows": rows}
        if s["train"]:
            out["dx"] = _back(s["drows"], row, None, k)
        return out
    row = s["route_row"]
    out = {"out": _back(s["rows"], row, s["wt"], k)}
    if s["train"]:
        T = row.numel() // k
        token = (s["sorted_route"].clamp_min(0) // k).long()
        here = s["sorted_route"] >= 0
        w = s["wt"].reshape(-1)[s["sorted_route"].clamp_min(0).long()]
        given = s["dout"].float()[token]
        out["drows"] = torch.where(here[:, None], w[:, None] * given, 0.0).to(s["rows"].dtype)
        dot = (given * s["rows"].float()).sum(1)
        out["dw"] = torch.where(row >= 0, dot[row.clamp_min(0).long()], 0.0).view(T, k)
    return out


def _back(rows, row, wt, k):
    """Each token's kept rows, weighted, added in float32."""
    T = row.numel() // k
    row = row.view(T, k)
    out = torch.zeros(T, rows.shape[1], device=rows.device)
    for j in range(k):
        here = (row[:, j] >= 0)[:, None]
        part = rows[row[:, j].clamp_min(0).long()].float()
        if wt is not None:
            part = part * wt[:, j, None]
        out += torch.where(here, part, 0.0)
    return out.to(rows.dtype)


# ---------------------------------------------------------------------------
# The definitions in 64 bits.

def _quantised64(x):
    """The nearest E4M3 numbers to the tokens over their block's scale, times the scale."""
    parts = []
    for f in x.double().split(BLOCK, 1):
        scale = (f.abs().amax(1, keepdim=True) / E4M3_MAX).clamp_min(2.0 ** -126)
        v = f / scale
        # E4M3's steps: an eighth of the power of two at or below |v|, 2^-9 below 2^-6.
        step = torch.exp2(torch.floor(torch.log2(v.abs().clamp_min(2.0 ** -6))) - 3.0)
        parts.append(torch.round(v / step) * step * scale)
    return torch.cat(parts, 1)


def _weight64(w, w_s):
    out = w.to(F32).double()
    for i in range(w_s.shape[0]):
        for j in range(w_s.shape[1]):
            out[i * BLOCK:(i + 1) * BLOCK, j * BLOCK:(j + 1) * BLOCK] *= w_s[i, j].double()
    return out


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "linear":
        return torch.matmul(_quantised64(s["x"]), _weight64(s["w"], s["w_s"]).t())
    k = case["top_k"]
    if op == "grouped":
        x = _quantised64(s["x"])
        out = torch.zeros(s["out"].shape, dtype=F64, device=x.device)
        ends = s["offsets"].tolist()
        for e, (a, b) in enumerate(zip(ends, ends[1:])):
            if a == b:
                continue
            mine = torch.arange(a, b, device=x.device)
            if case["gather"]:
                mine = torch.div(s["sorted_route"][a:b].long(), k, rounding_mode="floor")
            out[a:b] = torch.matmul(x[mine], _weight64(s["w"][e], s["w_s"][e]).t())
        return out
    T, H = case["T"], case["H"]
    if op == "sort":
        # Expert by expert: its routes in order.
        ids = s["idx"].reshape(-1)
        first, lists = _window(case), []
        for e in range(case["E_local"]):
            lists.append(torch.nonzero(ids == first + e)[:, 0])
        routes = torch.cat(lists)
        n = routes.numel()
        ends = torch.tensor([0] + [v.numel() for v in lists]).cumsum(0)
        order = torch.full((T * k,), -1, dtype=torch.int32, device=ids.device)
        order[:n] = routes.to(torch.int32)
        place = torch.full((T * k,), -1, dtype=torch.int32, device=ids.device)
        place[routes] = torch.arange(n, dtype=torch.int32, device=ids.device)
        rows = torch.zeros(T * k, H, dtype=F64, device=ids.device)
        rows[:n] = s["x"].double()[torch.div(routes, k, rounding_mode="floor")]
        out = {"offsets": ends.to(torch.int32).to(ids.device), "sorted_route": order,
               "route_row": place, "rows": rows}
        if case["train"]:
            dx = torch.zeros(T, H, dtype=F64, device=ids.device)
            token = torch.div(routes, k, rounding_mode="floor")
            out["dx"] = dx.index_add_(0, token, s["drows"][:n].double())
        return out
    routes = s["sorted_route"][s["sorted_route"] >= 0].long()
    n, token = routes.numel(), torch.div(routes, k, rounding_mode="floor")
    w = s["wt"].double().reshape(-1)[routes]
    rows = s["rows"][:n].double()
    out = torch.zeros(T, H, dtype=F64, device=rows.device)
    out = {"out": out.index_add_(0, token, w[:, None] * rows)}
    if case["train"]:
        dout = s["dout"].double()[token]
        drows = torch.zeros(T * k, H, dtype=F64, device=rows.device)
        drows[:n] = w[:, None] * dout
        dw = torch.zeros(T * k, dtype=F64, device=rows.device)
        dw[routes] = torch.einsum("rh,rh->r", dout, rows)
        out["drows"], out["dw"] = drows, dw.view(T, k)
    return out
