"""Tokens into expert order and back: refusals (no GPU needed), the forward and backward calls
against 64-bit references and differences, and a run through grouped FP8 experts."""
import math
import os

import pytest
import torch

import fp8_ref as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "mxfp8_mxfp4_experts_amd", "libmi355moe.so")
pytestmark = pytest.mark.skipif(not os.path.exists(LIB), reason="libmi355moe.so not built")
gpu = pytest.mark.gpu

FAKE = 1 << 20          # aligned, never dereferenced by a failing call
OK, NULL, SHAPE, ALIGN, ENUM = 0, 1, 2, 3, 4
BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64
NAN, INF = math.nan, math.inf
DEV = "cuda"


@pytest.fixture(scope="module")
def lib():
    from mxfp8_mxfp4_experts_amd import _binding
    return _binding.load_library(LIB)


@pytest.fixture(scope="module")
def m():
    import mxfp8_mxfp4_experts_amd as m
    return m


# ---------------------------------------------------------------------------
# Refusals: the C entries check before any HIP call.

BAD_SHAPES = (dict(T=-1), dict(H=0), dict(H=(1 << 20) + 1, ld=1 << 21, ldr=1 << 21), dict(k=0),
              dict(k=65), dict(T=1 << 25, k=64), dict(n=-1), dict(n=(1 << 30) + 1), dict(ld=8),
              dict(ldr=8))


def test_sort_refusals(lib):
    def call(x=FAKE, ld=9, T=4, H=9, k=2, rr=FAKE, kind=0, rows=FAKE, ldr=9, n=8):
        return lib.moe_sort_tokens(x, ld, T, H, k, rr, kind, rows, ldr, n, None)
    for bad in BAD_SHAPES:
        assert call(**bad) == SHAPE, bad
    assert call(kind=2) == ENUM and call(kind=-1) == ENUM
    for name in ("x", "rr", "rows"):
        assert call(**{name: None}) == NULL
        assert call(**{name: FAKE + 1}) == ALIGN
    assert call(kind=1, x=FAKE + 2) == ALIGN and call(kind=1, rows=FAKE + 2) == ALIGN
    assert call(T=0, x=None, rr=None) == OK and call(n=0, rows=None) == OK


def test_unsort_refusals(lib):
    def call(rows=FAKE, ldr=9, n=8, T=4, H=9, k=2, rr=FAKE, w=FAKE, kind=0, out=FAKE, ld=9):
        return lib.moe_unsort_tokens(rows, ldr, n, T, H, k, rr, w, kind, out, ld, None)
    for bad in BAD_SHAPES:
        assert call(**bad) == SHAPE, bad
    assert call(kind=2) == ENUM
    for name in ("rows", "rr", "out"):
        assert call(**{name: None}) == NULL
    for name in ("rows", "rr", "out", "w"):
        assert call(**{name: FAKE + 1}) == ALIGN
    assert call(T=0, rows=None, out=None) == OK


def test_unsort_grad_refusals(lib):
    def call(dout=FAKE, ld=9, rows=FAKE, ldr=9, n=8, T=4, H=9, k=2, rr=FAKE, w=FAKE, kind=0,
             drows=FAKE, ldd=9, dw=FAKE):
        return lib.moe_unsort_tokens_grad(dout, ld, rows, ldr, n, T, H, k, rr, w, kind, drows, ldd,
                                          dw, None)
    for bad in BAD_SHAPES + (dict(ldd=8),):
        assert call(**bad) == SHAPE, bad
    assert call(kind=2) == ENUM
    for bad in (dict(dout=None), dict(rows=None), dict(rr=None), dict(w=None),
                dict(drows=None, dw=None)):
        assert call(**bad) == NULL, bad
    for name in ("dout", "rows", "rr", "w", "drows", "dw"):
        assert call(**{name: FAKE + 1}) == ALIGN, name
    assert call(T=0, dout=None) == OK


# ---------------------------------------------------------------------------
# On the GPU.

def routes(T, k, E, seed, kind):
    g = torch.Generator().manual_seed(seed)
    if kind == "none":
        return torch.full((T, k), -1, dtype=torch.int32, device=DEV)
    idx = torch.randint(0, E, (T, k), generator=g) if k > E or kind == "repeats" else \
        torch.rand(T, E, generator=g).argsort(1)[:, :k]
    if kind == "masked":
        idx = torch.where(torch.rand(T, k, generator=g) < 0.4, -1, idx)
        idx[T // 2] = -1                            # a token without an expert
    return idx.to(torch.int32).contiguous().to(DEV)


def grouped(m, T, k, E, E_local, seed, kind):
    idx = routes(T, k, E, seed, kind)
    ws = torch.empty(m.moe_workspace_size(T, k, E_local, 128, 128), dtype=torch.uint8, device=DEV)
    offs, sorted_route, route_row = m.moe_permute(idx, (E - E_local) // 2, E_local, ws)
    return int(offs[-1]), sorted_route, route_row


def values(shape, kind, seed):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g)).to(kind).to(DEV)


def step(kind):
    """Half a step of a type, relative."""
    return torch.finfo(kind).eps / 2


CASES = [
    # T, top_k, E, E_local, H, routing
    (1, 1, 1, 1, 1, ""), (1, 16, 32, 32, 7168, ""), (2, 3, 5, 5, 3, ""), (3, 2, 4, 2, 7, ""),
    (5, 4, 8, 4, 8, "masked"), (7, 5, 9, 9, 9, ""), (9, 8, 16, 16, 17, ""), (33, 9, 12, 6, 65, ""),
    (40, 3, 6, 3, 512, "masked"), (64, 2, 3, 3, 513, ""), (100, 17, 30, 10, 1037, ""),
    (20, 64, 64, 40, 130, ""), (50, 4, 4, 4, 2050, "repeats"), (12, 3, 8, 8, 40, "none"),
    (1000, 8, 28, 28, 520, ""), (3000, 2, 64, 8, 72, ""),
    (4200, 8, 28, 28, 1301, ""), (5000, 7, 20, 10, 1025, "masked"),   # past the caches
]


@gpu
@pytest.mark.parametrize("kind", [BF16, F32])
@pytest.mark.parametrize("T,k,E,E_local,H,how", CASES)
def test_forward_and_gradients(m, T, k, E, E_local, H, how, kind):
    R = T * k
    n, sorted_route, row = grouped(m, T, k, E, E_local, T + H, how)
    here = (row >= 0).view(T, k)
    at = row.view(T, k).long().clamp_min(0)
    x = values((T, H), kind, 1)
    # Into expert order, other rows left as they were.
    rows = torch.full((R, H), 7.0, dtype=kind, device=DEV)
    assert m.moe_sort_tokens(x, row, k, rows=rows) is rows
    assert torch.equal(rows[:n], x[(sorted_route[:n] // k).long()])
    assert (rows[n:] == 7.0).all()
    # Back with weights, and without.
    y = values((R, H), kind, 2)
    y[n:] = NAN                                    # no route has these
    w = values((T, k), F32, 3)
    for weights in (w, None):
        out = m.moe_unsort_tokens(y, row, weights, k)
        each = torch.where(here[..., None], y.double()[at], 0.0)
        if weights is not None:
            each = each * w.double()[..., None]
        want = each.sum(1)
        # k products and sums in float, one rounding to the rows' type.
        tol = want.abs() * step(kind) * 1.01 + each.abs().sum(1) * (k + 1) * 2.0 ** -24 + 1e-38
        assert ((out.double() - want).abs() <= tol).all()
    # Gradients of the weighted way back.
    dout = values((T, H), kind, 4)
    drows = torch.full((R, H), 7.0, dtype=kind, device=DEV)
    got, dw = m.moe_unsort_tokens_grad(dout, y, row, w, drows=drows)
    assert got is drows and (drows[n:] == 7.0).all()
    route = sorted_route[:n].long()
    want = w.view(-1)[route].double()[:, None] * dout.double()[route // k]
    assert ((drows[:n].double() - want).abs() <=
            want.abs() * (step(kind) * 1.01 + 2.0 ** -24) + 1e-38).all()
    terms = torch.where(here[..., None], y.double()[at], 0.0) * dout.double()[:, None, :]
    # A lane adds every 256th piece in turn, then 64 lanes and 4 wavefronts.
    chain = (H // 256 + 8) + 12
    assert ((dw.double() - terms.sum(2)).abs() <=
            terms.abs().sum(2) * chain * 2.0 ** -24 + 1e-38).all()
    assert (dw[~here] == 0).all()
    # Either alone gives the same bits.
    assert m.moe_unsort_tokens_grad(dout, y, row, w, want_drows=False)[0] is None
    assert torch.equal(m.moe_unsort_tokens_grad(dout, y, row, w, want_drows=False)[1], dw)
    alone, none = m.moe_unsort_tokens_grad(dout, y, row, w, want_dw=False)
    assert none is None and torch.equal(alone[:n], drows[:n])


@gpu
@pytest.mark.parametrize("H", [24, 1037])
def test_gradients_against_differences(m, H):
    """<dout, out> is linear in the weights, in each row and in each token: the difference that a
    step of one gives, in float rows."""
    T, k, E = 19, 3, 6
    n, _, row = grouped(m, T, k, E, 4, 1, "masked")
    y, w, dout = values((T * k, H), F32, 1), values((T, k), F32, 2), values((T, H), F32, 3)
    drows, dw = m.moe_unsort_tokens_grad(dout, y, row, w)

    def loss(y, w):
        return (m.moe_unsort_tokens(y, row, w, k).double() * dout.double()).sum().item()
    mag = (m.moe_unsort_tokens(y.abs(), row, w.abs() + 1, k).double() * dout.double().abs()).sum()
    tol = 2 * mag.item() * (k + 2) * 2.0 ** -24
    for t in range(T):
        for j in range(k):
            step = torch.zeros_like(w)
            step[t, j] = 1.0
            diff = (loss(y, w + step) - loss(y, w - step)) / 2
            assert abs(diff - dw[t, j].item()) <= tol + 1e-5 * abs(diff)
    for r in range(0, n, 7):
        for h in (0, H // 2, H - 1):
            step = torch.zeros_like(y)
            step[r, h] = 1.0
            diff = (loss(y + step, w) - loss(y - step, w)) / 2
            assert abs(diff - drows[r, h].item()) <= tol + 1e-5 * abs(diff)
    # The sort's gradient: <drows, sort(x)> in x.
    x, drows = values((T, H), F32, 5), values((T * k, H), F32, 6)
    dx = m.moe_unsort_tokens(drows, row, None, k)
    for t in range(0, T, 3):
        e = torch.zeros_like(x)
        e[t, H // 3] = 1.0
        moved = m.moe_sort_tokens(e, row, k, rows=torch.zeros_like(drows))
        diff = (moved.double() * drows.double()).sum().item()
        assert abs(diff - dx[t, H // 3].item()) <= (k + 1) * 2.0 ** -24 * 10


@gpu
@pytest.mark.parametrize("kind", [BF16, F32])
@pytest.mark.parametrize("H", [5, 136, 1001])
def test_strides_and_any_start(m, H, kind):
    """Windows of wider buffers, starting at any element: the columns outside stay."""
    T, k = 21, 3
    n, _, row = grouped(m, T, k, 8, 5, 2, "masked")

    def window(t, start, pad):
        wide = torch.full((t.shape[0], H + pad), 7.0, dtype=kind, device=DEV)
        view = wide[:, start:start + H]
        view.copy_(t)
        return wide, view
    x, y, dout = values((T, H), kind, 1), values((T * k, H), kind, 2), values((T, H), kind, 3)
    w = values((T, k), F32, 4)
    for start, pad in ((1, 3), (3, 8), (8, 16)):
        zero = torch.zeros(T * k, H, dtype=kind, device=DEV)
        wide, rows = window(zero, start, pad)
        m.moe_sort_tokens(window(x, start, pad + 5)[1], row, k, rows=rows)
        assert torch.equal(rows, m.moe_sort_tokens(x, row, k, rows=zero.clone()))
        wide_o, out = window(x, start, pad)
        m.moe_unsort_tokens(window(y, start, pad)[1], row, w, k, out=out)
        assert torch.equal(out, m.moe_unsort_tokens(y, row, w, k))
        wide_d, drows = window(zero, start, pad)
        _, dw = m.moe_unsort_tokens_grad(window(dout, start, pad)[1], window(y, start, pad)[1],
                                         row, w, drows=drows)
        want, want_w = m.moe_unsort_tokens_grad(dout, y, row, w, drows=zero.clone())
        assert torch.equal(drows, want) and torch.equal(dw, want_w)
        for b in (wide, wide_o, wide_d):
            assert (b[:, :start] == 7).all() and (b[:, start + H:] == 7).all()


@gpu
@pytest.mark.parametrize("kind", [BF16, F32])
def test_fewer_rows_and_wrong_places(m, kind):
    """A buffer of the kept rows only serves; a place past the buffer or below zero has no part."""
    T, k, H = 30, 4, 100
    n, _, row = grouped(m, T, k, 8, 4, 2, "")
    assert 0 < n < T * k
    x, y, dout = values((T, H), kind, 1), values((T * k, H), kind, 2), values((T, H), kind, 3)
    w = values((T, k), F32, 4)
    rows = m.moe_sort_tokens(x, row, k, rows=torch.empty(n, H, dtype=kind, device=DEV))
    assert torch.equal(rows, m.moe_sort_tokens(x, row, k)[:n])
    assert torch.equal(m.moe_unsort_tokens(y[:n], row, w, k), m.moe_unsort_tokens(y, row, w, k))
    a, b = m.moe_unsort_tokens_grad(dout, y[:n], row, w)
    c, d = m.moe_unsort_tokens_grad(dout, y, row, w)
    assert a.shape == (n, H) and torch.equal(a, c[:n]) and torch.equal(b, d)
    odd = row.clone()
    odd[row == 0], odd[row == 1] = 1 << 29, -(1 << 30)
    gone = torch.where((row == 0) | (row == 1), -1, row)
    guard = torch.full((n, H), 7.0, dtype=kind, device=DEV)
    assert torch.equal(m.moe_sort_tokens(x, odd, k, rows=guard.clone()),
                       m.moe_sort_tokens(x, gone, k, rows=guard.clone()))
    assert torch.equal(m.moe_unsort_tokens(y, odd, w, k), m.moe_unsort_tokens(y, gone, w, k))
    a, b = m.moe_unsort_tokens_grad(dout, y, odd, w, drows=guard.clone().new_zeros(T * k, H))
    c, d = m.moe_unsort_tokens_grad(dout, y, gone, w, drows=guard.clone().new_zeros(T * k, H))
    assert torch.equal(a, c) and torch.equal(b, d)
    none = torch.empty(0, H, dtype=kind, device=DEV)
    assert (m.moe_unsort_tokens(none, row, w, k) == 0).all()
    assert m.moe_sort_tokens(x, row, k, rows=none).shape == (0, H)
    assert (m.moe_unsort_tokens_grad(dout, none, row, w)[1] == 0).all()
    empty = row[:0]
    assert m.moe_unsort_tokens(y, empty, w[:0], k).shape == (0, H)
    assert m.moe_sort_tokens(x[:0], empty, k).shape == (0, H)


@gpu
def test_odd_values_stay_in_their_token(m):
    """An infinity or NaN in one row reaches its token only; rows of dropped routes reach none."""
    T, k, H = 17, 3, 200
    n, sorted_route, row = grouped(m, T, k, 6, 4, 3, "masked")
    y, w, dout = values((T * k, H), BF16, 1), values((T, k), F32, 2), values((T, H), BF16, 3)
    y[n:] = NAN
    plain = m.moe_unsort_tokens(y, row, w, k)
    assert torch.isfinite(plain).all()
    y[4, 7], y[9, 100] = INF, NAN
    out = m.moe_unsort_tokens(y, row, w, k)
    hit = torch.zeros(T, H, dtype=torch.bool, device=DEV)
    hit[sorted_route[4] // k, 7] = True
    hit[sorted_route[9] // k, 100] = True
    assert torch.equal(~torch.isfinite(out), hit)
    assert torch.equal(out[~hit], plain[~hit])
    _, dw = m.moe_unsort_tokens_grad(dout, y, row, w)
    bad = torch.zeros(T * k, dtype=torch.bool, device=DEV)
    bad[sorted_route[4].long()], bad[sorted_route[9].long()] = True, True
    assert torch.equal(~torch.isfinite(dw.view(-1)), bad)


@gpu
def test_rows_far_apart(m):
    """Row strides that pass 2^31 elements from the first row to the last."""
    T, k, H = 3, 2, 136
    n, _, row = grouped(m, T, k, 4, 4, 2, "")
    assert n == T * k
    far = (1 << 31) // (n - 1) + 8
    x, w = values((T, H), BF16, 1), values((T, k), F32, 2)
    big = torch.empty(far * (n - 1) + H, dtype=BF16, device=DEV).as_strided((n, H), (far, 1))
    near = m.moe_sort_tokens(x, row, k)
    assert torch.equal(m.moe_sort_tokens(x, row, k, rows=big), near)
    assert torch.equal(m.moe_unsort_tokens(big, row, w, k), m.moe_unsort_tokens(near, row, w, k))
    dout = values((T, H), BF16, 3)
    a, b = m.moe_unsort_tokens_grad(dout, near, row, w)
    c, d = m.moe_unsort_tokens_grad(dout, big, row, w)
    assert torch.equal(a, c) and torch.equal(b, d)
    assert torch.equal(m.moe_unsort_tokens_grad(dout, near, row, w, drows=big)[0], a)


@gpu
@pytest.mark.parametrize("T", [3, 500])
def test_graphs_and_streams(m, T):
    k, H = 4, 264
    n, _, row = grouped(m, T, k, 16, 16, 2, "")
    x, w = values((T, H), BF16, 1), values((T, k), F32, 2)
    rows, out = torch.empty(T * k, H, dtype=BF16, device=DEV), torch.empty_like(x)
    drows, dw = torch.empty_like(rows), torch.empty_like(w)

    def run():
        m.moe_sort_tokens(x, row, k, rows=rows)
        m.moe_unsort_tokens(rows, row, w, k, out=out)
        m.moe_unsort_tokens_grad(x, rows, row, w, drows=drows, dw=dw)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        run()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for seed in range(4):
        x.copy_(values((T, H), BF16, seed + 5))
        run()
        want = [t.clone() for t in (rows, out, drows, dw)]
        for t in (rows, out, drows, dw):
            t.fill_(NAN)
        graph.replay()
        torch.cuda.synchronize()
        for got, t in zip((rows, out, drows, dw), want):
            assert torch.equal(got, t)


@gpu
def test_binding_refusals(m):
    T, k, H = 4, 2, 40
    _, _, row = grouped(m, T, k, 4, 4, 2, "")
    x, y, w = values((T, H), BF16, 1), values((T * k, H), BF16, 2), values((T, k), F32, 3)
    bad = [
        lambda: m.moe_sort_tokens(x.half(), row, k), lambda: m.moe_sort_tokens(x, row[:7], k),
        lambda: m.moe_sort_tokens(x, row.long(), k), lambda: m.moe_sort_tokens(x.cpu(), row, k),
        lambda: m.moe_sort_tokens(x, row, k, rows=y.float()),
        lambda: m.moe_sort_tokens(x, row, k, rows=y[:, :39]), lambda: m.moe_sort_tokens(x, row, 0),
        lambda: m.moe_sort_tokens(x.t(), row, k),
        lambda: m.moe_unsort_tokens(y, row, w.double(), k),
        lambda: m.moe_unsort_tokens(y, row, w[:3], k), lambda: m.moe_unsort_tokens(y, row, w, 3),
        lambda: m.moe_unsort_tokens(y, row, w, k, out=x.float()),
        lambda: m.moe_unsort_tokens_grad(x, y.float(), row, w),
        lambda: m.moe_unsort_tokens_grad(x, y, row, w.view(-1)),
        lambda: m.moe_unsort_tokens_grad(x, y, row, w, drows=y[:3]),
        lambda: m.moe_unsort_tokens_grad(x, y, row, w, dw=w.view(-1)),
    ]
    for i, f in enumerate(bad):
        with pytest.raises(ValueError):
            f()
            pytest.fail(f"call {i} was taken")
    for f in (lambda: m.moe_unsort_tokens_grad(x[:1].expand(T, H), y, row, w),
              lambda: m.moe_unsort_tokens_grad(x, y, row, w, want_drows=False, want_dw=False)):
        with pytest.raises(m.MoEError):
            f()


# ---------------------------------------------------------------------------
# Together: a chunk through experts in FP8, as they would be used.

def situ(gate, up, alpha=4.0, beta=25.0):
    return (alpha * torch.tanh(gate / alpha) * torch.sigmoid(gate)) * (beta * torch.tanh(up / beta))


@gpu
@pytest.mark.parametrize("T,k,E,E_local", [(5, 4, 16, 16), (300, 3, 12, 6)])
def test_fp8_experts_from_routing_to_output(m, T, k, E, E_local):
    """Routing, grouping, tokens in FP8, gate and up of every expert, the activation, down, and the
    weighted way back: each step against 64 bits on the step's own inputs, and all of it with the
    tokens copied into expert order first."""
    H, I = 272, 144
    first = (E - E_local) // 2
    x = ref.tokens(T, H, 1).to(DEV)
    logits = values((T, E), F32, 2)
    w13, s13 = (t.to(DEV) for t in ref.weight(2 * I, H, 3, E_local, 0.3))
    w2, s2 = (t.to(DEV) for t in ref.weight(H, I, 4, E_local, 0.3))
    idx, w = m.moe_route_groups(logits, None, k)
    ws = torch.empty(m.moe_workspace_size(T, k, E_local, 128, 128), dtype=torch.uint8, device=DEV)
    offs, sorted_route, row = m.moe_permute(idx, first, E_local, ws)
    at = offs.tolist()
    n = at[-1]
    xq, xs = m.moe_quant_fp8(x)
    gu = m.moe_fp8_grouped(xq, xs, w13, s13, offs, sorted_route, k)
    h = torch.zeros(T * k, I, dtype=BF16, device=DEV)
    h[:n] = situ(gu[:n, :I].float(), gu[:n, I:].float()).to(BF16)
    hq, hs = m.moe_quant_fp8(h)
    y = m.moe_fp8_grouped(hq, hs, w2, s2, offs)
    out = m.moe_unsort_tokens(y, row, w, k)
    token = (sorted_route[:n] // k).long()
    for e in range(E_local):
        a, b = at[e], at[e + 1]
        if a < b:
            ref.check(gu[a:b], *ref.product(xq[token[a:b]], xs[:, token[a:b]], w13[e], s13[e]))
            ref.check(y[a:b], *ref.product(hq[a:b], hs[:, a:b], w2[e], s2[e]))
    here = (row >= 0).view(T, k)
    each = torch.where(here[..., None], y.double()[row.view(T, k).long().clamp_min(0)], 0.0)
    each = each * w.double()[..., None]
    tol = each.sum(1).abs() * 2.0 ** -8 * 1.01 + each.abs().sum(1) * (k + 1) * 2.0 ** -24
    assert ((out.double() - each.sum(1)).abs() <= tol + 1e-38).all()
    # Tokens copied into expert order first: the same bits.
    rows = m.moe_sort_tokens(x, row, k, rows=torch.zeros(T * k, H, dtype=BF16, device=DEV))
    rq, rs = m.moe_quant_fp8(rows)
    assert torch.equal(m.moe_fp8_grouped(rq, rs, w13, s13, offs)[:n], gu[:n])
