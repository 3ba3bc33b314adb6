"""Block-scaled FP8 products: refusals (no GPU needed) and parity with 64-bit references."""
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
MIS = FAKE + 2
OK, NULL, SHAPE, ALIGN, ENUM, WORKSPACE = 0, 1, 2, 3, 4, 5
BF16, F32 = torch.bfloat16, torch.float32
INF, NAN = math.inf, math.nan


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

def test_quant_refusals(lib):
    def call(x=FAKE, ld=64, T=4, H=64, xq=FAKE, xs=FAKE, ld_s=4):
        return lib.moe_quant_fp8(x, ld, T, H, xq, xs, ld_s, None)
    for bad in (dict(T=-1), dict(T=1 << 22), dict(H=0), dict(H=72, ld=80), dict(ld=56),
                dict(ld_s=3), dict(H=(1 << 20) + 16, ld=1 << 21)):
        assert call(**bad) == SHAPE, bad
    for name in ("x", "xq", "xs"):
        assert call(**{name: None}) == NULL
        assert call(**{name: MIS}) == ALIGN
    assert call(ld=68) == ALIGN
    assert call(T=0, x=None, xq=None, xs=None, ld_s=0) == OK


def test_matmul_refusals(lib):
    def call(xq=FAKE, ld=64, xs=FAKE, ld_s=4, w=FAKE, ws=FAKE, M=4, N=7, K=64, out=FAKE, ldo=7,
             wk=FAKE, nb=1 << 40):
        return lib.moe_fp8_matmul(xq, ld, xs, ld_s, w, ws, M, N, K, out, ldo, wk, nb, None)
    for bad in (dict(M=-1), dict(M=1 << 22, ld_s=1 << 22), dict(N=0), dict(N=(1 << 20) + 1),
                dict(K=0), dict(K=72, ld=80), dict(ld=48), dict(ldo=6), dict(ld_s=3)):
        assert call(**bad) == SHAPE, bad
    for name in ("xq", "xs", "w", "ws", "out"):
        assert call(**{name: None}) == NULL, name
    for bad in (dict(xq=MIS), dict(w=MIS), dict(xs=MIS), dict(ws=MIS), dict(out=MIS), dict(ld=72),
                dict(wk=FAKE + 16)):
        assert call(**bad) == ALIGN, bad
    assert call(M=0, xq=None, out=None) == OK


def test_linear_refusals(lib):
    def call(x=FAKE, ld=64, w=FAKE, ws=FAKE, M=4, N=7, K=64, out=FAKE, ldo=7, wk=FAKE, nb=1 << 40):
        return lib.moe_fp8_linear(x, ld, w, ws, M, N, K, out, ldo, wk, nb, None)
    for bad in (dict(M=-1), dict(N=0), dict(K=72, ld=80), dict(ld=48), dict(ldo=6)):
        assert call(**bad) == SHAPE, bad
    for name in ("x", "w", "ws", "out", "wk"):
        assert call(**{name: None}) == NULL, name
    for bad in (dict(x=MIS), dict(w=MIS), dict(ws=MIS), dict(out=MIS), dict(ld=68),
                dict(wk=FAKE + 16)):
        assert call(**bad) == ALIGN, bad
    assert call(nb=lib.moe_fp8_workspace_size(4, 7, 64) - 1) == WORKSPACE
    assert call(M=0, x=None) == OK


def test_matmul_refuses_a_small_workspace(lib):
    for M, N, K in ((64, 896, 7168), (256, 896, 7168), (256, 3584, 7168)):
        need = lib.moe_fp8_matmul_workspace_size(M, N, K)
        if need:
            assert lib.moe_fp8_matmul(FAKE, K, FAKE, M, FAKE, FAKE, M, N, K, FAKE, N, FAKE,
                                      need - 1, None) == WORKSPACE
            assert lib.moe_fp8_matmul(FAKE, K, FAKE, M, FAKE, FAKE, M, N, K, FAKE, N, None, 0,
                                      None) == NULL


def test_workspaces_grow_with_the_rows(lib):
    for N, K in ((1, 64), (896, 7168), (2051, 1040), (3584, 7168)):
        for f in (lib.moe_fp8_workspace_size, lib.moe_fp8_matmul_workspace_size):
            sizes = [f(M, N, K) for M in range(0, 3000, 7)]
            assert sizes == sorted(sizes)
            assert f(-1, N, K) == 0 and f(4, 0, K) == 0 and f(4, N, 24) == 0
    assert lib.moe_fp8_workspace_size(8, 100, 64) >= 8 * 64 + 8 * 4


def test_grouped_refusals(lib):
    def call(xq=FAKE, ld=64, xs=FAKE, ld_s=8, rows=8, w=FAKE, ws=FAKE, E=3, N=7, K=64, offs=FAKE,
             route=None, top_k=1, R=8, out=FAKE, ldo=7):
        return lib.moe_fp8_grouped(xq, ld, xs, ld_s, rows, w, ws, E, N, K, offs, route, top_k, R,
                                   out, ldo, None)
    for bad in (dict(rows=-1), dict(R=-1), dict(rows=7), dict(E=0), dict(E=4097), dict(N=0),
                dict(K=72, ld=80), dict(ld=48), dict(ld_s=7), dict(ldo=6),
                dict(top_k=0, route=FAKE), dict(top_k=65, route=FAKE),
                dict(R=(1 << 30) + 1, route=FAKE)):
        assert call(**bad) == SHAPE, bad
    for name in ("xq", "xs", "w", "ws", "offs", "out"):
        assert call(**{name: None}) == NULL, name
    for bad in (dict(xq=MIS), dict(xs=MIS), dict(w=MIS), dict(ws=MIS), dict(out=MIS),
                dict(offs=MIS), dict(route=MIS), dict(ld=72)):
        assert call(**bad) == ALIGN, bad
    assert call(R=0, xq=None) == OK and call(rows=0, R=0, out=None) == OK


# ---------------------------------------------------------------------------
# On the GPU.

DEV = "cuda"


def dense(m, M, N, K, seed=0):
    """Inputs on the GPU, and the reference for the codes that the library's rule gives."""
    x = ref.tokens(M, K, seed)
    q, xs = ref.quant(x)
    w, w_s = ref.weight(N, K, seed + 1)
    on = [t.to(DEV) for t in (x, q, xs, w, w_s)]
    return on, ref.product(*on[1:])


@gpu
@pytest.mark.parametrize("T,H", [(1, 16), (1, 128), (3, 144), (5, 1040), (17, 7168), (300, 272),
                                 (4099, 128)])
def test_quant(m, T, H):
    x = ref.tokens(T, H, T + H)
    if T > 2 and H > 16:
        x[0, :H // 2] = 0.0                       # zero blocks
        x[1] *= 1e-38                             # below the smallest scale
    q, s = ref.quant(x)
    xq, xs = m.moe_quant_fp8(x.to(DEV))
    assert torch.equal(xs.cpu(), s)
    assert torch.equal(xq.cpu(), q)


@gpu
def test_quant_odd_values_and_strides(m):
    x = ref.tokens(6, 400, 3)
    x[0, 5], x[1, 130], x[2, 399], x[3, 0] = INF, NAN, -INF, 3.38e38
    q, s = ref.quant(x)
    wide = torch.zeros(6, 512, dtype=BF16, device=DEV)
    wide[:, 64:464] = x.to(DEV)
    xs = torch.full((4, 11), -1.0, device=DEV)
    xq, xs2 = m.moe_quant_fp8(wide[:, 64:464], xs=xs[:, 2:8])
    assert torch.equal(xq.cpu(), q)
    assert torch.equal(xs2.cpu().nan_to_num(-2.0), s.nan_to_num(-2.0))
    assert torch.isnan(s[0, 0]) and torch.isnan(s[1, 1]) and torch.isnan(s[3, 2])
    assert (xs[:, :2] == -1).all() and (xs[:, 8:] == -1).all()   # the columns outside
    a, _ = m.moe_quant_fp8(x.to(DEV), xq=torch.empty(6, 400, dtype=ref.FP8, device=DEV))
    assert torch.equal(a.view(torch.uint8).cpu(), q)


SIZES = [(1, 1, 16), (1, 16, 128), (1, 3584, 7168), (2, 130, 272), (3, 17, 144), (5, 100, 7168),
         (8, 1000, 2048), (15, 129, 400), (16, 128, 256), (17, 129, 400), (31, 515, 1040),
         (33, 257, 1040), (64, 64, 128), (64, 896, 7168), (100, 31, 4112), (130, 300, 2048),
         (257, 515, 1296), (500, 1, 64), (700, 2051, 1040), (1000, 70, 160), (1025, 384, 512),
         (2049, 129, 272), (300, 3584, 1024), (4100, 260, 384)]


@gpu
@pytest.mark.parametrize("M,N,K", SIZES)
def test_matmul_and_linear(m, M, N, K):
    (x, q, xs, w, w_s), (want, mag) = dense(m, M, N, K, M + N + K)
    out = m.moe_fp8_matmul(q, xs, w, w_s)
    ref.check(out, want, mag, "matmul")
    ref.check(m.moe_fp8_linear(x, w.view(torch.uint8), w_s), want, mag, "linear")
    again = m.moe_fp8_matmul(q.view(ref.FP8), xs, w, w_s, out=torch.full_like(out, NAN))
    assert torch.equal(again, out)


@gpu
@pytest.mark.parametrize("M,N,K", [(1, 100, 272), (7, 130, 1040), (40, 200, 400), (300, 260, 1296),
                                   (600, 515, 528)])
def test_strides_and_untouched_columns(m, M, N, K):
    (x, q, xs, w, w_s), (want, mag) = dense(m, M, N, K, 7)
    wide_q = torch.zeros(M, K + 48, dtype=torch.uint8, device=DEV)
    wide_q[:, 16:16 + K] = q
    wide_s = torch.full((ref.blocks(K), M + 9), NAN, device=DEV)
    wide_s[:, 3:3 + M] = xs
    wide_x = torch.full((M, K + 24), NAN, dtype=BF16, device=DEV)
    wide_x[:, 8:8 + K] = x
    for pad in (8, 11):                            # with and without vector stores
        for call in ("matmul", "linear"):
            out = torch.full((M + 1, N + pad + 8), 7.0, dtype=BF16, device=DEV)
            view = out[:M, 8:8 + N]
            if call == "matmul":
                m.moe_fp8_matmul(wide_q[:, 16:16 + K], wide_s[:, 3:3 + M], w, w_s, out=view)
            else:
                m.moe_fp8_linear(wide_x[:, 8:8 + K], w, w_s, out=view)
            ref.check(view, want, mag, call)
            assert (out[M:] == 7).all() and (out[:, :8] == 7).all() and (out[:, 8 + N:] == 7).all()


@gpu
@pytest.mark.parametrize("M,N,K", [(1, 70, 400), (4, 300, 1040), (50, 200, 528), (400, 300, 400)])
def test_odd_values_stay_where_they_are(m, M, N, K):
    """A token with an infinity or a NaN gives NaN, all others what they gave without it; a NaN
    code of the weight its output column; an infinite or NaN scale its block's columns."""
    (x, q, xs, w, w_s), _ = dense(m, M, N, K, 11)
    x = x.clone()
    x[M // 2, 3], x[0, K - 1] = INF, NAN
    w8 = w.view(torch.uint8).clone()
    w8[N // 3, 1] = 0x7F
    if N > 128:
        w_s = w_s.clone()
        w_s[1, 0] = NAN
    q, s = (t.to(DEV) for t in ref.quant(x))
    want, mag = ref.product(q, s, w8.view(ref.FP8), w_s)
    assert torch.isnan(want[0]).all() and torch.isnan(want[:, N // 3]).all()
    ref.check(m.moe_fp8_linear(x, w8, w_s), want, mag.nan_to_num(1.0))
    ref.check(m.moe_fp8_matmul(q, s, w8, w_s), want, mag.nan_to_num(1.0))


@gpu
def test_infinite_scale_of_the_last_short_block(m):
    """Blocks past the end of K bring nothing, whatever the last block's scale."""
    for M, N, K in ((1, 64, 144), (40, 64, 144), (300, 64, 144)):
        (x, q, xs, w, w_s), _ = dense(m, M, N, K, 5)
        q = (q & 0x7F) | 1                       # positive codes, none of them 0
        q[q == 0x7F] = 0x38
        w8 = (w.view(torch.uint8) & 0x7F) | 1
        w8[w8 == 0x7F] = 0x38
        xs = xs.clone()
        xs[1] = INF
        out = m.moe_fp8_matmul(q, xs, w8, w_s)
        assert torch.isinf(out).all() and (out > 0).all()


@gpu
def test_no_rows(m):
    w, w_s = (t.to(DEV) for t in ref.weight(64, 128, 0))
    x = torch.empty(0, 128, dtype=BF16, device=DEV)
    assert m.moe_fp8_linear(x, w, w_s).shape == (0, 64)
    xq, xs = m.moe_quant_fp8(x)
    assert m.moe_fp8_matmul(xq, xs, w, w_s).shape == (0, 64)


@gpu
def test_gradient_of_the_tokens(m):
    """With the weight transposed the linear call is the gradient of <dout, x w^T> in x: against
    the formula, and against differences of the product itself (linear in x, so a step of any
    length will do)."""
    M, N, K = 37, 272, 400
    w, w_s = ref.weight(N, K, 1, spread=0.3)
    wt, wt_s = w.t().contiguous().to(DEV), w_s.t().contiguous().to(DEV)
    dout = ref.tokens(M, N, 2).to(DEV)
    dx = m.moe_fp8_linear(dout, wt, wt_s)
    q, s = (t.to(DEV) for t in ref.quant(dout.cpu()))
    want, mag = ref.product(q, s, wt, wt_s)
    ref.check(dx, want, mag)
    # d<dout, out> for a change of one element of one token by h: all other outputs stay.
    W, S = w.to(DEV), w_s.to(DEV)
    for t, k in ((0, 0), (36, 399), (5, 130)):
        e = torch.zeros(M, K, dtype=BF16, device=DEV)
        e[t, k] = 1.0
        moved = m.moe_fp8_linear(e, W, S)        # one code of 448, exact: w's column, rounded once
        diff = (moved.double() * dout.double()).sum()
        # dx is from dout's codes (half a step of E4M3, 2^-4) and rounded once (bf16, 2^-8), as moved is.
        scale = (moved.double() * dout.double()).abs().sum()
        floor = 448 * 2.0 ** -10 * (s.max() * moved.double().abs().sum()).item()
        assert abs(dx[t, k].double() - diff) <= (2.0 ** -4 + 2.0 ** -6) * scale + floor / 448


def routes(T, k, E, E_local, seed, kind="even"):
    """Global ids [T, k]; the window is [1, 1 + E_local) where E > E_local, else all."""
    g = torch.Generator().manual_seed(seed)
    if kind == "one":
        idx = torch.full((T, k), min(E - 1, 1 + E_local // 2))
    elif kind == "none":
        idx = torch.full((T, k), -1)
    elif kind == "duplicates":
        idx = torch.randint(0, E, (T, 1), generator=g).expand(T, k)
    else:
        idx = torch.rand(T, E, generator=g).argsort(1)[:, :k]
        if kind == "masked":
            idx = torch.where(torch.rand(T, k, generator=g) < 0.4, -1, idx)
    return idx.to(torch.int32).contiguous().to(DEV)


def grouping(m, idx, first, E_local):
    ws = torch.empty(m.moe_workspace_size(*idx.shape, E_local, 128, 128), dtype=torch.uint8,
                     device=DEV)
    return m.moe_permute(idx, first, E_local, ws)


GROUPED = [
    # T, top_k, E, E_local, N, K, routing
    (1, 1, 1, 1, 16, 16, "even"), (1, 8, 28, 28, 300, 400, "even"), (8, 8, 28, 28, 512, 1040, "even"),
    (3, 2, 900, 896, 64, 144, "even"), (40, 4, 16, 8, 129, 272, "even"),
    (17, 3, 9, 5, 100, 528, "masked"), (33, 4, 6, 4, 130, 256, "one"),
    (300, 2, 6, 4, 200, 384, "one"), (20, 5, 7, 7, 96, 160, "duplicates"),
    (50, 2, 8, 4, 64, 128, "none"), (700, 3, 66, 33, 259, 656, "even"),
    (1024, 4, 8, 8, 384, 512, "even"), (2048, 8, 28, 28, 256, 256, "even"),
    (257, 1, 2, 1, 515, 1296, "even"), (513, 6, 40, 20, 31, 80, "masked"),
    (64, 2, 4096, 4096, 48, 128, "even"), (5, 64, 64, 64, 128, 256, "even"),
]


@gpu
@pytest.mark.parametrize("T,k,E,E_local,N,K,kind", GROUPED)
@pytest.mark.parametrize("gather", [True, False])
def test_grouped(m, T, k, E, E_local, N, K, kind, gather):
    first = 1 if E > E_local else 0
    idx = routes(T, k, E, E_local, T + k, kind)
    offs, sorted_route, route_row = grouping(m, idx, first, E_local)
    R, n = T * k, int(offs[-1])
    rows = T if gather else R
    x = ref.tokens(rows, K, 3).to(DEV)
    w, w_s = (t.to(DEV) for t in ref.weight(N, K, 4, E_local))
    xq, xs = m.moe_quant_fp8(x)
    out = torch.full((R, N), 7.0, dtype=BF16, device=DEV)
    m.moe_fp8_grouped(xq, xs, w, w_s, offs, sorted_route if gather else None, k, out=out)
    assert (out[n:] == 7.0).all()                  # rows behind the last expert's
    at = offs.tolist()
    for e in range(E_local):
        a, b = at[e], at[e + 1]
        if a < b:
            mine = (sorted_route[a:b] // k).long() if gather else torch.arange(a, b, device=DEV)
            want, mag = ref.product(xq[mine], xs[:, mine], w[e], w_s[e])
            ref.check(out[a:b], want, mag, f"expert {e}")
    again = m.moe_fp8_grouped(xq, xs, w.view(torch.uint8), w_s, offs,
                              sorted_route if gather else None, k)
    assert torch.equal(again[:n], out[:n])


@gpu
def test_grouped_cuts_off_offsets_and_routes(m):
    """Offsets past the output's rows and routes past the tokens are cut off, not followed."""
    E, N, K, R = 4, 100, 256, 24
    x = ref.tokens(6, K, 1).to(DEV)
    w, w_s = (t.to(DEV) for t in ref.weight(N, K, 2, E))
    xq, xs = m.moe_quant_fp8(x)
    offs = torch.tensor([2, 5, 5, 20, 1000], dtype=torch.int32, device=DEV)
    route = torch.arange(R, dtype=torch.int32, device=DEV)   # tokens 0 .. 23 at top_k 1, of 6
    out = torch.full((R + 2, N), 7.0, dtype=BF16, device=DEV)
    m.moe_fp8_grouped(xq, xs, w, w_s, offs, route, 1, out=out[:R])
    assert (out[:2] == 7).all() and (out[R:] == 7).all()
    for e, a, b in ((0, 2, 5), (2, 5, 20), (3, 20, 24)):
        mine = torch.arange(a, b, device=DEV).clamp(max=5)
        want, mag = ref.product(xq[mine], xs[:, mine], w[e], w_s[e])
        ref.check(out[a:b], want, mag, str(e))


@gpu
@pytest.mark.parametrize("R,offs", [(50, [0, 40, 10, 30]), (700, [0, 600, 20, 520]),
                                    (64, [5, 5, 3, 64]), (40, [30, 20, 10, 0])])
def test_grouped_offsets_out_of_order(m, R, offs):
    """An end before its start is an empty expert; rows that no expert claims are untouched, rows
    that several claim hold, element by element, one's or what was there (such offsets may count
    more tiles than there are rows for)."""
    E, N, K = 3, 130, 272
    xq, xs = m.moe_quant_fp8(ref.tokens(R, K, 1).to(DEV))
    w, w_s = (t.to(DEV) for t in ref.weight(N, K, 2, E))
    out = torch.full((R, N), 7.0, dtype=BF16, device=DEV)
    m.moe_fp8_grouped(xq, xs, w, w_s, torch.tensor(offs, dtype=torch.int32, device=DEV), out=out)
    whole = [m.moe_fp8_matmul(xq, xs, w[e], w_s[e]) for e in range(E)]
    for j in range(R):
        mine = [e for e in range(E) if offs[e] <= j < offs[e + 1]]
        want = [whole[e][j] for e in mine] + [torch.full_like(out[j], 7.0)]
        near = [torch.isclose(out[j].float(), t.float(), rtol=2 ** -6,
                              atol=1e-3 * t.abs().max().item()) for t in want]
        assert torch.stack(near).any(0).all(), (j, mine)


@gpu
@pytest.mark.parametrize("T,k", [(9, 2), (200, 2)])
def test_grouped_strided_tokens_scales_and_output(m, T, k):
    E, N, K = 5, 130, 400
    idx = routes(T, k, E, E, 1)
    offs, sorted_route, _ = grouping(m, idx, 0, E)
    x = ref.tokens(T, K, 3).to(DEV)
    w, w_s = (t.to(DEV) for t in ref.weight(N, K, 4, E))
    xq, xs = m.moe_quant_fp8(x)
    wide_q = torch.zeros(T, K + 32, dtype=torch.uint8, device=DEV)
    wide_q[:, 16:16 + K] = xq
    wide_s = torch.full((ref.blocks(K), T + 5), NAN, device=DEV)
    wide_s[:, 1:1 + T] = xs
    out = torch.full((T * k, N + 19), 7.0, dtype=BF16, device=DEV)
    m.moe_fp8_grouped(wide_q[:, 16:16 + K], wide_s[:, 1:1 + T], w, w_s, offs, sorted_route, k,
                      out=out[:, 8:8 + N])
    want = m.moe_fp8_grouped(xq, xs, w, w_s, offs, sorted_route, k)
    assert torch.equal(out[:, 8:8 + N], want)
    assert (out[:, :8] == 7).all() and (out[:, 8 + N:] == 7).all()


@gpu
@pytest.mark.parametrize("M", [1, 3, 40, 300])
def test_rows_far_apart(m, M):
    """Row strides that pass 2^31 bytes from the first row to the last."""
    N, K = 140, 272
    (x, q, xs, w, w_s), (want, mag) = dense(m, M, N, K, 9)
    step = ((1 << 31) // max(1, M - 1) // 16 + 2) * 16 if M > 1 else K
    far = torch.empty(step * (M - 1) + K, dtype=torch.uint8, device=DEV)
    view = far.as_strided((M, K), (step, 1))
    view.copy_(q)
    ref.check(m.moe_fp8_matmul(view, xs, w, w_s), want, mag)
    offs = torch.tensor([0, M // 2, M], dtype=torch.int32, device=DEV)
    two, two_s = torch.stack([w, w]), torch.stack([w_s, w_s])
    for route in (None, torch.arange(M, dtype=torch.int32, device=DEV)):
        ref.check(m.moe_fp8_grouped(view, xs, two, two_s, offs, route, 1), want, mag)
    out = torch.empty(step * (M - 1) + N, dtype=BF16, device=DEV).as_strided((M, N), (step, 1))
    ref.check(m.moe_fp8_matmul(q, xs, w, w_s, out=out), want, mag)


@gpu
def test_experts_past_two_gib(m):
    """Weights of all experts together pass 2^31 bytes."""
    E, N, K = 180, 3584, 3584
    w = torch.empty(E, N, K, dtype=torch.uint8, device=DEV)
    w_s = torch.ones(E, ref.blocks(N), ref.blocks(K), device=DEV)
    last, _ = ref.weight(N, K, 1)
    w[E - 1] = last.view(torch.uint8).to(DEV)
    x = ref.tokens(3, K, 2).to(DEV)
    xq, xs = m.moe_quant_fp8(x)
    offs = torch.zeros(E + 1, dtype=torch.int32, device=DEV)
    offs[E] = 3
    out = m.moe_fp8_grouped(xq, xs, w, w_s, offs)
    ref.check(out, *ref.product(xq, xs, w[E - 1], w_s[E - 1]))


@gpu
@pytest.mark.parametrize("M", [1, 40, 300])
def test_other_streams_and_graphs(m, M):
    """Two streams with a workspace each at the same time; a captured graph, replayed with other
    inputs beside eager work, gives the eager results."""
    N, K = 520, 1040
    sets = [dense(m, M, N, K, s)[0] for s in range(4)]
    want = [m.moe_fp8_linear(x, w, w_s) for x, _, _, w, w_s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [None] * 4
    for i, (x, _, _, w, w_s) in enumerate(sets):
        with torch.cuda.stream(streams[i % 2]):
            got[i] = m.moe_fp8_linear(x, w, w_s)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    x0, w, w_s = sets[0][0].clone(), sets[0][3], sets[0][4]
    out = torch.empty_like(want[0])
    ws = torch.empty(m.moe_fp8_workspace_size(M, N, K), dtype=torch.uint8, device=DEV)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        m.moe_fp8_linear(x0, w, w_s, out=out, workspace=ws)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        m.moe_fp8_linear(x0, w, w_s, out=out, workspace=ws)
    for i in range(4):
        x0.copy_(sets[i][0])
        eager = m.moe_fp8_linear(x0, w, w_s)
        out.fill_(NAN)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, eager)


@gpu
def test_binding_refusals(m):
    (x, q, xs, w, w_s), _ = dense(m, 4, 130, 272, 1)
    bad = [
        lambda: m.moe_fp8_linear(x.float(), w, w_s), lambda: m.moe_fp8_linear(x.cpu(), w, w_s),
        lambda: m.moe_fp8_linear(x, w[:, :256], w_s), lambda: m.moe_fp8_linear(x, w.float(), w_s),
        lambda: m.moe_fp8_linear(x, w, w_s[:1]), lambda: m.moe_fp8_linear(x, w, w_s.half()),
        lambda: m.moe_fp8_linear(x, w, w_s, out=torch.empty(4, 129, dtype=BF16, device=DEV)),
        lambda: m.moe_fp8_linear(x, w, w_s, out=torch.empty(4, 130, device=DEV)),
        lambda: m.moe_fp8_linear(x.t(), w, w_s), lambda: m.moe_fp8_matmul(q, xs.t(), w, w_s),
        lambda: m.moe_fp8_matmul(q, xs[:2], w, w_s), lambda: m.moe_fp8_matmul(q.int(), xs, w, w_s),
        lambda: m.moe_quant_fp8(x, xs=torch.empty(4, 3, device=DEV)),
        lambda: m.moe_fp8_grouped(q, xs, w, w_s, xs),
        lambda: m.moe_fp8_grouped(q, xs, w[None], w_s[None], torch.zeros(3, dtype=torch.int32,
                                                                         device=DEV)),
        lambda: m.moe_fp8_grouped(q, xs, w[None], w_s, torch.zeros(2, dtype=torch.int32,
                                                                   device=DEV)),
        lambda: m.moe_fp8_grouped(q, xs, w[None], w_s[None],
                                  torch.zeros(2, dtype=torch.int32, device=DEV),
                                  torch.zeros(4, dtype=torch.int64, device=DEV), 1),
    ]
    for i, f in enumerate(bad):
        with pytest.raises(ValueError):
            f()
            pytest.fail(f"call {i} was taken")
    with pytest.raises(m.MoEError):
        m.moe_fp8_linear(x, w, w_s, workspace=torch.empty(16, dtype=torch.uint8, device=DEV))
