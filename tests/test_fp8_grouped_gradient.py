"""The gradient of a grouped FP8 product in its tokens: each expert's weight and scales transposed,
the rows' gradients in expert order, and the unweighted way back to the tokens."""
import os

import pytest
import torch

import fp8_ref as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "mxfp8_mxfp4_experts_amd", "libmi355moe.so")
pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not os.path.exists(LIB), reason="libmi355moe.so not built")]
DEV = "cuda"


@pytest.fixture(scope="module")
def m():
    import mxfp8_mxfp4_experts_amd as mod
    return mod


def setup(m, T, k, E, E_local, N, K, masked):
    g = torch.Generator().manual_seed(T + N + K)
    idx = torch.rand(T, E, generator=g).argsort(1)[:, :k]
    idx = torch.where(torch.rand(T, k, generator=g) < masked, -1, idx).int().to(DEV)
    ws = torch.empty(m.moe_workspace_size(T, k, E_local, 128, 128), dtype=torch.uint8, device=DEV)
    offs, sorted_route, row = m.moe_permute(idx, (E - E_local) // 2, E_local, ws)
    w, w_s = ref.weight(N, K, 4, E_local, 0.3)
    turned = (w.transpose(1, 2).contiguous(), w_s.transpose(1, 2).contiguous())
    return offs, sorted_route, row, (w.to(DEV), w_s.to(DEV)), tuple(t.to(DEV) for t in turned)


CASES = [(1, 1, 1, 1, 16, 16, 0.0), (5, 4, 16, 8, 144, 272, 0.0), (64, 2, 7, 7, 400, 130 * 16, 0.3),
         (300, 3, 12, 6, 272, 144, 0.2), (1024, 4, 8, 8, 512, 384, 0.0), (30, 2, 900, 896, 48, 64, 0.1)]


@pytest.mark.parametrize("T,k,E,E_local,N,K,masked", CASES)
def test_against_the_formula(m, T, k, E, E_local, N, K, masked):
    """drows = dout . w[e] row by row, dx[t] = the sum over t's kept routes: 64 bits on each step's
    own inputs."""
    offs, sorted_route, row, _, turned = setup(m, T, k, E, E_local, N, K, masked)
    R, at = T * k, offs.tolist()
    n = at[-1]
    dout = ref.tokens(R, N, 2).to(DEV)                 # in expert order
    dq, ds = m.moe_quant_fp8(dout)
    drows = torch.full((R, K), 77.0, dtype=torch.bfloat16, device=DEV)
    m.moe_fp8_grouped(dq, ds, *turned, offs, out=drows)
    assert (drows[n:] == 77.0).all()
    drows[n:] = float("nan")                           # no route has these
    for e, (a, b) in enumerate(zip(at, at[1:])):
        if a < b:
            ref.check(drows[a:b], *ref.product(dq[a:b], ds[:, a:b], turned[0][e], turned[1][e]))
    dx = m.moe_unsort_tokens(drows, row, None, k)
    here = (row >= 0).view(T, k)
    each = torch.where(here[..., None], drows.double()[row.view(T, k).long().clamp_min(0)], 0.0)
    want = each.sum(1)
    tol = want.abs() * 2.0 ** -8 * 1.01 + each.abs().sum(1) * (k + 1) * 2.0 ** -24 + 1e-38
    assert ((dx.double() - want).abs() <= tol).all()


def test_against_differences(m):
    """<dout, product> is linear in a token: the difference that one element's step gives. Whole
    numbers and scales of one, so that codes, products and sums are exact and so is the gradient,
    but for its rounding to bf16 and that of the routes' sum."""
    T, k, E, N, K = 37, 3, 6, 272, 144
    offs, sorted_route, row, (w, w_s), _ = setup(m, T, k, E, E, N, K, 0.3)
    g = torch.Generator(device=DEV).manual_seed(1)
    whole = lambda *n: torch.randint(-4, 5, n, generator=g, device=DEV).float()  # noqa: E731
    w, w_s = whole(E, N, K).to(ref.FP8), torch.ones_like(w_s)
    turned = w.transpose(1, 2).contiguous(), w_s.transpose(1, 2).contiguous()
    R, n = T * k, int(offs[-1])
    dout = whole(R, N)
    ones = lambda cols, rows: torch.ones(ref.blocks(cols), rows, device=DEV)  # noqa: E731
    drows = m.moe_fp8_grouped(dout.to(ref.FP8), ones(N, R), *turned, offs)
    dx = m.moe_unsort_tokens(drows, row, None, k)
    kept = torch.zeros(T, dtype=torch.long, device=DEV)
    for t, h in ((0, 0), (T - 1, K - 1), (T // 2, 130), (5, 127), (6, 128)):
        step = torch.zeros(T, K, device=DEV)
        step[t, h] = 1.0
        moved = m.moe_fp8_grouped(step.to(ref.FP8), ones(K, T), w, w_s, offs, sorted_route, k)
        terms = (moved[:n].double() * dout[:n].double()).sum(1)       # exact: |w| <= 4
        diff = terms.sum()
        kept[t] = (terms != 0).sum()
        # Each route's gradient and their sum are rounded to bf16, half a step each.
        assert abs(dx[t, h].double() - diff) <= 2.0 ** -8 * (terms.abs().sum() * 1.01 + diff.abs())
    assert kept.max() > 1                                             # tokens of several routes
