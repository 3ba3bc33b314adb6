"""Routes that name the same row, as the grouping never gives them: a sum counts the row for each,
a written row gets what one of them brings."""
import os

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "mxfp8_mxfp4_experts_amd", "libmi355moe.so")
pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not os.path.exists(LIB), reason="libmi355moe.so not built")]
DEV = "cuda"


@pytest.mark.parametrize("kind", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,k,H", [(2, 2, 3), (40, 3, 136), (200, 8, 1037)])
def test_the_same_row_twice(T, k, H, kind):
    import mxfp8_mxfp4_experts_amd as m
    g = torch.Generator().manual_seed(T)
    n = T * k
    row = torch.randint(0, n // 2, (T, k), generator=g)
    row[0] = row[1, 0]                                 # twice in one token, and in another
    whole = lambda *s: torch.randint(-8, 9, s, generator=g).to(kind).to(DEV)  # noqa: E731
    x, y, dout = whole(T, H), whole(n, H), whole(T, H)
    w = (2.0 ** torch.randint(-1, 2, (T, k), generator=g)).to(DEV)
    d_row = row.int().to(DEV).view(-1)
    rows = m.moe_sort_tokens(x, d_row, k, rows=torch.full((n, H), 77.0, dtype=kind, device=DEV))
    drows = torch.full((n, H), 77.0, dtype=kind, device=DEV)
    _, dw = m.moe_unsort_tokens_grad(dout, y, d_row, w, drows=drows)
    for r in range(n):
        routes = (row == r).nonzero().tolist()
        for got, may in ((rows[r], [x[t] for t, _ in routes]),
                         (drows[r], [w[t, j].item() * dout[t] for t, j in routes])):
            may = may or [torch.full_like(got, 77.0)]
            assert torch.stack([got == v for v in may]).any(0).all(), r
    # Whole numbers up to 8 and powers of two: exact in float, one rounding to the rows' type.
    each = y.double()[row.to(DEV)]                     # [T, k, H]
    out = m.moe_unsort_tokens(y, d_row, w, k)
    assert torch.equal(out, (each * w.double()[..., None]).sum(1).to(kind))
    assert torch.equal(dw, (each * dout.double()[:, None]).sum(2).float())
