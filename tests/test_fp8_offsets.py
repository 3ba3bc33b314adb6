"""Grouped FP8 products with offsets that descend. Whole numbers: exact, bit for bit."""
import os

import pytest
import torch

import fp8_ref as ref
from test_fp8_far import apart, exact, powers, whole

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "mxfp8_mxfp4_experts_amd", "libmi355moe.so")
pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not os.path.exists(LIB), reason="libmi355moe.so not built")]
DEV = "cuda"
N, K = 130, 272

# Offsets, and whether the experts' rows come to no more tiles than as many rows in order may have
# (rows / height + experts, of any height): then every claimed row is written.
CASES = [([5, 5, 3, 64], True), ([30, 20, 10, 0], True), ([64, 3, 64], True), ([0, 40, 38, 40], True),
         ([-3, 7, 2, 64], True), ([9, 64, 0, 0, 5], True),
         ([0, 64, 0, 64, 0, 64, 0, 64], False), ([0, 600, 20, 520], False),
         ([0, 60, 0, 1 << 30, -(1 << 30), 1 << 30], False)]


@pytest.mark.parametrize("far", [False, True])
@pytest.mark.parametrize("offs,fits", CASES)
def test_rows_are_a_claimants(offs, fits, far):
    import mxfp8_mxfp4_experts_amd as m
    E, R = len(offs) - 1, 700 if max(offs) > 64 else 64
    q, xs = whole(1, R, K), powers(2, ref.blocks(K), R)
    w, w_s = whole(3, E, N, K), powers(4, E, ref.blocks(N), ref.blocks(K))
    out = torch.full((R, N), 77.0, dtype=torch.bfloat16, device=DEV)
    scales = apart(xs, (1 << 29) // 3 + 16) if far else xs
    m.moe_fp8_grouped(q, scales, w, w_s, torch.tensor(offs, dtype=torch.int32, device=DEV), out=out)
    whole_out = [exact(q, xs, w[e], w_s[e]) for e in range(E)]
    for j in range(R):
        mine = [e for e in range(E) if max(offs[e], 0) <= j < min(offs[e + 1], R)]
        may = [whole_out[e][j] for e in mine]
        if not mine or not fits:
            may.append(torch.full_like(out[j], 77.0))
        assert torch.stack([out[j] == t for t in may]).any(0).all(), (j, mine)
