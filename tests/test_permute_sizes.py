"""The grouping at the sizes where its launches change: one workgroup up to 2048 routes, one launch
up to 16384, and above that two launches with few counts or four, against a plain stable sort."""
import os

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "mxfp8_mxfp4_experts_amd", "libmi355moe.so")
pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not os.path.exists(LIB), reason="libmi355moe.so not built")]
DEV = "cuda"
TILES = (32, 256)          # tile heights of the schedule in the workspace

SIZES = [
    # T, top_k, experts in all, experts here, share of masked slots
    (2049, 1, 1, 1, 0.0), (700, 3, 66, 33, 0.1), (2049, 1, 4096, 4096, 0.0), (255, 64, 80, 7, 0.3),
    (5461, 3, 28, 28, 0.0), (2048, 8, 28, 28, 1.0), (2048, 8, 1200, 1100, 0.0),
    (16385, 1, 40, 20, 0.2), (4096, 8, 28, 28, 0.0), (8192, 8, 56, 28, 0.0), (8192, 16, 400, 64, 0.1),
    (8192, 16, 400, 65, 0.1), (4096, 16, 896, 224, 0.0), (5000, 5, 3000, 2500, 0.0),
    (20000, 4, 9, 3, 0.0),
]


@pytest.mark.parametrize("T,k,E,E_local,masked", SIZES)
def test_grouping(T, k, E, E_local, masked):
    import mxfp8_mxfp4_experts_amd as m
    g = torch.Generator().manual_seed(T + k + E)
    idx = torch.randint(0, E, (T, k), generator=g)
    idx = torch.where(torch.rand(T, k, generator=g) < masked, -1, idx).to(torch.int32)
    first, R = (E - E_local) // 2, T * k
    local = idx.view(-1).long() - first
    kept = (idx.view(-1) >= 0) & (local >= 0) & (local < E_local)
    key = torch.where(kept, local, E_local)
    order = torch.sort(key, stable=True)[1]
    counts = torch.bincount(key, minlength=E_local + 1)[:E_local]
    offsets = torch.cat([torch.zeros(1, dtype=torch.long), counts.cumsum(0)])
    n = int(offsets[-1])
    want = torch.full((R,), -1)
    want[:n] = order[:n]
    row = torch.full((R,), -1)
    row[order[:n]] = torch.arange(n)
    ws = torch.full((m.moe_workspace_size(T, k, E_local, 128, 128),), 0xA5, dtype=torch.uint8,
                    device=DEV)
    bufs = [torch.full((s,), -7, dtype=torch.int32, device=DEV) for s in (E_local + 1, R, R)]
    d_idx = idx.to(DEV)
    for _ in range(2):
        got = m.moe_permute(d_idx, first, E_local, ws, *bufs)
        for a, b in zip(got, (offsets, want, row)):
            assert torch.equal(a.cpu().long(), b)
        # The schedule behind it: tile prefixes, and the expert of every 32-row tile.
        head = ws[:4 * (2 * (E_local + 1) + R // 32 + E_local)].view(torch.int32).cpu().long()
        for i, h in enumerate(TILES):
            tiles = (counts + h - 1) // h
            prefix = torch.cat([torch.zeros(1, dtype=torch.long), tiles.cumsum(0)])
            assert torch.equal(head[i * (E_local + 1):(i + 1) * (E_local + 1)], prefix)
        owner = torch.repeat_interleave(torch.arange(E_local), (counts + 31) // 32)
        at = 2 * (E_local + 1)
        assert torch.equal(head[at:at + owner.numel()], owner)
