"""The grouping where most routes or all go to one expert, and with few experts and many routes:
every launch form, against a plain stable sort."""
import os

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "mxfp8_mxfp4_experts_amd", "libmi355moe.so")
pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not os.path.exists(LIB), reason="libmi355moe.so not built")]
DEV = "cuda"

# T, top_k, experts (one launch up to 16384 routes; above, two up to 512 chunks of 512 with 16384
# counts or fewer; else four)
SIZES = [(257, 8, 1), (257, 8, 3), (700, 3, 64), (2048, 8, 1), (2048, 8, 28), (2047, 8, 896),
         (2049, 8, 2), (4096, 8, 28), (32768, 8, 8), (32768, 8, 32), (32769, 8, 1), (32800, 8, 40),
         (16000, 8, 896), (65536, 16, 2)]


@pytest.mark.parametrize("how", ["one", "first", "last", "hot", "hot and masked"])
@pytest.mark.parametrize("T,k,E", SIZES)
def test_grouping(T, k, E, how):
    import mxfp8_mxfp4_experts_amd as m
    g = torch.Generator(device=DEV).manual_seed(T + k + E)
    at = dict(first=0, last=E - 1).get(how, E // 2)
    idx = torch.full((T, k), at, dtype=torch.int32, device=DEV)
    if how.startswith("hot"):
        other = torch.randint(0, E, (T, k), generator=g, device=DEV, dtype=torch.int32)
        idx = torch.where(torch.rand(T, k, generator=g, device=DEV) < 0.9, idx, other)
    if how.endswith("masked"):
        idx = torch.where(torch.rand(T, k, generator=g, device=DEV) < 0.3, -1, idx)
    R = T * k
    key = torch.where(idx.view(-1) >= 0, idx.view(-1).long(), E)
    order = torch.sort(key, stable=True)[1]
    counts = torch.bincount(key, minlength=E + 1)[:E]
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)])
    n = int(offsets[-1])
    want = torch.full((R,), -1, device=DEV)
    want[:n] = order[:n]
    row = torch.full((R,), -1, device=DEV)
    row[order[:n]] = torch.arange(n, device=DEV)
    ws = torch.full((m.moe_workspace_size(T, k, E, 128, 128),), 0xA5, dtype=torch.uint8, device=DEV)
    bufs = [torch.full((s,), -7, dtype=torch.int32, device=DEV) for s in (E + 1, R, R)]
    got = m.moe_permute(idx, 0, E, ws, *bufs)
    for a, b in zip(got, (offsets, want, row)):
        assert torch.equal(a.long(), b)
    # The schedule behind it: tile prefixes of both heights, the expert of every 32-row tile, and
    # nothing past it.
    head = ws[:4 * (2 * (E + 1) + R // 32 + E)].view(torch.int32).long()
    for i, h in enumerate((32, 256)):
        tiles = (counts + h - 1) // h
        prefix = torch.cat([tiles.new_zeros(1), tiles.cumsum(0)])
        assert torch.equal(head[i * (E + 1):(i + 1) * (E + 1)], prefix)
    owner = torch.repeat_interleave(torch.arange(E, device=DEV), (counts + 31) // 32)
    owners = head[2 * (E + 1):]
    assert torch.equal(owners[:owner.numel()], owner)
    assert (owners[owner.numel():] == 0xA5A5A5A5 - (1 << 32)).all()
