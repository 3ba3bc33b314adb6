"""Grouped FP8 products whose tokens or scales lie past 31-bit offsets. Whole numbers as codes and
powers of two as scales: the outputs are exact, bit for bit."""
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


def whole(seed, *shape):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randint(-4, 5, shape, generator=g, device=DEV, dtype=torch.int8).float().to(ref.FP8)


def powers(seed, *shape):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return 2.0 ** torch.randint(-1, 2, shape, generator=g, device=DEV).float()


def apart(xs, far):
    """The same scales with their blocks `far` floats apart."""
    KB, T = xs.shape
    return torch.empty(far * (KB - 1) + T, device=DEV).as_strided((KB, T), (far, 1)).copy_(xs)


def exact(q, xs, w, w_s):
    a = q.float() * xs.t().repeat_interleave(128, 1)[:, :q.shape[1]]
    b = w.float() * w_s.repeat_interleave(128, 0)[:w.shape[0]].repeat_interleave(128, 1)[:, :w.shape[1]]
    return (a @ b.t().contiguous()).to(torch.bfloat16)


def expected(out, q, xs, w, w_s, offs, route, k):
    """`out` with every expert's rows in their place."""
    want = out.clone()
    at = [min(max(o, 0), out.shape[0]) for o in offs]
    for e, (a, b) in enumerate(zip(at, at[1:])):
        if a < b:
            mine = (route[a:b].long() // k).clamp(0, q.shape[0] - 1) if route is not None \
                else torch.arange(a, b, device=DEV)
            want[a:b] = exact(q[mine], xs[:, mine], w[e], w_s[e])
    return want


@pytest.mark.parametrize("T,k,E,N,K", [(1, 1, 1, 1, 144), (5, 2, 3, 17, 144), (40, 3, 7, 130, 272),
                                       (300, 2, 4, 260, 144), (200, 4, 130, 64, 400)])
@pytest.mark.parametrize("gather", [True, False])
def test_scales_far_apart(m, T, k, E, N, K, gather):
    """Blocks of scales 2^31 bytes and more from the first to the last."""
    R = T * k
    rows = T if gather else R
    KB = ref.blocks(K)
    q, xs = whole(1, rows, K), powers(2, KB, rows)
    w, w_s = whole(3, E, N, K), powers(4, E, ref.blocks(N), KB)
    g = torch.Generator().manual_seed(R)
    offs = [0] + sorted(torch.randint(0, R + 1, (E - 1,), generator=g).tolist()) + [R]
    route = torch.randperm(R, generator=g).int().to(DEV) if gather else None
    d_offs = torch.tensor(offs, dtype=torch.int32, device=DEV)
    out = torch.full((R, N), 77.0, dtype=torch.bfloat16, device=DEV)
    want = expected(out, q, xs, w, w_s, offs, route, k)
    far = apart(xs, (1 << 29) // KB + 16)
    m.moe_fp8_grouped(q, far, w, w_s, d_offs, route, k, out=out)
    assert torch.equal(out, want)
    assert torch.equal(m.moe_fp8_grouped(q, xs, w, w_s, d_offs, route, k), want)


@pytest.mark.parametrize("offs", [[2, 5, 5, 20, 1000], [-7, 3, 3, 9, 30], [0, 0, 0, 0, 0],
                                  [30, 30, 31, 31, 40], [0, 1, 2, 3, 40]])
def test_far_offsets_and_routes_are_cut_off(m, offs):
    """Offsets past the rows, rows of nobody before and after, and routes of no token."""
    E, N, K, R, T = 4, 100, 272, 40, 6
    q, xs = whole(1, T, K), powers(2, ref.blocks(K), T)
    w, w_s = whole(3, E, N, K), powers(4, E, 1, ref.blocks(K))
    route = (torch.arange(R, device=DEV) - 3).int()
    out = torch.full((R + 2, N + 5), 77.0, dtype=torch.bfloat16, device=DEV)
    want = out.clone()
    want[:R, :N] = expected(out[:R, :N], q, xs, w, w_s, offs, route, 1)
    m.moe_fp8_grouped(q, apart(xs, (1 << 29) // 3 + 16), w, w_s,
                      torch.tensor(offs, dtype=torch.int32, device=DEV), route, 1, out=out[:R, :N])
    assert torch.equal(out, want)


def test_tokens_of_two_gib_and_many_routes(m):
    """300000 tokens, 7168 bytes from one to the next, 8 routes each."""
    T, k, E, N, K = 300000, 8, 28, 512, 128
    q = torch.empty(T, 7168, dtype=torch.uint8, device=DEV)[:, :K]
    q.copy_(whole(1, T, K).view(torch.uint8))
    xs = powers(2, 1, T)
    w, w_s = whole(3, E, N, K), powers(4, E, ref.blocks(N), 1)
    g = torch.Generator(device=DEV).manual_seed(1)
    route = torch.randperm(T * k, generator=g, device=DEV).int()
    offs = [T * k * e // E for e in range(E)] + [T * k - 5]
    out = torch.full((T * k, N), 77.0, dtype=torch.bfloat16, device=DEV)
    m.moe_fp8_grouped(q, xs, w, w_s, torch.tensor(offs, dtype=torch.int32, device=DEV), route, k,
                      out=out)
    assert (out[T * k - 5:] == 77.0).all()
    codes = q.contiguous().view(ref.FP8)
    for e in range(E):
        mine = (route[offs[e]:offs[e + 1]] // k).long()
        assert torch.equal(out[offs[e]:offs[e + 1]], exact(codes[mine], xs[:, mine], w[e], w_s[e]))
