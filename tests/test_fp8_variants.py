"""Every kernel, tile variant and split that the sizes of a block-scaled FP8 product choose, with
whole numbers up to 4 as codes and powers of two as scales: every product, block sum and running
sum is exact in any order, so the outputs are the exact sum rounded once to bf16, bit for bit.

Which kernel a shape takes is asked of the library's own choice (csrc/fp8_pick.h, through the
test-only probe library), so the lists below fail on the CPU when a new estimate leaves a variant
without a shape."""
import ctypes
import os

import pytest
import torch

import fp8_ref as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "mxfp8_mxfp4_experts_amd", "libmi355moe.so")
PROBE = os.path.join(ROOT, "tests", "probe", "libnumprobe.so")
pytestmark = pytest.mark.skipif(not (os.path.exists(LIB) and os.path.exists(PROBE)),
                                reason="libmi355moe.so or libnumprobe.so not built")
gpu = pytest.mark.gpu
DEV = "cuda"

# (rows, columns, K): for every variant of the tiled kernel, with K whole and split, at most 64
# scale blocks and more (its weight scales come 64 at a time), a product with odd edges (rows,
# columns and K past whole tiles and stages), one with edges and rows of whole pieces of 16 bytes,
# and one of whole tiles.
TILED = {
    (0, False, False): [(2371, 3345, 2080), (4432, 2768, 1296), (5120, 2560, 1312)],
    (0, False, True): [(3595, 2201, 8256), (3105, 2624, 8224), (3328, 2560, 8224)],
    (1, False, False): [(1796, 1095, 1344), (1154, 1784, 1296), (896, 2432, 1328)],
    (1, False, True): [(1688, 1164, 8256), (1218, 1624, 8256), (1664, 1280, 8208)],
    (1, True, False): [(3287, 259, 8096), (4328, 208, 7984)],
    (1, True, True): [(2817, 132, 8464), (2751, 136, 8304), (1664, 640, 9104)],
    (2, False, False): [(812, 1230, 1312), (1167, 840, 1328), (640, 1664, 1296)],
    (2, False, True): [(1025, 981, 8208), (1094, 912, 8208), (768, 1408, 8224)],
    (2, True, False): [(332, 902, 6256), (452, 656, 6192), (704, 512, 7984)],
    (2, True, True): [(260, 783, 9680), (648, 328, 9648), (704, 512, 8224)],
    (3, False, False): [(1163, 404, 1312), (898, 520, 1344), (704, 768, 1312)],
    (3, False, True): [(900, 642, 8336), (1105, 520, 8256), (960, 704, 8208)],
    (3, True, False): [(1078, 65, 3472), (690, 200, 3392), (320, 576, 3792)],
    (3, True, True): [(391, 65, 10640), (450, 72, 9312), (256, 448, 8720)],
    (4, False, False): [(241, 260, 1328), (542, 72, 1312), (576, 64, 1296)],
    (4, False, True): [(780, 582, 8416), (579, 776, 8352), (480, 2112, 9056)],
    (4, True, False): [(106, 151, 4592), (153, 104, 4960), (576, 64, 2064)],
    (4, True, True): [(146, 105, 8240), (114, 144, 8208), (160, 128, 8656)],
}
# Few stages: fewer than the ring has, one, and a part of one.
SHORT = [(8942, 1306, 16), (4864, 2816, 272), (8487, 204, 16), (1280, 1664, 400), (8223, 65, 16),
         (640, 1664, 272), (8380, 1, 16), (640, 832, 160), (517, 1, 16), (544, 64, 272)]
# The direct kernel: Q, and its batches of K (8: more than four, which loop).
DIRECT = {
    (1, 1): [(89, 169, 16), (17, 682, 272), (116, 288, 1392)],
    (1, 2): [(156, 208, 2064), (32, 1152, 3792)], (1, 4): [(159, 104, 4112), (134, 411, 6784)],
    (1, 8): [(385, 156, 8480), (4, 2816, 12752)], (2, 1): [(1, 1, 2816), (14, 728, 224)],
    (2, 2): [(73, 55, 4208), (11, 550, 4784)], (2, 4): [(1, 1, 12432), (167, 35, 8240)],
    (2, 8): [(1, 1, 16544), (32, 64, 17440)], (4, 1): [(1, 1, 16), (9, 72, 32)],
    (4, 2): [(1, 1, 8224), (175, 9, 8912)],
}
# One launch that quantises and multiplies: Q, steps of K at once, more than 64 blocks to quantise
# (more than one piece a thread), more steps than it takes at once.
RAW = {
    (1, 1, False, False): [(89, 169, 16), (14, 1067, 272)],
    (1, 1, True, False): [(175, 192, 528), (19, 816, 1856)],
    (1, 2, False, False): [(2, 2056, 2064), (2, 2720, 3280)],
    (1, 2, True, False): [(10, 1046, 2096), (5, 2705, 3856)],
    (1, 4, False, False): [(1, 2077, 4192), (1, 3396, 5952)],
    (1, 4, True, False): [(4, 2072, 4208), (2, 2904, 5632)],
    (1, 4, True, True): [(3, 2144, 8432), (2, 2568, 15040)],
    (2, 1, False, False): [(37, 101, 16), (61, 124, 256)],
    (2, 1, True, False): [(4, 5, 4096), (267, 24, 1488)],
    (2, 2, False, False): [(1, 1042, 4128), (1, 1354, 5520)],
    (2, 2, True, False): [(5, 533, 4128), (6, 1965, 4544)],
    (2, 4, True, False): [(2, 1031, 8336), (1, 1129, 14752)],
    (2, 4, True, True): [(1, 1032, 16448), (1, 1971, 16736)],
    (4, 1, False, False): [(1, 1, 16), (32, 128, 2000)],
    (4, 1, True, False): [(4, 1, 2080), (3, 314, 5136)],
    (4, 2, True, False): [(1, 1, 8224), (2, 164, 14448)],
    (4, 4, True, False): [(1, 1, 16544), (1, 8, 17200)],
}
# Grouped: (routes, experts, columns, K) for every variant, K up to 64 blocks and more.
GROUPED = {
    (0, False): [(16669, 23, 659, 16), (10480, 4, 1526, 320)],
    (0, True): [(2410, 7, 3134, 8480), (5806, 2, 1436, 8224)],
    (1, False): [(703, 17, 1675, 32), (1644, 4, 1232, 656)],
    (1, True): [(1440, 26, 955, 8416), (2977, 55, 396, 8224)],
    (2, False): [(34, 59, 1442, 16), (9028, 2, 106, 144)],
    (2, True): [(674, 31, 864, 8368), (7878, 60, 119, 9152)],
    (3, False): [(7810, 29, 1, 16), (854, 5, 868, 400)],
    (3, True): [(522, 22, 589, 8208), (415, 17, 902, 8256)],
    (4, False): [(1, 1, 1, 16), (606, 36, 2, 144)],
    (4, True): [(1, 11, 1, 8320), (142, 40, 149, 9504)],
}


def flat(shapes):
    return [pytest.param(*s, id="-".join(map(str, key)) + ":" + "x".join(map(str, s)))
            for key, many in shapes.items() for s in many]


@pytest.fixture(scope="module")
def probe():
    lib = ctypes.CDLL(PROBE)
    lib.probe_fp8_pick.argtypes = [ctypes.c_int] * 3 + [ctypes.POINTER(ctypes.c_int32)]
    lib.probe_fp8_pick.restype = None
    return lib


def picked(probe, M, N, K):
    out = (ctypes.c_int32 * 6)()
    probe.probe_fp8_pick(M, N, K, out)
    return tuple(out)


def batch(steps):
    return steps if steps <= 2 else 4 if steps <= 4 else 8


# ---------------------------------------------------------------------------
# The lists reach what they say (no GPU needed).

def test_tiled_shapes(probe):
    assert {v for v, _, _ in TILED} == set(range(probe.probe_fp8_variants()))
    for (v, split, long), shapes in TILED.items():
        kinds = set()
        for M, N, K in shapes:
            got, splits, bm, bn, _, _ = picked(probe, M, N, K)
            assert (got, splits > 1, K > 8192) == (v, split, long), (M, N, K)
            if M % bm == 0 and N % bn == 0:
                kinds.add("whole")
            else:
                assert M % bm and N % bn and K % 128, (M, N, K)
                kinds.add("edges" if N % 8 == 0 else "odd")
        assert kinds >= {"odd", "edges"}, v
    assert {picked(probe, *s)[0] for s in SHORT} == {v for v, _, _ in TILED}


def test_direct_shapes(probe):
    assert set(DIRECT) == {(q, b) for q in (1, 2, 4) for b in (1, 2, 4, 8)} - {(4, 4), (4, 8)}
    for (q, b), shapes in DIRECT.items():
        for M, N, K in shapes:
            v, _, _, _, got, steps = picked(probe, M, N, K)
            assert (v, got, batch(steps)) == (-1, q, b), (M, N, K)


def test_raw_shapes(probe):
    for (q, b, pieces, loop), shapes in RAW.items():
        for M, N, K in shapes:
            assert probe.probe_fp8_raw(M, N, K) == q, (M, N, K)
            steps, KB = -(-K // (2048 * q)), ref.blocks(K)
            got = (min(batch(steps), 4), min(M, 16 // q) * KB > 64, steps > 4)
            assert got == (b, pieces, loop), (M, N, K)


def test_grouped_shapes(probe):
    assert {v for v, _ in GROUPED} == set(range(probe.probe_fp8_variants()))
    for (v, long), shapes in GROUPED.items():
        for R, E, N, K in shapes:
            assert (probe.probe_fp8_grouped(R, E, N, K), K > 8192) == (v, long), (R, E, N, K)


# ---------------------------------------------------------------------------
# The products.

@pytest.fixture(scope="module")
def m():
    import mxfp8_mxfp4_experts_amd as mod
    return mod


def whole(seed, *shape):
    """Codes of whole numbers -4 .. 4."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randint(-4, 5, shape, generator=g, device=DEV, dtype=torch.int8).float().to(ref.FP8)


def powers(seed, *shape):
    """1/2, 1, 2: a block's scaled sum is a multiple of 1/4 and below 2^14 (with one code of 448 in
    it; else 2^13), so a sum of up to 256 blocks is below 2^22: 24 bits."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    return 2.0 ** torch.randint(-1, 2, shape, generator=g, device=DEV).float()


def exact(q, xs, w, w_s):
    """In float32, where these sums are exact in any order."""
    a = q.float() * xs.t().repeat_interleave(128, 1)[:, :q.shape[1]]
    b = w.float() * w_s.repeat_interleave(128, 0)[:w.shape[0]].repeat_interleave(128, 1)[:, :w.shape[1]]
    return (a @ b.t().contiguous()).to(torch.bfloat16)


def operands(M, N, K):
    assert ref.blocks(K) < 256
    NB, KB = ref.blocks(N), ref.blocks(K)
    return whole(M + N, M, K), powers(M, KB, M), whole(K, N, K), powers(N, NB, KB)


def windows(M, N):
    """None (a new tensor) and windows of buffers whose rows are 16, 8 and 2 bytes' multiples
    long, with what lies beside them."""
    yield None, None
    for extra in (16, 20, 17):
        wide = torch.full((M, (N + 7) // 8 * 8 + extra), 77.0, device=DEV, dtype=torch.bfloat16)
        yield wide[:, 8:8 + N], wide


def same(got, want, wide, N):
    assert torch.equal(got, want)
    assert wide is None or ((wide[:, :8] == 77).all() and (wide[:, 8 + N:] == 77).all())


@gpu
@pytest.mark.parametrize("M,N,K", flat(TILED) + [pytest.param(*s, id="short:" + "x".join(map(str, s)))
                                                 for s in SHORT] + flat(DIRECT))
def test_product(m, M, N, K):
    q, xs, w, w_s = operands(M, N, K)
    want = exact(q, xs, w, w_s)
    for out, wide in windows(M, N):
        same(m.moe_fp8_matmul(q, xs, w, w_s, out=out), want, wide, N)


@gpu
@pytest.mark.parametrize("M,N,K", flat(RAW))
def test_one_launch(m, M, N, K):
    """Tokens whose blocks' largest value is 448 s, so that their codes are whole numbers too."""
    q, xs, w, w_s = operands(M, N, K)
    x = q.float() * xs.t().repeat_interleave(128, 1)[:, :K]
    top = 448.0 * xs.t()
    x[:, ::128] = torch.where(torch.rand(M, ref.blocks(K), device=DEV) < 0.5, top, -top)
    x = x.to(torch.bfloat16)
    codes, s = m.moe_quant_fp8(x)
    assert torch.equal(s, xs)
    want = exact(codes.view(ref.FP8), s, w, w_s)
    assert torch.equal(m.moe_fp8_matmul(codes, s, w, w_s), want)
    for out, wide in windows(M, N):
        same(m.moe_fp8_linear(x, w, w_s, out=out), want, wide, N)


def ends(R, E, seed):
    """Ends of E experts' rows in 0 .. R, with empty experts and one large one; rows before the
    first and after the last are nobody's."""
    g = torch.Generator().manual_seed(seed)
    cuts = torch.randint(0, R + 1, (E + 1,), generator=g)
    cuts[: (E + 1) // 3] = R // 3
    return cuts.sort().values.to(torch.int32)


@gpu
@pytest.mark.parametrize("R,E,N,K", flat(GROUPED))
@pytest.mark.parametrize("gather", [True, False])
def test_grouped(m, R, E, N, K, gather):
    T, k = (R + 2) // 3, 3
    rows = T if gather else R
    q, xs = whole(R, rows, K), powers(R, ref.blocks(K), rows)
    w, w_s = whole(K, E, N, K), powers(N, E, ref.blocks(N), ref.blocks(K))
    at = ends(R, E, R + E)
    g = torch.Generator(device=DEV).manual_seed(R)
    route = torch.randperm(T * k, generator=g, device=DEV)[:R].to(torch.int32)
    out = torch.full((R, N + 5), 77.0, device=DEV, dtype=torch.bfloat16)
    m.moe_fp8_grouped(q, xs, w, w_s, at.to(DEV), route if gather else None, k, out=out[:, :N])
    want = torch.full_like(out, 77.0)
    for e, (a, b) in enumerate(zip(at.tolist(), at.tolist()[1:])):
        if a < b:
            mine = (route[a:b] // k).long() if gather else slice(a, b)
            want[a:b, :N] = exact(q[mine], xs[:, mine], w[e], w_s[e])
    assert torch.equal(out, want)


@gpu
@pytest.mark.parametrize("R,E,N,K", [(40, 6, 260, 400), (900, 9, 300, 528)])
def test_grouped_on_two_streams_and_in_a_graph(m, R, E, N, K):
    """Two products at once, and a captured one replayed with other tokens and other offsets
    beside eager work."""
    sets = []
    for s in range(3):
        q, xs = whole(s, R, K), powers(s, ref.blocks(K), R)
        w, w_s = whole(10 + s, E, N, K), powers(20 + s, E, ref.blocks(N), ref.blocks(K))
        sets.append((q, xs, w, w_s, ends(R, E, s).to(DEV)))
    base = torch.zeros(R, N, device=DEV, dtype=torch.bfloat16)
    want = [m.moe_fp8_grouped(*t, out=base.clone()) for t in sets]
    got = [base.clone() for _ in range(6)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for i in range(6):
        with torch.cuda.stream(streams[i % 2]):
            m.moe_fp8_grouped(*sets[i % 3], out=got[i])
    torch.cuda.synchronize()
    assert all(torch.equal(got[i], want[i % 3]) for i in range(6))
    own = [t.clone() for t in sets[0]]
    out = base.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        m.moe_fp8_grouped(*own, out=out)
    for i in (1, 2, 0, 1):
        for mine, new in zip(own, sets[i]):
            mine.copy_(new)
        out.zero_()
        eager = m.moe_fp8_grouped(*own, out=base.clone())
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[i]) and torch.equal(eager, want[i])
