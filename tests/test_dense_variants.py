"""Every kernel, tile variant and split that the sizes of a dense product choose,
with random operands: INT8 products bit for bit, router products of whole
numbers (whose float32 sums are exact in any order) likewise.

Which kernel a shape takes is asked of the library's own choice
(csrc/dense_pick.h, through the test-only probe library), so the lists below
fail on the CPU when a new estimate leaves a variant without a shape."""
import ctypes
import os

import pytest
import torch

import block_ref as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "mxfp8_mxfp4_experts_amd", "libmi355moe.so")
PROBE = os.path.join(ROOT, "tests", "probe", "libnumprobe.so")
pytestmark = pytest.mark.skipif(not (os.path.exists(LIB) and os.path.exists(PROBE)),
                                reason="libmi355moe.so or libnumprobe.so not built")
gpu = pytest.mark.gpu

# (rows, columns, bytes of K): for every variant of the tiled kernel, with K whole and split, a
# product with odd edges (rows, columns and K past whole tiles and stages, no vector stores), one
# with edges whose rows take vector stores, and one of whole tiles.
TILED = {
    (0, False): [(7817, 1585, 4640), (5511, 2192, 4672), (5120, 2464, 4656)],
    (1, False): [(5265, 871, 1296), (8162, 520, 1376), (6656, 672, 1296)],
    (1, True): [(4125, 457, 12528), (6564, 280, 11920), (8320, 224, 12032)],
    (2, False): [(8211, 201, 1840), (8416, 208, 1680), (1280, 1664, 1680)],
    (2, True): [(2149, 199, 8896), (2124, 200, 8896), (1408, 384, 9616)],
    (3, False): [(6250, 195, 1344), (6255, 200, 1296), (512, 2944, 1296)],
    (3, True): [(139, 1137, 10768), (34, 3384, 10400), (192, 1408, 8464)],
    (4, False): [(8199, 65, 1360), (8270, 72, 1296), (8256, 128, 1280)],
    (4, True): [(1620, 73, 9232), (65, 1352, 10512), (96, 1856, 8848)],
    (5, False): [(5560, 69, 1296), (5639, 72, 1328), (640, 832, 1280)],
    (5, True): [(676, 67, 5568), (34, 1176, 7008), (704, 192, 5776)],
    (6, False): [(5450, 67, 3104), (5619, 72, 3168), (192, 2752, 3120)],
    (6, True): [(1958, 67, 12768), (33, 3592, 12656), (64, 3328, 12688)],
    (7, False): [(2764, 69, 1296), (65, 2920, 1312), (1376, 192, 1280)],
    (7, True): [(33, 453, 7520), (33, 416, 7120), (832, 64, 3728)],
    (8, False): [(531, 33, 1344), (519, 40, 1296), (608, 32, 1280)],
    (8, True): [(560, 33, 3360), (513, 40, 3472), (544, 32, 3216)],
}
# The direct kernel: Q, and the steps of K that its loads are batched for (8: the looping form).
DIRECT = {
    (1, 1): [(1, 2049, 16), (17, 682, 272)], (1, 2): [(17, 1522, 2144), (3, 2147, 2064)],
    (1, 4): [(17, 1411, 4128), (13, 2589, 4128)], (1, 8): [(1, 2244, 8272), (15, 3300, 17200)],
    (2, 1): [(9, 1, 16), (7, 130, 272)], (2, 2): [(364, 9, 4128), (7, 130, 4160)],
    (2, 4): [(350, 9, 8288), (7, 1003, 8272)], (2, 8): [(9, 359, 17136), (7, 722, 17024)],
    (4, 1): [(5, 1, 6496), (7, 18, 8192)], (4, 2): [(5, 1, 8240), (7, 130, 8208)],
    (4, 4): [(5, 1, 16464), (3, 18, 16400)], (4, 8): [(5, 1, 32896), (1, 33, 70000)],
}
# One launch that quantises and multiplies: Q, most steps of K at once, more than 16 units of 512.
FUSED = {
    (1, 2, False): [(17, 696, 16), (9, 2060, 272)], (1, 2, True): [(17, 701, 528), (9, 1046, 528)],
    (1, 4, False): [(1, 2133, 2064), (3, 2133, 2064)], (1, 4, True): [(3, 2154, 2576)],
    (1, 8, False): [(1, 2060, 4144)], (1, 8, True): [(2, 2050, 4112)],
    (2, 2, False): [(513, 5, 16), (7, 1026, 272)], (2, 2, True): [(513, 5, 1072), (6, 513, 1120)],
    (2, 4, False): [(1, 1057, 4240)], (2, 4, True): [(2, 1036, 4128)],
    (2, 8, True): [(1, 1055, 8272)],
    (4, 2, False): [(5, 1, 16), (3, 130, 272)], (4, 2, True): [(5, 1, 2080), (3, 34, 2576)],
    (4, 4, True): [(1, 35, 8224), (2, 3, 8240)], (4, 8, True): [(1, 34, 16400), (1, 130, 20000)],
}


def flat(shapes):
    return [pytest.param(key, s, id="-".join(map(str, key)) + ":" + "x".join(map(str, s)))
            for key, many in shapes.items() for s in many]


@pytest.fixture(scope="module")
def probe():
    lib = ctypes.CDLL(PROBE)
    lib.probe_dense_pick.argtypes = [ctypes.c_int, ctypes.c_int, ctypes.c_int64,
                                     ctypes.POINTER(ctypes.c_int32)]
    lib.probe_dense_pick.restype = None
    return lib


def picked(probe, M, N, Kb):
    out = (ctypes.c_int32 * 6)()
    probe.probe_dense_pick(M, N, Kb, out)
    return tuple(out)


def batch(steps):
    return 1 if steps <= 2 else 2 if steps <= 4 else 4 if steps <= 8 else 8


# ---------------------------------------------------------------------------
# The lists reach what they say (no GPU needed).

def test_tiled_shapes(probe):
    assert {v for v, _ in TILED} == set(range(probe.probe_num_variants()))
    for (v, split), shapes in TILED.items():
        kinds = set()
        for M, N, Kb in shapes:
            got, splits, bm, bn, _, _ = picked(probe, M, N, Kb)
            assert (got, splits > 1) == (v, split), (M, N, Kb)
            assert Kb % 16 == 0 and Kb >= 1280 and M >= 33     # every stage of the ring, twice
            if M % bm == 0 and N % bn == 0:
                kinds.add("whole")
            else:
                assert M % bm and N % bn and Kb % 128, (M, N, Kb)
                kinds.add("edges" if N % 8 == 0 else "odd")
        assert kinds == {"odd", "edges", "whole"}, v


def test_direct_shapes(probe):
    assert set(DIRECT) == {(q, b) for q in (1, 2, 4) for b in (1, 2, 4, 8)}
    for (q, b), shapes in DIRECT.items():
        for M, N, Kb in shapes:
            v, _, _, _, got, steps = picked(probe, M, N, Kb)
            assert (v, got, batch(steps)) == (-1, q, b), (M, N, Kb)


def test_fused_shapes(probe):
    # One unit per wavefront ends at K = 8192, where the longer batches begin for larger Q.
    assert set(FUSED) == {(q, b, more) for q in (1, 2, 4) for b in (2, 4, 8)
                          for more in (False, True) if more or b == 2 or b * q < 16}
    for (q, b, more), shapes in FUSED.items():
        for M, N, K in shapes:
            assert probe.probe_fused_q(M, N, K) == q, (M, N, K)
            steps = -(-K // (1024 * q))
            units = min(M, 16 // q) * -(-K // 512)
            assert (2 if steps <= 2 else 4 if steps <= 4 else 8, units > 16) == (b, more), (M, N, K)


# ---------------------------------------------------------------------------
# The products.

@pytest.fixture(scope="module")
def m():
    import mxfp8_mxfp4_experts_amd as mod
    return mod


def whole(seed, low, high, *shape):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(low, high, shape, generator=g, dtype=torch.int32, device="cuda")


def strided(t, pad):
    """The same rows as a window of a wider buffer."""
    wide = torch.full((t.shape[0], t.shape[1] + 2 * pad), 99, device="cuda").to(t.dtype)
    wide[:, pad:pad + t.shape[1]] = t
    return wide[:, pad:pad + t.shape[1]]


def outputs(M, N, dtype):
    """None (a new tensor) and windows of buffers whose rows are 8, 4 and 1 elements' multiples
    long: each way of storing a row, with what lies beside them."""
    yield None, None
    for extra in (16, 20, 17):
        wide = torch.full((M, (N + 7) // 8 * 8 + extra), 77.0, device="cuda").to(dtype)
        yield wide[:, 8:8 + N], wide


def beside(wide, N):
    return (wide[:, :8] == 77).all() and (wide[:, 8 + N:] == 77).all()


def int8_operands(M, N, K):
    q = whole(M + N, -128, 128, M, K).to(torch.int8)
    w = whole(K, -128, 128, N, K).to(torch.int8)
    g = torch.Generator(device="cuda").manual_seed(M)
    sx = 0.01 + torch.rand(M, generator=g, device="cuda")
    sw = 0.001 + 0.01 * torch.rand(N, generator=g, device="cuda")
    return q, sx, w, sw


def int8_product(q, sx, w, sw):
    """The sum exact (far below 2^53), then the three factors in float32."""
    return ((q.double() @ w.double().t().contiguous()).float() * sx[:, None]) * sw


def check_int8(m, M, N, K):
    q, sx, w, sw = int8_operands(M, N, K)
    want = int8_product(q, sx, w, sw)
    tokens = strided(q, 16)
    for dtype in (torch.float32, torch.bfloat16):
        for out, wide in outputs(M, N, dtype):
            got = m.moe_int8_matmul(tokens if wide is None else q, sx, w, sw, out=out,
                                    out_dtype=dtype)
            assert torch.equal(got, want.to(dtype)), (dtype, out is not None)
            assert wide is None or beside(wide, N)


def check_gate(m, T, E, H):
    """Whole numbers up to 8: every partial sum is one below 2^24."""
    assert 64 * H < 1 << 24
    x, w = (whole(s, -8, 9, n, H).to(torch.bfloat16) for s, n in ((T + E, T), (H, E)))
    want = (x.double() @ w.double().t().contiguous()).float()
    tokens = strided(x, 8)
    for out, wide in outputs(T, E, torch.float32):
        got = m.moe_gate_logits(tokens if wide is None else x, w, out=out)
        assert torch.equal(got, want), out is not None
        assert wide is None or beside(wide, E)


@gpu
@pytest.mark.parametrize("key,shape", flat(TILED))
def test_tiled_products(m, key, shape):
    M, N, Kb = shape
    check_int8(m, M, N, Kb)
    check_gate(m, M, N, Kb // 2)


@gpu
@pytest.mark.parametrize("key,shape", flat(DIRECT))
def test_direct_products(m, key, shape):
    M, N, Kb = shape
    check_int8(m, M, N, Kb)
    check_gate(m, M, N, Kb // 2)


@gpu
@pytest.mark.parametrize("key,shape", flat(FUSED))
def test_fused_products(m, key, shape):
    """The one launch against the definition: codes and scales by NumPy's float32, product exact."""
    M, N, K = shape
    g = torch.Generator(device="cuda").manual_seed(M + N + K)
    x = (2 * torch.randn(M, K, generator=g, device="cuda")).to(torch.bfloat16)
    _, _, w, sw = int8_operands(1, N, K)
    q, s = (torch.from_numpy(a).cuda() for a in ref.quant_int8(x.float().cpu().numpy()))
    want = int8_product(q, s, w, sw)
    tokens = strided(x, 8)
    for dtype in (torch.float32, torch.bfloat16):
        for out, wide in outputs(M, N, dtype):
            got = m.moe_int8_linear(tokens if wide is None else x, w, sw, out=out, out_dtype=dtype)
            assert torch.equal(got, want.to(dtype)), (dtype, out is not None)
            assert wide is None or beside(wide, N)


@gpu
@pytest.mark.parametrize("M", [40, 600])
def test_rows_too_far_apart_for_the_tiles(m, M):
    """Rows 8 MB apart: past the tiled kernel's 31-bit offsets the direct kernel takes the product,
    whatever the number of tokens."""
    N, K, ld = 130, 1040, (1 << 23) + 16
    q, sx, w, sw = int8_operands(M, N, K)
    wide = torch.empty(M, ld, dtype=torch.int8, device="cuda")
    wide[:, :K] = q
    got = m.moe_int8_matmul(wide[:, :K], sx, w, sw, out_dtype=torch.float32)
    assert torch.equal(got, int8_product(q, sx, w, sw))
    x, wg = (whole(s, -8, 9, n, K // 2).to(torch.bfloat16) for s, n in ((1, M), (2, N)))
    far = wide.view(torch.bfloat16)
    far[:, :K // 2] = x
    want = (x.double() @ wg.double().t().contiguous()).float()
    assert torch.equal(m.moe_gate_logits(far[:, :K // 2], wg), want)


@gpu
def test_one_dirty_workspace_for_split_products(m, probe):
    """One buffer for the largest batch, full of NaN bits at first and then of the batches' before:
    products with K split by several numbers add their own partial sums only."""
    N, H, most = 896, 7168, 700
    wg = whole(1, -8, 9, N, H).to(torch.bfloat16)
    q, sx, w8, sw = int8_operands(most, N, H)
    x = whole(2, -8, 9, most, H).to(torch.bfloat16)
    want8, want = int8_product(q, sx, w8, sw), (x.double() @ wg.double().t().contiguous()).float()
    ws = torch.full((max(m.moe_gate_workspace_size(most, N, H),
                         m.moe_int8_matmul_workspace_size(most, N, H)),), 0xFF, dtype=torch.uint8,
                    device="cuda")
    splits = set()
    for T in (17, 64, 100, 33, 128, 250, 1, 400, most, 48):
        splits |= {picked(probe, T, N, Kb)[1] for Kb in (H, 2 * H)}
        assert torch.equal(m.moe_gate_logits(x[:T], wg, workspace=ws), want[:T]), T
        got = m.moe_int8_matmul(q[:T], sx[:T], w8, sw, out_dtype=torch.float32, workspace=ws)
        assert torch.equal(got, want8[:T]), T
    assert len(splits) >= 5
