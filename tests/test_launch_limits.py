"""Calls with more work than one launch takes (fewer than 2^32 threads): every row is done."""
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
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def probe():
    lib = ctypes.CDLL(PROBE)
    lib.probe_most_blocks.argtypes, lib.probe_most_blocks.restype = [ctypes.c_int], ctypes.c_int64
    lib.probe_most_items.argtypes = [ctypes.c_int, ctypes.c_int64, ctypes.c_int64]
    lib.probe_most_items.restype = ctypes.c_int64
    return lib


@pytest.fixture(scope="module")
def m():
    import mxfp8_mxfp4_experts_amd as mod
    return mod


@pytest.fixture(autouse=True)
def memory_given_back():
    """These tests take up to 200 GiB."""
    yield
    if torch.cuda.is_available():
        torch.cuda.empty_cache()


@pytest.mark.parametrize("threads", [64, 256, 512, 1024])
def test_a_launch_stays_below_its_limit(probe, threads):
    most = probe.probe_most_blocks(threads)
    assert most * threads < 1 << 32 <= (most + 1) * threads
    for per_block in (1, 4, 8):
        for units in (1, 3, 7, 2048, 65536):
            items = probe.probe_most_items(threads, per_block, units)
            assert items >= 1 and -(-items * units // per_block) <= most
            assert -(-(items + 1) * units // per_block) >= most


@pytest.mark.parametrize("R", [1, 2048, 1 << 29, (1 << 30) - 5, 1 << 30])
def test_grouped_launches_fit(probe, R):
    """Whatever the routes and experts, the tile taken has a workgroup for each of them (columns as
    many as memory holds)."""
    tiles = [(256, 256, 512), (128, 128, 256), (64, 128, 256), (64, 64, 256), (32, 64, 256)]
    for E in (1, 2, 64, 4096):
        for N in (1, 16, 64, 128, 129):
            for K in (16, 128, 1024, 7168):
                bm, bn, threads = tiles[probe.probe_fp8_grouped(R, E, N, K)]
                blocks = (R // bm + min(E, R)) * (-(-N // bn)) + 7
                assert blocks * threads < 1 << 32, (E, N, K)


@gpu
@pytest.mark.parametrize("kind", [BF16, F32])
def test_sort_and_unsort_of_many_short_tokens(m, kind):
    """2^26 + 5 tokens of few elements, of which some have a row: the first, those around the
    launches' border, the last."""
    T, H, n = (1 << 26) + 5, 2, 16
    at = torch.tensor([0, 3, (1 << 24) - 1, 1 << 24, (1 << 26) - 5, (1 << 26) - 4, (1 << 26) - 1,
                       1 << 26, T - 1], device=DEV)
    row = torch.full((T,), -1, dtype=torch.int32, device=DEV)
    row[at] = torch.arange(len(at), dtype=torch.int32, device=DEV) + 2
    x = torch.zeros(T, H, dtype=kind, device=DEV)
    x[at] = torch.arange(1, 1 + len(at) * H, device=DEV).view(-1, H).to(kind)
    rows = torch.full((n, H), 77.0, dtype=kind, device=DEV)
    m.moe_sort_tokens(x, row, 1, rows=rows)
    want = torch.full_like(rows, 77.0)
    want[2:2 + len(at)] = x[at]
    assert torch.equal(rows, want)
    w = torch.full((T, 1), 2.0, device=DEV)
    out = torch.full_like(x, 77.0)
    for weights, scale in ((None, 1.0), (w, 2.0)):
        out.fill_(77.0)
        m.moe_unsort_tokens(rows, row, weights, 1, out=out)
        assert torch.equal(out, x * scale)
    drows, dw = torch.full_like(rows, 77.0), torch.full_like(w, 77.0)
    m.moe_unsort_tokens_grad(x, rows, row, w, drows=drows, dw=dw)
    assert torch.equal(drows[2:2 + len(at)], 2.0 * x[at]) and (drows[2 + len(at):] == 77.0).all()
    dots = torch.zeros_like(dw)
    dots[at, 0] = (x[at].double() ** 2).sum(1).float()   # whole numbers: exact
    assert torch.equal(dw, dots)


@gpu
def test_gradients_of_many_longer_tokens(m):
    """2^24 + 3 tokens whose rows take a workgroup each."""
    T, H, n = (1 << 24) + 3, 520, 8
    at = torch.tensor([0, 1 << 23, (1 << 24) - 2, (1 << 24) - 1, 1 << 24, T - 1], device=DEV)
    row = torch.full((T,), -1, dtype=torch.int32, device=DEV)
    row[at] = torch.arange(len(at), dtype=torch.int32, device=DEV)
    dout = torch.empty(T, H, dtype=BF16, device=DEV)     # only the rows that have a route count
    dout[at] = torch.randint(-4, 5, (len(at), H), device=DEV).to(BF16)
    rows = torch.randint(-4, 5, (n, H), device=DEV).to(BF16)
    w = torch.full((T, 1), 0.5, device=DEV)
    drows, dw = torch.full_like(rows, 77.0), torch.full_like(w, 77.0)
    m.moe_unsort_tokens_grad(dout, rows, row, w, drows=drows, dw=dw)
    k = len(at)
    assert torch.equal(drows[:k], 0.5 * dout[at]) and (drows[k:] == 77.0).all()
    dots = torch.zeros_like(dw)
    dots[at, 0] = (dout[at].float() * rows[:k].float()).sum(1)
    assert torch.equal(dw, dots)


@gpu
def test_quantising_many_long_tokens(m):
    """4194303 tokens of 16400 elements (137 GB): 2^27 pieces of 512 and more."""
    T, H = (1 << 22) - 1, 16400
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 215 << 30:
        pytest.skip("needs 215 GiB of GPU memory")
    border = (1 << 27) // 33                       # 33 pieces a token
    at = torch.tensor([0, border - 1, border, border + 1, T - 1], device=DEV)
    x = torch.empty(T, H, dtype=BF16, device=DEV)  # other tokens hold anything
    some = ref.tokens(len(at), H, 1)
    x[at] = some.to(DEV)
    xq = torch.empty(T, H, dtype=torch.uint8, device=DEV)
    xq[at] = 0xAA
    xs = torch.full((ref.blocks(H), T), -1.0, device=DEV)
    m.moe_quant_fp8(x, xq=xq, xs=xs)
    del x
    q, s = ref.quant(some)
    assert torch.equal(xq[at].cpu(), q) and torch.equal(xs[:, at].cpu(), s)
    assert not (xs == -1.0).any()                  # a scale is positive or NaN


@gpu
def test_direct_product_of_many_tokens(m):
    """4194303 tokens whose scales' blocks are 1 GiB apart, so that the tiled kernel does not reach
    them; 2^22 workgroups and more. Whole numbers: exact in any order."""
    M, N, K = (1 << 22) - 1, 272, 144
    g = torch.Generator(device=DEV).manual_seed(1)
    codes = lambda *n: torch.randint(-4, 5, n, generator=g, device=DEV, dtype=torch.int8  # noqa: E731
                                     ).float().to(ref.FP8)
    q, w, w_s = codes(M, K), codes(N, K), torch.ones(3, 2, device=DEV)
    xs = 2.0 ** torch.randint(-1, 2, (2, M), generator=g, device=DEV).float()
    want = m.moe_fp8_matmul(q, xs, w, w_s)
    rows = torch.arange(0, M, 65537, device=DEV)
    exact = (q[rows].float() * xs[:, rows].t().repeat_interleave(128, 1)[:, :K]) @ w.float().t().contiguous()
    assert torch.equal(want[rows], exact.to(BF16))
    step = 1 << 28
    far = torch.empty(step + M, device=DEV).as_strided((2, M), (step, 1))
    far.copy_(xs)
    out = torch.full_like(want, 77.0)
    m.moe_fp8_matmul(q, far, w, w_s, out=out)
    assert torch.equal(out, want)


@gpu
def test_grouped_product_of_many_routes(m):
    """2^30 routes to 16 tokens, one column: 2^24 tiles of 64 rows and more."""
    R, E, T, k, K = 1 << 30, 3, 16, 64, 16
    g = torch.Generator(device=DEV).manual_seed(1)
    codes = lambda *n: torch.randint(-4, 5, n, generator=g, device=DEV, dtype=torch.int8  # noqa: E731
                                     ).float().to(ref.FP8)
    q, w = codes(T, K), codes(E, 1, K)
    route = torch.arange(R, dtype=torch.int32, device=DEV) % (T * k)
    offs = torch.tensor([0, R // 3, R - 77, R], dtype=torch.int32, device=DEV)
    out = torch.full((R, 1), 77.0, dtype=BF16, device=DEV)
    m.moe_fp8_grouped(q, torch.ones(1, T, device=DEV), w, torch.ones(E, 1, 1, device=DEV), offs,
                      route, k, out=out)
    each = (q.float() @ w[:, 0].float().t().contiguous()).to(BF16)         # [T, E], exact
    at = offs.tolist()
    for e in range(E):
        for a in range(at[e], at[e + 1], 1 << 27):
            b = min(a + (1 << 27), at[e + 1])
            assert torch.equal(out[a:b, 0], each[(route[a:b] // k).long(), e])


@gpu
def test_mxfp8_quantisation_of_many_tokens(m):
    """2^24 + 3 tokens, a workgroup each."""
    T, H = (1 << 24) + 3, 32
    at = torch.tensor([0, 1, (1 << 24) - 2, (1 << 24) - 1, 1 << 24, T - 1], device=DEV)
    x = torch.zeros(T, H, dtype=BF16, device=DEV)
    x[at] = ref.tokens(len(at), H, 1).to(DEV)
    xq = torch.full((T, H), 0xAA, dtype=torch.uint8, device=DEV)
    xs = torch.full((T, 1), 0xAA, dtype=torch.uint8, device=DEV)
    m.moe_quant_mxfp8(x, xq=xq, xs=xs)
    q, s = m.moe_quant_mxfp8(x[at].contiguous())
    assert torch.equal(xq[at], q) and torch.equal(xs[at], s)
    assert not (xs == 0xAA).any()                  # 2^43: none of these values has it


@gpu
@pytest.mark.parametrize("T,E", [((1 << 24) + 3, 5), ((1 << 24) + 3, 1025)])
def test_routing_of_many_tokens(m, T, E):
    """2^24 + 3 tokens, a workgroup each up to 1024 experts."""
    logits = torch.zeros(T, E, device=DEV)
    at = torch.tensor([0, 1, (1 << 24) - 2, (1 << 24) - 1, 1 << 24, T - 1], device=DEV)
    logits[at] = torch.randn(len(at), E, generator=torch.Generator().manual_seed(1)).to(DEV)
    idx = torch.full((T, 2), -7, dtype=torch.int32, device=DEV)
    w = torch.full((T, 2), -7.0, device=DEV)
    m.moe_route(logits, None, 2, topk_idx=idx, topk_w=w)
    want, want_w = m.moe_route(logits[at].contiguous(), None, 2)
    assert torch.equal(idx[at], want) and torch.equal(w[at], want_w)
    assert (idx >= 0).all() and (w > 0).all()


@gpu
@pytest.mark.parametrize("atomic", [False, True])
def test_combine_of_many_tokens(m, atomic):
    """2^26 + 3 tokens of 256 columns, of which some have an expert: those around the launches'
    border and the last."""
    T, H, I = (1 << 26) + 3, 256, 128
    mode = m.COMBINE_ATOMIC if atomic else m.COMBINE_DETERMINISTIC
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 130 << 30:
        pytest.skip("needs 130 GiB of GPU memory")
    at = torch.tensor([0, 5, (1 << 26) - 2, (1 << 26) - 1, 1 << 26, T - 1], device=DEV)
    n = len(at)
    g = torch.Generator().manual_seed(1)
    w2 = torch.randint(0, 256, (1, H, I // 2), generator=g, dtype=torch.uint8).to(DEV)
    w2_s = torch.full((1, H, I // 32), 127, dtype=torch.uint8, device=DEV)
    codes = torch.randint(0, 0x40, (n, I), generator=g, dtype=torch.uint8).to(DEV)

    def run(T, at):
        idx = torch.full((T, 1), -1, dtype=torch.int32, device=DEV)
        idx[at] = 0
        ws = torch.full((m.moe_workspace_size(T, 1, 1, H, I, mode),), 0x42, dtype=torch.uint8,
                        device=DEV)
        offs, sorted_route, row = m.moe_permute(idx, 0, 1, ws)
        hq = torch.empty(T, I, dtype=torch.uint8, device=DEV)
        hq[:n] = codes
        hs = torch.empty(T, I // 32, dtype=torch.uint8, device=DEV)
        hs[:n] = 127
        w = torch.ones(T, 1, device=DEV)
        out = torch.full((T, H), 77.0, dtype=BF16, device=DEV)
        m.moe_fc2_combine(hq, hs, T, 1, offs, sorted_route, row, w, w2, w2_s, ws, out=out, mode=mode)
        return out
    want = run(n, torch.arange(n, device=DEV))
    assert torch.isfinite(want).all() and (want != 0).any(1).all()
    out = run(T, at)
    # The two may take another kernel: one rounding of the float sum to bf16 apart (the sums differ
    # by their order, far below that).
    assert ((out[at].float() - want.float()).abs() <= 2.0 ** -7 * want.float().abs() + 1e-3).all()
    out[at] = 0.0
    assert not out.any()
