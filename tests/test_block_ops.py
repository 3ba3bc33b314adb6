"""The operators around the experts: refusals (no GPU needed) and parity with
plain 64-bit references on the GPU."""
import math
import os

import numpy as np
import pytest
import torch

import block_ref as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "mxfp8_mxfp4_experts_amd", "libmi355moe.so")
pytestmark = pytest.mark.skipif(not os.path.exists(LIB), reason="libmi355moe.so not built")

FAKE = 1 << 20          # aligned, never dereferenced by a failing call
MIS = FAKE + 2
INF, NAN = math.inf, math.nan
OK, NULL, SHAPE, ALIGN, ENUM, WORKSPACE = 0, 1, 2, 3, 4, 5


@pytest.fixture(scope="module")
def lib():
    from mxfp8_mxfp4_experts_amd import _binding
    return _binding.load_library(LIB)


# ---------------------------------------------------------------------------
# Refusals: the C entries check before any HIP call.

def test_add_rmsnorm_refusals(lib):
    def call(x=FAKE, ld_x=64, r=FAKE, ld_r=64, w=FAKE, eps=1e-6, T=4, H=64, q8=1, h=FAKE, ld_h=64,
             y=FAKE, ld_y=64, xq=FAKE, xs=FAKE):
        return lib.moe_add_rmsnorm(x, ld_x, r, ld_r, w, eps, T, H, q8, h, ld_h, y, ld_y, xq, xs,
                                   None)
    assert call(q8=3) == ENUM and call(q8=-1) == ENUM
    for bad in (dict(T=-1), dict(T=1 << 22), dict(H=0), dict(H=60), dict(H=32776, ld_x=40000),
                dict(ld_x=56), dict(ld_r=56), dict(ld_h=56), dict(ld_y=56), dict(eps=-1.0),
                dict(eps=NAN), dict(eps=INF), dict(H=40)):   # H % 32 with MXFP8
        assert call(**bad) == SHAPE, bad
    for bad in (dict(x=None), dict(w=None), dict(xq=None), dict(xs=None), dict(y=None, q8=0)):
        assert call(**bad) == NULL, bad
    for bad in (dict(x=MIS), dict(r=MIS), dict(w=MIS), dict(h=MIS), dict(y=MIS), dict(xq=MIS),
                dict(xs=FAKE + 2), dict(ld_x=68), dict(ld_r=68), dict(ld_h=68), dict(ld_y=68)):
        assert call(**bad) == ALIGN, bad
    assert call(T=0, x=None, w=None, xq=None) == OK
    assert call(r=None, ld_r=0, h=None, ld_h=0, y=None, ld_y=0, T=0) == OK


def test_quant_int8_refusals(lib):
    f = lib.moe_quant_int8
    assert f(FAKE, 64, -1, 64, FAKE, FAKE, None) == SHAPE
    assert f(FAKE, 64, 1, 60, FAKE, FAKE, None) == SHAPE
    assert f(FAKE, 56, 1, 64, FAKE, FAKE, None) == SHAPE
    assert f(FAKE, 40000, 1, 32776, FAKE, FAKE, None) == SHAPE
    for k in range(3):
        p = [FAKE] * 3
        p[k] = None
        assert f(p[0], 64, 1, 64, p[1], p[2], None) == NULL
        p[k] = MIS
        assert f(p[0], 64, 1, 64, p[1], p[2], None) == ALIGN
    assert f(FAKE, 68, 2, 64, FAKE, FAKE, None) == ALIGN
    assert f(None, 64, 0, 64, None, None, None) == OK


def test_int8_matmul_refusals(lib):
    def call(xq=FAKE, ld=64, xs=FAKE, w=FAKE, ws=FAKE, M=4, N=7, K=64, kind=0, out=FAKE, ldo=7,
             wk=FAKE, nb=1 << 40):
        return lib.moe_int8_matmul(xq, ld, xs, w, ws, M, N, K, kind, out, ldo, wk, nb, None)
    assert call(kind=2) == ENUM and call(kind=-1) == ENUM
    for bad in (dict(M=-1), dict(M=1 << 22), dict(N=0), dict(N=(1 << 20) + 1), dict(K=0),
                dict(K=72, ld=80), dict(K=131072, ld=131072), dict(ld=48), dict(ldo=6)):
        assert call(**bad) == SHAPE, bad
    for name in ("xq", "xs", "w", "ws", "out"):
        assert call(**{name: None}) == NULL, name
    for bad in (dict(xq=MIS), dict(w=MIS), dict(xs=MIS), dict(ws=MIS), dict(out=MIS), dict(ld=72),
                dict(wk=FAKE + 16), dict(kind=1, out=MIS)):
        assert call(**bad) == ALIGN, bad
    assert call(M=0, xq=None, out=None) == OK
    for M, N, K in ((0, 7, 64), (4, 0, 64), (4, 7, 24), (-1, 7, 64)):
        n = lib.moe_int8_workspace_size(M, N, K)
        assert (n == 0) == (M < 0 or N == 0 or K == 24)
    assert lib.moe_int8_workspace_size(8, 100, 64) >= 8 * 64 + 8 * 4


def test_int8_linear_refusals(lib):
    def call(x=FAKE, ld=64, w=FAKE, ws=FAKE, M=4, N=7, K=64, kind=0, out=FAKE, ldo=7, wk=FAKE,
             nb=1 << 40):
        return lib.moe_int8_linear(x, ld, w, ws, M, N, K, kind, out, ldo, wk, nb, None)
    assert call(kind=2) == ENUM
    for bad in (dict(M=-1), dict(N=0), dict(K=72, ld=80), dict(K=32784, ld=32784), dict(ld=48),
                dict(ldo=6)):
        assert call(**bad) == SHAPE, bad
    for name in ("x", "w", "ws", "out", "wk"):
        assert call(**{name: None}) == NULL, name
    for bad in (dict(x=MIS), dict(w=MIS), dict(ws=MIS), dict(out=MIS), dict(ld=68),
                dict(wk=FAKE + 16)):
        assert call(**bad) == ALIGN, bad
    assert call(nb=lib.moe_int8_workspace_size(4, 7, 64) - 1) == WORKSPACE
    assert call(M=0, x=None) == OK


def test_gate_refusals(lib):
    def call(x=FAKE, ld=64, w=FAKE, T=4, E=7, H=64, out=FAKE, ldo=7, wk=FAKE, nb=1 << 40):
        return lib.moe_gate_logits(x, ld, w, T, E, H, out, ldo, wk, nb, None)
    for bad in (dict(T=-1), dict(T=1 << 22), dict(E=0), dict(E=4097, ldo=4097), dict(H=0),
                dict(H=60), dict(H=(1 << 20) + 8, ld=1 << 21), dict(ld=56), dict(ldo=6)):
        assert call(**bad) == SHAPE, bad
    for name in ("x", "w", "out"):
        assert call(**{name: None}) == NULL, name
    for bad in (dict(x=MIS), dict(w=MIS), dict(out=MIS), dict(ld=68), dict(wk=FAKE + 16)):
        assert call(**bad) == ALIGN, bad
    assert call(T=0, x=None) == OK
    assert lib.moe_gate_workspace_size(-1, 7, 64) == 0


def test_gate_and_int8_refuse_a_small_workspace(lib):
    """Where partial sums are needed, one byte too few is refused."""
    need = lib.moe_gate_workspace_size(256, 896, 7168)
    if need:
        assert lib.moe_gate_logits(FAKE, 7168, FAKE, 256, 896, 7168, FAKE, 896, FAKE, need - 1,
                                   None) == WORKSPACE
        assert lib.moe_gate_logits(FAKE, 7168, FAKE, 256, 896, 7168, FAKE, 896, None, 0,
                                   None) == NULL


def test_workspaces_grow_with_the_rows(lib):
    """A workspace for M rows serves every smaller M."""
    for N, K in ((1, 64), (896, 7168), (2051, 1040), (3584, 7168)):
        sizes = [lib.moe_int8_workspace_size(M, N, K) for M in range(0, 3000, 7)]
        assert sizes == sorted(sizes)
    sizes = [lib.moe_gate_workspace_size(T, 896, 7168) for T in range(0, 9000, 13)]
    assert sizes == sorted(sizes) and sizes[0] == 0 < sizes[1]


def test_route_groups_refusals(lib):
    def call(l=FAKE, ld=64, b=FAKE, T=4, E=64, K=4, G=4, KG=2, score=0, group=1, ren=1, idx=FAKE,
             w=FAKE):
        return lib.moe_route_groups(l, ld, b, T, E, K, G, KG, score, group, ren, 1.0, idx, w, None)
    for bad in (dict(T=-1), dict(T=1 << 22), dict(E=0), dict(E=4160, ld=5000, G=64), dict(K=0),
                dict(K=33), dict(K=65, KG=4, E=512, ld=512), dict(G=0), dict(G=3), dict(KG=0),
                dict(KG=5), dict(G=65, E=65, ld=65), dict(ld=63)):
        assert call(**bad) == SHAPE, bad
    for bad in (dict(score=2), dict(score=-1), dict(group=2), dict(group=-1)):
        assert call(**bad) == ENUM, bad
    for name in ("l", "idx", "w"):
        assert call(**{name: None}) == NULL, name
    for name in ("l", "idx", "w", "b"):
        assert call(**{name: MIS}) == ALIGN, name
    assert call(T=0, l=None, idx=None) == OK


def test_binding_refuses_cpu_tensors():
    import mxfp8_mxfp4_experts_amd as m
    x = torch.zeros(2, 64, dtype=torch.bfloat16)
    w = torch.ones(64, dtype=torch.bfloat16)
    for call in (lambda: m.moe_add_rmsnorm(x, w, 1e-6), lambda: m.moe_quant_int8(x),
                 lambda: m.moe_gate_logits(x, x), lambda: m.moe_route_groups(x.float(), None, 2),
                 lambda: m.moe_int8_linear(x, x, w), lambda: m.moe_int8_matmul(x, w, x, w)):
        with pytest.raises(ValueError, match="GPU tensor"):
            call()


# ---------------------------------------------------------------------------
# GPU parity.

def test_tensor_checks_answer_without_throwing(lib):
    """The compiled checks say no to what is not a plain GPU tensor, and no
    exception passes through them."""
    from mxfp8_mxfp4_experts_amd import _tensor_args as ck
    bf = torch.bfloat16
    odd = [torch.zeros(2, 4, dtype=bf), torch.zeros(2, 4, dtype=bf).to_sparse(), torch.zeros(()),
           torch.zeros(2, 4, dtype=bf, device="meta"), None, 3, [1.0]]
    for t in odd:
        assert ck.head(t) is None and ck.plain(t, bf, 2, 4, 0) == -1, type(t)
    for args in ((odd[0], bf, 2, 4), (odd[0], "bf16", 2, 4, 0), (odd[0], bf, 2.5, 4, 0)):
        with pytest.raises(TypeError):
            ck.plain(*args)


gpu = pytest.mark.gpu


@gpu
@pytest.mark.parametrize("M,N,K", [(9, 33, 16), (16, 896, 1024), (17, 64, 512), (33, 131, 528),
                                   (64, 512, 512), (15, 70, 2048), (24, 40, 3600), (28, 66, 1104),
                                   (130, 77, 176), (257, 18, 272), (5, 9, 7168)])
@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32])
def test_int8_linear_equals_its_two_calls(M, N, K, out_dtype):
    """One launch or two, with one block of tokens or several: the same bits
    (also where a token holds a NaN), into rows of a wider buffer."""
    import mxfp8_mxfp4_experts_amd as m
    g = torch.Generator().manual_seed(M * N + K)
    x = torch.randn(M, K, generator=g).bfloat16()
    x[M // 2, K - 1] = NAN
    x = torch.cat([x, x], 1).cuda()[:, :K]
    w = torch.randint(-127, 128, (N, K), generator=g, dtype=torch.int8).cuda()
    sw = torch.rand(N, generator=g).cuda()
    q, s = m.moe_quant_int8(x)
    want = m.moe_int8_matmul(q, s, w, sw, out_dtype=out_dtype)
    wide = torch.full((M, N + 24), 7.0, dtype=out_dtype, device="cuda")
    got = m.moe_int8_linear(x, w, sw, out=wide[:, :N])
    assert torch.equal(got.isnan(), want.isnan()) and want.isnan().any(1).sum() == 1
    assert torch.equal(got.nan_to_num(0), want.nan_to_num(0))
    assert (wide[:, N:] == 7).all()


@gpu
def test_binding_refusals():
    """What the compiled checks refuse is named by the binding."""
    import mxfp8_mxfp4_experts_amd as m
    e = dict(device="cuda")
    x = torch.zeros(4, 64, dtype=torch.bfloat16, **e)
    w = torch.ones(64, dtype=torch.bfloat16, **e)
    q, s = torch.zeros(4, 64, dtype=torch.int8, **e), torch.zeros(4, **e)
    w8, s8 = torch.zeros(32, 64, dtype=torch.int8, **e), torch.ones(32, **e)
    logits = torch.zeros(4, 16, **e)
    for call in (
            lambda: m.moe_add_rmsnorm(x.cpu(), w, 1e-6), lambda: m.moe_add_rmsnorm(x[0], w, 1e-6),
            lambda: m.moe_add_rmsnorm(x.float(), w, 1e-6),
            lambda: m.moe_add_rmsnorm(x, w[:-1], 1e-6),
            lambda: m.moe_add_rmsnorm(x, w.repeat(2)[::2], 1e-6),
            lambda: m.moe_add_rmsnorm(x, w, 1e-6, residual=x[:3]),
            lambda: m.moe_add_rmsnorm(x, w, 1e-6, y=x.t().contiguous().t()),
            lambda: m.moe_add_rmsnorm(x, w, 1e-6, q8=m.Q8_INT8, xq=q.view(torch.uint8)),
            lambda: m.moe_add_rmsnorm(x, w, 1e-6, q8=m.Q8_MXFP8, xs=s),
            lambda: m.moe_quant_int8(x, xs=s[:3]), lambda: m.moe_quant_int8(x.to_sparse()),
            lambda: m.moe_int8_matmul(q, s, w8[:, :32], s8),
            lambda: m.moe_int8_matmul(q, s, w8, s8.cpu()),
            lambda: m.moe_int8_matmul(q, s.double(), w8, s8),
            lambda: m.moe_int8_linear(x, w8, s8, out=torch.zeros(4, 31, **e)),
            lambda: m.moe_int8_linear(x, w8, s8, out_dtype=torch.float16),
            lambda: m.moe_int8_linear(x, w8, s8, workspace=s),
            lambda: m.moe_gate_logits(x, w), lambda: m.moe_gate_logits(x, x[:, :32]),
            lambda: m.moe_gate_logits(x, x, out=torch.zeros(4, 4, dtype=torch.bfloat16, **e)),
            lambda: m.moe_route_groups(logits, s, 2),
            lambda: m.moe_route_groups(logits, None, 2, topk_w=torch.zeros(4, 3, **e)),
            lambda: m.moe_route_groups(logits.half(), None, 2)):
        with pytest.raises((ValueError, RuntimeError)):
            call()


@pytest.fixture(scope="module")
def m():
    import mxfp8_mxfp4_experts_amd as mod
    return mod


def rand(seed, *shape, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return scale * torch.randn(*shape, generator=g)


def window(t, pad=8):
    """The same rows as a column window of a wider buffer on the GPU (and that buffer)."""
    T, C = t.shape
    wide = torch.full((T, C + 3 * pad), 77.0, device="cuda").to(t.dtype)
    wide[:, pad:pad + C] = t.cuda()
    return wide[:, pad:pad + C], wide


def check_y(got, y64, H):
    """bf16(y): half a bf16 step (2^-8 relative, 2^-134 below the normal range) past y's own
    float32 error."""
    tol = np.abs(y64) * (2.0 ** -8 + ref.norm_rel(H)) * (1 + 2.0 ** -8) + 2.0 ** -133
    assert (np.abs(ref.f64(got) - y64) <= tol).all()


def check_mxfp8(xq, xs, y64, H):
    """Each block's exponent is the rule's for its absmax within y's float32 error; each code lies
    between the nearest codes of y at both ends of that error."""
    d = 2 * ref.norm_rel(H)
    g = y64.reshape(len(y64), -1, 32)
    e = xs.cpu().numpy().astype(np.int64) - 127
    amax = np.abs(g).max(2)
    with np.errstate(divide="ignore"):
        lo, hi = (np.clip(np.ceil(np.log2(amax * f / 448.0) - 1e-12), -127, 127)
                  for f in (1 - d, 1 + d))
    assert ((e >= lo) & (e <= hi)).all()
    v = xq.cpu().view(torch.float8_e4m3fn).double().numpy().reshape(g.shape)
    s = np.ldexp(g, -e[..., None])
    near = [np.clip(s * f, -448, 448).astype(np.float32) for f in (1 - d, 1 + d)]
    near = [torch.from_numpy(n).to(torch.float8_e4m3fn).double().numpy() for n in near]
    assert ((v >= np.minimum(*near)) & (v <= np.maximum(*near))).all()


def check_int8(xq, xs, y64, H):
    d = ref.norm_rel(H) + 4 * ref.U
    s64 = np.maximum(np.abs(y64).max(1) / 127.0, 2.0 ** -126)
    s = ref.f64(xs)
    assert (np.abs(s - s64) <= d * s64).all()
    z = y64 / s64[:, None]
    q = ref.f64(xq.float())
    lo, hi = np.rint(z - 2 * d * np.abs(z)), np.rint(z + 2 * d * np.abs(z))
    assert ((q >= lo) & (q <= hi)).all()


NORM_SHAPES = [(1, 8), (3, 24), (1, 32), (5, 96), (2, 512), (7, 1000), (1, 7168), (9, 7168),
               (3, 8200), (2, 16416), (2, 32768), (300, 160)]


@gpu
@pytest.mark.parametrize("T,H", NORM_SHAPES)
@pytest.mark.parametrize("q8", ["none", "mxfp8", "int8"])
def test_add_rmsnorm(m, T, H, q8):
    if q8 == "mxfp8" and H % 32:
        pytest.skip("MXFP8 blocks are 32 wide")
    x = rand(T * H, T, H, scale=1.5).to(torch.bfloat16)
    r = rand(T * H + 1, T, H, scale=4.0).to(torch.bfloat16)
    w = (1 + 0.2 * rand(H, H)).to(torch.bfloat16)
    mode = dict(none=m.Q8_NONE, mxfp8=m.Q8_MXFP8, int8=m.Q8_INT8)[q8]
    h, y, xq, xs = m.moe_add_rmsnorm(x.cuda(), w.cuda(), 1e-6, residual=r.cuda(), q8=mode)
    h64, y64, hb = ref.norm(x, r, w, float(np.float32(1e-6)))
    assert np.array_equal(ref.f64(h), hb)
    check_y(y, y64, H)
    if q8 == "mxfp8":
        check_mxfp8(xq, xs, y64, H)
    elif q8 == "int8":
        check_int8(xq, xs, y64, H)
    else:
        assert xq is None and xs is None


@gpu
def test_add_rmsnorm_without_residual_or_y(m):
    x, w = rand(1, 5, 7168).to(torch.bfloat16), torch.ones(7168, dtype=torch.bfloat16)
    _, y64, _ = ref.norm(x, None, w, 0.0)
    h, y, xq, xs = m.moe_add_rmsnorm(x.cuda(), w.cuda(), 0.0, q8=m.Q8_MXFP8, want_y=False)
    assert h is None and y is None
    check_mxfp8(xq, xs, y64, 7168)
    h, y, xq, xs = m.moe_add_rmsnorm(x.cuda(), w.cuda(), 0.0)
    assert h is None and xq is None
    check_y(y, y64, 7168)
    with pytest.raises(m.MoEError):
        m.moe_add_rmsnorm(x.cuda(), w.cuda(), 0.0, want_y=False)


@gpu
def test_add_rmsnorm_windows_and_in_place(m):
    T, H = 6, 256
    x, r = rand(3, T, H).to(torch.bfloat16), rand(4, T, H).to(torch.bfloat16)
    w = (1 + 0.1 * rand(5, H)).to(torch.bfloat16)
    _, y64, hb = ref.norm(x, r, w, float(np.float32(1e-5)))
    (xw, xb), (rw, rb) = window(x), window(r)
    yw, yb = window(torch.zeros(T, H, dtype=torch.bfloat16))
    h, y, xq, xs = m.moe_add_rmsnorm(xw, w.cuda(), 1e-5, residual=rw, residual_out=rw, y=yw,
                                     q8=m.Q8_INT8)
    assert h.data_ptr() == rw.data_ptr() and y.data_ptr() == yw.data_ptr()
    assert np.array_equal(ref.f64(rw), hb)
    check_y(yw, y64, H)
    check_int8(xq, xs, y64, H)
    for wide in (rb, yb, xb):   # the columns outside the windows
        assert (wide[:, :8].float() == 77).all() and (wide[:, 8 + H:].float() == 77).all()
    # y over x, the sum over the residual
    xc, rc = x.cuda(), r.cuda()
    m.moe_add_rmsnorm(xc, w.cuda(), 1e-5, residual=rc, residual_out=rc, y=xc)
    assert np.array_equal(ref.f64(rc), hb)
    check_y(xc, y64, H)


@gpu
def test_add_rmsnorm_zero_tiny_and_odd_rows(m):
    """Zero rows, values near both ends of bf16, and rows holding NaN or an infinity."""
    H = 512
    x = rand(11, 8, H).to(torch.bfloat16)
    x[0] = 0
    x[1] *= 2.0 ** -120
    x[2] *= 2.0 ** 50                 # squares stay finite
    x[3, 5] = NAN
    x[4, 7] = INF
    x[5] *= 2.0 ** 100                # squares overflow float: rstd is 0
    w = torch.ones(H, dtype=torch.bfloat16)
    fine = [0, 1, 2, 6, 7]
    _, y64, _ = ref.norm(x, None, w, float(np.float32(1e-6)))
    _, y, xq, xs = m.moe_add_rmsnorm(x.cuda(), w.cuda(), 1e-6, q8=m.Q8_INT8)
    check_y(y[fine], y64[fine], H)
    check_int8(xq[fine], xs[fine], y64[fine], H)
    assert (xs[0].item() == 2.0 ** -126) and (xq[0] == 0).all()
    assert torch.isnan(y[3]).all() and torch.isnan(xs[3]) and (xq[3] == 0).all()
    assert torch.isnan(xs[4]) and (xq[4] == 0).all()
    assert (y[5] == 0).all() and (xq[5] == 0).all()
    _, _, xq, xs = m.moe_add_rmsnorm(x.cuda(), w.cuda(), 1e-6, q8=m.Q8_MXFP8)
    check_mxfp8(xq[fine], xs[fine], y64[fine], H)
    assert (xq[3] == 0).all() and (xs[3] == 0).all()      # NaN encodes as 0, ignored by the absmax
    # eps = 0 on a zero row: 0 times infinity
    _, y, _, _ = m.moe_add_rmsnorm(x[:1].cuda(), w.cuda(), 0.0)
    assert torch.isnan(y).all()


@gpu
@pytest.mark.parametrize("T,H", [(1, 8), (3, 24), (17, 1040), (2, 7168), (5, 8200), (2, 32768)])
def test_quant_int8_bit_exact(m, T, H):
    x = rand(T + H, T, H, scale=3.0).to(torch.bfloat16)
    x[0, 0] = 0.0
    x[0, H // 2] = x[0].abs().max() / 2      # falls between two whole numbers
    xw, _ = window(x)
    xq, xs = m.moe_quant_int8(xw)
    q, s = ref.quant_int8(x.float().numpy())
    assert np.array_equal(xs.cpu().numpy(), s)
    assert np.array_equal(xq.cpu().numpy(), q)


@gpu
def test_quant_int8_odd_rows(m):
    x = rand(2, 6, 64).to(torch.bfloat16)
    x[0] = 0
    x[1, 3] = NAN
    x[2, 63] = -INF
    x[3] = 9.2e-41                          # subnormal
    x[4] = 3.38e38
    xq, xs = m.moe_quant_int8(x.cuda())
    assert xs[0].item() == 2.0 ** -126 and (xq[0] == 0).all()
    for t in (1, 2):
        assert torch.isnan(xs[t]) and (xq[t] == 0).all()
    assert xs[3].item() == 2.0 ** -126
    assert (xq[4] == 127).all()
    q, s = ref.quant_int8(x[3:].float().numpy())
    assert np.array_equal(xq[3:].cpu().numpy(), q) and np.array_equal(xs[3:].cpu().numpy(), s)


def int8_case(seed, M, N, K):
    g = torch.Generator().manual_seed(seed)
    q = torch.randint(-127, 128, (M, K), generator=g, dtype=torch.int8)
    w = torch.randint(-128, 128, (N, K), generator=g, dtype=torch.int8)
    sx = 0.01 + torch.rand(M, generator=g)
    sw = 0.001 + 0.01 * torch.rand(N, generator=g)
    return q, sx, w, sw


# Tokens from one to 300 and more, odd widths, K with and without a rest below one stage: mostly the
# direct kernel and the small tiles (every variant and split has its shapes in
# test_dense_variants.py).
INT8_SHAPES = [(1, 1, 16), (1, 17, 48), (2, 16, 64), (15, 33, 112), (16, 64, 128), (17, 5, 144),
               (31, 100, 256), (33, 129, 272), (48, 224, 1040), (63, 255, 512), (65, 257, 640),
               (100, 96, 4096), (127, 448, 400), (129, 449, 1008), (255, 31, 2064),
               (257, 225, 1152), (300, 1000, 336), (513, 700, 176), (1, 3584, 7168),
               (64, 3584, 7168), (300, 2051, 1040)]


@gpu
@pytest.mark.parametrize("M,N,K", INT8_SHAPES)
@pytest.mark.parametrize("kind", [torch.bfloat16, torch.float32])
def test_int8_matmul_bit_exact(m, M, N, K, kind):
    q, sx, w, sw = int8_case(M + N + K, M, N, K)
    out = m.moe_int8_matmul(q.cuda(), sx.cuda(), w.cuda(), sw.cuda(), out_dtype=kind)
    want = ref.int8_matmul(q.numpy(), sx.numpy(), w.numpy(), sw.numpy())
    want = want.astype(np.float64) if kind is torch.float32 else ref.bf16_rne(want)
    assert out.dtype is kind and np.array_equal(ref.f64(out), want)


@gpu
@pytest.mark.parametrize("M", [2, 40, 200, 600])
def test_int8_matmul_windows(m, M):
    """Strided tokens and a strided output; the columns outside stay."""
    N, K = 136, 320
    q, sx, w, sw = int8_case(M, M, N, K)
    wide = torch.full((M, K + 32), 99, dtype=torch.int8, device="cuda")
    wide[:, 16:16 + K] = q.cuda()
    want = ref.int8_matmul(q.numpy(), sx.numpy(), w.numpy(), sw.numpy())
    for kind in (torch.bfloat16, torch.float32):
        ow, ob = window(torch.zeros(M, N, dtype=kind))
        m.moe_int8_matmul(wide[:, 16:16 + K], sx.cuda(), w.cuda(), sw.cuda(), out=ow)
        assert np.array_equal(ref.f64(ow), want if kind is torch.float32 else ref.bf16_rne(want))
        assert (ob[:, :8].float() == 77).all() and (ob[:, 8 + N:].float() == 77).all()


@gpu
def test_int8_matmul_largest_sums(m):
    """The largest K at codes whose sum reaches 2^31 - 2^21 does not overflow."""
    K = 131056
    q = torch.full((20, K), -128, dtype=torch.int8)
    w = torch.full((3, K), -128, dtype=torch.int8)
    one = torch.ones(20)
    out = m.moe_int8_matmul(q.cuda(), one.cuda(), w.cuda(), one[:3].cuda(), out_dtype=torch.float32)
    assert (out.cpu().double() == float(np.float32(K * 16384))).all()


@gpu
def test_int8_nonfinite_scale_shows(m):
    x = rand(1, 20, 64).to(torch.bfloat16)
    x[3, 3] = NAN
    x[4, 3] = INF
    _, _, w, sw = int8_case(1, 1, 24, 64)
    out = m.moe_int8_linear(x.cuda(), w.cuda(), sw.cuda())
    bad = torch.isnan(out).cpu()
    assert bad[3].all() and bad[4].all() and not bad[[0, 1, 2, 5, 19]].any()


@gpu
@pytest.mark.parametrize("M,N,K", [(1, 40, 64), (1, 3584, 7168), (3, 100, 1040), (8, 64, 32768),
                                   (16, 130, 528), (17, 129, 528), (300, 257, 272),
                                   (700, 300, 4096)])
def test_int8_linear_is_its_two_calls(m, M, N, K):
    x = rand(M, M, K, scale=2.0).to(torch.bfloat16)
    x[0, 1] = x[0].abs().max() / 2
    xw, _ = window(x)
    _, _, w, sw = int8_case(M + N, 1, N, K)
    got = m.moe_int8_linear(xw, w.cuda(), sw.cuda(), out_dtype=torch.float32)
    xq, xs = m.moe_quant_int8(xw)
    two = m.moe_int8_matmul(xq, xs, w.cuda(), sw.cuda(), out_dtype=torch.float32)
    assert torch.equal(got, two)
    q, s = ref.quant_int8(x.float().numpy())
    assert np.array_equal(got.cpu().numpy(), ref.int8_matmul(q, s, w.numpy(), sw.numpy()))


def check_gate(got, x, w):
    """Every logit within the bound of a float32 sum in any order (a rounding of up to 2^-23 of the
    partial sums' size per term), and the errors' rms within a random walk's."""
    x64, w64 = ref.f64(x), ref.f64(w)
    want, size = x64 @ w64.T, np.abs(x64) @ np.abs(w64).T
    err = np.abs(ref.f64(got) - want)
    n = x64.shape[1]
    assert (err <= (n + 1) * 2.0 ** -23 * size + 1e-45).all()
    walk = math.sqrt(n) * 2.0 ** -23 * math.sqrt((size ** 2).mean())
    assert math.sqrt((err ** 2).mean()) <= walk + 1e-45


GATE_SHAPES = [(1, 1, 8), (1, 896, 7168), (2, 17, 24), (8, 896, 7168), (16, 33, 64), (17, 64, 72),
               (33, 100, 136), (63, 129, 520), (65, 7, 4096), (130, 257, 1000), (256, 896, 7168),
               (257, 225, 584), (300, 1024, 264), (520, 449, 88)]


@gpu
@pytest.mark.parametrize("T,E,H", GATE_SHAPES)
def test_gate_logits(m, T, E, H):
    x, w = rand(T, T, H).to(torch.bfloat16), rand(E, E, H, scale=H ** -0.5).to(torch.bfloat16)
    check_gate(m.moe_gate_logits(x.cuda(), w.cuda()), x, w)
    (xw, _), (ow, ob) = window(x), window(torch.zeros(T, E))
    got = m.moe_gate_logits(xw, w.cuda(), out=ow)
    check_gate(got, x, w)
    assert (ob[:, :8] == 77).all() and (ob[:, 8 + E:] == 77).all()
    assert torch.equal(got, m.moe_gate_logits(xw, w.cuda()))     # the same sums every time


@gpu
@pytest.mark.parametrize("T", [3, 40, 300])
def test_gate_logits_nonfinite(m, T):
    """A token's NaN or infinity reaches its own logits only; the rest below a stage of K stays
    out of the sums."""
    H, E = 72, 40
    x, w = rand(1, T, H).to(torch.bfloat16), (1 + rand(2, E, H).abs()).to(torch.bfloat16)
    x[0, H - 1] = NAN
    x[1, 0] = INF
    got = m.moe_gate_logits(x.cuda(), w.cuda()).cpu()
    assert torch.isnan(got[0]).all() and (got[1] == INF).all()
    check_gate(got[2:], x[2:], w)


def route_case(seed, T, E, masked=0.0):
    l = rand(seed, T, E, scale=1.5)
    if masked:
        g = torch.Generator().manual_seed(seed + 1)
        hide = torch.rand(T, E, generator=g) < masked
        half = torch.rand(T, E, generator=g) < 0.5
        l = torch.where(hide, torch.where(half, torch.tensor(float(ref.LOWEST)),
                                          torch.tensor(-INF)), l)
    return l


def check_route(m, l, b, K, G, KG, score, group, renorm, scaling=1.0):
    idx, w = m.moe_route_groups(
        l if l.is_cuda else l.cuda(), None if b is None else b.cuda(), K, n_group=G, topk_group=KG,
        score=m.SCORE_SOFTMAX if score == "softmax" else m.SCORE_SIGMOID,
        group_score=m.GROUP_TOP2 if group == "top2" else m.GROUP_MAX, renormalise=renorm,
        routed_scaling=scaling)
    ri, rw = ref.route(l.cpu().numpy(), None if b is None else b.numpy(), K, G, KG, score, group,
                       renorm, scaling)
    assert np.array_equal(idx.cpu().numpy(), ri)
    got = w.cpu().double().numpy()
    assert np.array_equal(np.isnan(got), np.isnan(rw))
    fine = ~np.isnan(rw)
    # both round a double to float: at most 4 float steps apart (2^-24 each, 2^-149 at the bottom)
    assert (np.abs(got - rw)[fine] <= 4 * 2.0 ** -23 * np.abs(rw)[fine] + 2.0 ** -147).all()
    return idx, w


ROUTE_SHAPES = [  # T, E, K, G, KG
    (1, 1, 1, 1, 1), (3, 4, 2, 1, 1), (1, 896, 16, 8, 4), (20, 896, 16, 8, 4), (9, 896, 16, 1, 1),
    (5, 64, 8, 64, 10), (4, 128, 64, 4, 4), (7, 120, 6, 8, 3), (6, 1024, 64, 16, 2),
    (3, 1056, 16, 4, 3), (2, 4096, 64, 64, 5), (4, 4096, 8, 1, 1), (2, 105, 7, 7, 2),
    (3, 60, 30, 30, 30)]


@gpu
@pytest.mark.parametrize("T,E,K,G,KG", ROUTE_SHAPES)
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("group", ["top2", "max"])
def test_route_groups(m, T, E, K, G, KG, score, group):
    l = route_case(T + E, T, E)
    b = 0.1 * rand(E, E)
    check_route(m, l, b, K, G, KG, score, group, True, 2.5)
    check_route(m, l, None, K, G, KG, score, group, False)


@gpu
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("masked", [0.3, 0.95, 1.0])
def test_route_groups_masks(m, score, masked):
    """Masked experts are never taken; rows with few or none left give -1 and weight 0."""
    for T, E, K, G, KG in ((12, 64, 8, 8, 3), (6, 896, 16, 8, 4), (5, 1536, 16, 4, 2),
                           (9, 16, 8, 1, 1)):
        l = route_case(E, T, E, masked)
        l[0] = -INF
        l[1] = float(ref.LOWEST)
        for group in ("top2", "max"):
            idx, w = check_route(m, l, 0.1 * rand(E, E), K, G, KG, score, group, True)
            assert (idx[:2] == -1).all() and (w[:2] == 0).all()
            check_route(m, l, None, K, G, KG, score, group, False)


@gpu
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_route_groups_ties_and_extremes(m, score):
    T, E, K, G, KG = 10, 256, 12, 8, 3
    l = route_case(5, T, E)
    l[0] = 0.25                              # every key alike
    l[1] = torch.round(l[1])                 # many alike
    l[2, :128] = 100.0                       # scores that saturate
    l[3] = -200.0
    l[3, 7] = -100.0
    l[4, 33] = NAN
    l[5] = NAN
    l[6, 200] = INF
    l[7, 3] = -INF
    l[8] = 1e-30
    for group in ("top2", "max"):
        for b in (None, torch.round(10 * rand(1, E)) / 8):
            check_route(m, l, b, K, G, KG, score, group, True)
            check_route(m, l, b, K, 1, 1, score, group, False)
    b = torch.zeros(E)
    b[:100] = -INF                           # a bias of -inf masks too
    b[101] = NAN
    check_route(m, l, b, K, G, KG, score, "top2", True)
    check_route(m, l, b, K, 1, 1, score, "max", True)


@gpu
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("group", ["top2", "max"])
def test_route_groups_near_worths(m, score, group):
    """Groups of equal worth (the same logits, and biases, in another order) and of worths one
    float step apart: the choice follows the exact float values."""
    T, E, G = 40, 512, 8
    per = E // G
    l, b = route_case(7, T, E), 0.1 * rand(8, E)
    for t in range(T):
        a, c = t % G, (t * 3 + 1) % G
        if a == c:
            continue
        l[t, c * per:(c + 1) * per] = l[t, a * per:(a + 1) * per].flip(0)
        if t % 3 == 1:     # one step up in the best expert of the copy
            e = c * per + int(l[t, c * per:(c + 1) * per].argmax())
            l[t, e] = torch.nextafter(l[t, e], torch.tensor(INF))
    for g in range(1, G):
        b[g * per:(g + 1) * per] = b[:per].flip(0) if g % 2 else b[:per]
    for KG in (1, 3, 4, 7):
        check_route(m, l, b, 16, G, KG, score, group, True)
        check_route(m, l, None, 8, G, KG, score, group, False)


@gpu
def test_route_groups_matches_route(m):
    for T, E, K in ((7, 896, 16), (3, 2000, 16)):
        l, b = route_case(T, T, E).cuda(), 0.1 * rand(E, E).cuda()
        i0, w0 = m.moe_route(l, b, K, 1.5)
        i1, w1 = m.moe_route_groups(l, b, K, routed_scaling=1.5)
        assert torch.equal(i0, i1) and torch.equal(w0, w1)


@gpu
def test_route_groups_strided_logits_and_given_outputs(m):
    l, _ = window(route_case(2, 9, 96))
    check_route(m, l, None, 8, 4, 2, "sigmoid", "top2", True)
    idx = torch.full((9, 8), 5, dtype=torch.int32, device="cuda")
    w = torch.full((9, 8), 5.0, device="cuda")
    a, b = m.moe_route_groups(l, None, 8, n_group=4, topk_group=2, topk_idx=idx, topk_w=w)
    assert a is idx and b is w and (w < 5).all()


@gpu
def test_no_tokens(m):
    e = dict(device="cuda")
    x = torch.empty(0, 64, dtype=torch.bfloat16, **e)
    w = torch.ones(64, dtype=torch.bfloat16, **e)
    h, y, xq, xs = m.moe_add_rmsnorm(x, w, 1e-6, residual=x, q8=m.Q8_MXFP8)
    assert h.shape == y.shape == xq.shape == (0, 64) and xs.shape == (0, 2)
    assert m.moe_quant_int8(x)[0].shape == (0, 64)
    assert m.moe_gate_logits(x, torch.ones(5, 64, dtype=torch.bfloat16, **e)).shape == (0, 5)
    w8, s8 = torch.ones(5, 64, dtype=torch.int8, **e), torch.ones(5, **e)
    assert m.moe_int8_linear(x, w8, s8).shape == (0, 5)
    assert m.moe_int8_matmul(x.to(torch.int8), torch.empty(0, **e), w8, s8).shape == (0, 5)
    assert m.moe_route_groups(torch.empty(0, 16, **e), None, 2)[0].shape == (0, 2)


@gpu
def test_binding_refusals_on_gpu(m):
    x = torch.zeros(4, 64, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    q, s = m.moe_quant_int8(x)
    w8, s8 = q.clone(), s.clone()
    bad = [
        lambda: m.moe_add_rmsnorm(x.float(), w, 1e-6),
        lambda: m.moe_add_rmsnorm(x, w[:32], 1e-6),
        lambda: m.moe_add_rmsnorm(x, w, 1e-6, residual=x[:2]),
        lambda: m.moe_add_rmsnorm(x.t(), w[:4], 1e-6),
        lambda: m.moe_add_rmsnorm(x, w, 1e-6, q8=m.Q8_MXFP8, xq=q),
        lambda: m.moe_add_rmsnorm(x, w, 1e-6, q8=m.Q8_INT8, xq=q, xs=s[:3]),
        lambda: m.moe_quant_int8(x, xq=q[:, :32]),
        lambda: m.moe_int8_matmul(q, s, w8[:, :32], s8),
        lambda: m.moe_int8_matmul(q, s[:2], w8, s8),
        lambda: m.moe_int8_matmul(q, s, w8, s8, out_dtype=torch.float16),
        lambda: m.moe_int8_matmul(q, s, w8, s8, out=x),
        lambda: m.moe_int8_linear(x, w8.float(), s8),
        lambda: m.moe_int8_linear(x, w8, s8, workspace=torch.empty(4, device="cuda")),
        lambda: m.moe_gate_logits(x, x[:, :32]),
        lambda: m.moe_gate_logits(x, x, out=torch.empty(4, 5, device="cuda")),
        lambda: m.moe_route_groups(x, None, 2),
        lambda: m.moe_route_groups(x.float(), s, 2),
    ]
    for call in bad:
        with pytest.raises(ValueError):
            call()
    with pytest.raises(m.MoEError):
        m.moe_int8_linear(x, w8, s8, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    for call in (lambda: m.moe_add_rmsnorm(x, w, 1e-6, q8=7), lambda: m.moe_add_rmsnorm(x, w, -1.0),
                 lambda: m.moe_route_groups(x.float(), None, 2, n_group=3),
                 lambda: m.moe_route_groups(x.float(), None, 2, score=9)):
        with pytest.raises(m.MoEError):
            call()


@gpu
def test_offsets_past_32_bits(m):
    """Operands and outputs of more than 2^32 bytes or elements: the last rows are right."""
    M, K, N = (1 << 18) + 3, 16400, 5
    q, sx, w, sw = int8_case(9, 8, N, K)
    big = torch.zeros(M, K, dtype=torch.int8, device="cuda")
    big[-8:] = q.cuda()
    s = torch.ones(M, device="cuda")
    s[-8:] = sx.cuda()
    out = m.moe_int8_matmul(big, s, w.cuda(), sw.cuda(), out_dtype=torch.float32)
    want = ref.int8_matmul(q.numpy(), sx.numpy(), w.numpy(), sw.numpy())
    assert np.array_equal(out[-8:].cpu().numpy(), want) and (out[:-8] == 0).all()
    del big, out
    T, H = 140000, 32768                                   # 2^32.1 elements
    x = torch.zeros(T, H, dtype=torch.bfloat16, device="cuda")
    tail = rand(3, 4, H).to(torch.bfloat16)
    x[-4:] = tail.cuda()
    wt = torch.ones(H, dtype=torch.bfloat16)
    _, y, xq, xs = m.moe_add_rmsnorm(x, wt.cuda(), 1e-6, q8=m.Q8_MXFP8, y=x)
    _, y64, _ = ref.norm(tail, None, wt, float(np.float32(1e-6)))
    check_y(y[-4:], y64, H)
    check_mxfp8(xq[-4:], xs[-4:], y64, H)
    del x, y, xq
    wide = torch.zeros(3, 1 << 31, device="cuda")          # rows 2^33 bytes apart
    l = route_case(4, 3, 64)
    wide[:, :64] = l.cuda()
    check_route(m, wide[:, :64], None, 4, 4, 2, "sigmoid", "top2", True)


@gpu
def test_one_workspace_for_all_batches(m):
    """One buffer sized for the largest batch, used and left dirty by every smaller one."""
    N, H, most = 896, 1024, 700
    w = rand(1, N, H, scale=H ** -0.5).to(torch.bfloat16).cuda()
    w8, s8 = m.moe_quant_int8(w)
    x = rand(2, most, H).to(torch.bfloat16).cuda()
    wsg = torch.full((m.moe_gate_workspace_size(most, N, H),), 0x7F, dtype=torch.uint8,
                     device="cuda")
    ws8 = torch.full((m.moe_int8_workspace_size(most, N, H),), 0x7F, dtype=torch.uint8,
                     device="cuda")
    q, s = ref.quant_int8(x.float().cpu().numpy())
    for T in (1, 5, 16, 17, 31, 64, 100, 128, 250, 400, most):
        check_gate(m.moe_gate_logits(x[:T], w, workspace=wsg), x[:T], w)
        got = m.moe_int8_linear(x[:T], w8, s8, out_dtype=torch.float32, workspace=ws8)
        want = ref.int8_matmul(q[:T], s[:T], w8.cpu().numpy(), s8.cpu().numpy())
        assert np.array_equal(got.cpu().numpy(), want)


@gpu
def test_streams_and_graph_replays(m):
    """The calls on another stream than the default, and replays of their graph against eager
    results, with other work between the replays."""
    T, H, E, K, N = 24, 512, 128, 8, 320
    x, r = rand(1, T, H).to(torch.bfloat16).cuda(), rand(2, T, H).to(torch.bfloat16).cuda()
    wn = (1 + 0.1 * rand(3, H)).to(torch.bfloat16).cuda()
    wg = rand(4, E, H, scale=H ** -0.5).to(torch.bfloat16).cuda()
    w8, s8 = m.moe_quant_int8(rand(5, N, H, scale=0.05).to(torch.bfloat16).cuda())
    ws8 = torch.empty(m.moe_int8_workspace_size(T, N, H), dtype=torch.uint8, device="cuda")
    wsg = torch.empty(m.moe_gate_workspace_size(T, E, H), dtype=torch.uint8, device="cuda")

    def block(x, bufs):
        h, y, q, s = m.moe_add_rmsnorm(x, wn, 1e-6, residual=r, q8=m.Q8_INT8,
                                       residual_out=bufs["h"], y=bufs["y"], xq=bufs["q"],
                                       xs=bufs["s"])
        l = m.moe_gate_logits(y, wg, out=bufs["l"], workspace=wsg)
        i, w = m.moe_route_groups(l, None, K, n_group=8, topk_group=4, topk_idx=bufs["i"],
                                  topk_w=bufs["w"])
        z = m.moe_int8_matmul(q, s, w8, s8, out=bufs["z"], workspace=ws8)
        return h, y, l, i, w, z, m.moe_int8_linear(y, w8, s8, out=bufs["z2"], workspace=ws8)

    def buffers():
        e = dict(device="cuda")
        return dict(h=torch.empty(T, H, dtype=torch.bfloat16, **e),
                    y=torch.empty(T, H, dtype=torch.bfloat16, **e),
                    q=torch.empty(T, H, dtype=torch.int8, **e), s=torch.empty(T, **e),
                    l=torch.empty(T, E, **e), i=torch.empty(T, K, dtype=torch.int32, **e),
                    w=torch.empty(T, K, **e), z=torch.empty(T, N, dtype=torch.bfloat16, **e),
                    z2=torch.empty(T, N, dtype=torch.bfloat16, **e))

    eager = [t.clone() for t in block(x, buffers())]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = block(x, buffers())
    side.synchronize()
    for a, b in zip(eager, other):
        assert torch.equal(a, b)
    held, xin = buffers(), x.clone()
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            outs = block(xin, held)
    torch.cuda.synchronize()
    for rep in range(4):
        xin.copy_(x if rep % 2 == 0 else x.flip(0))
        for t in outs:
            t.fill_(3)
        graph.replay()
        torch.cuda.synchronize()
        want = eager if rep % 2 == 0 else [t.clone() for t in block(xin, buffers())]
        for a, b in zip(want, outs):
            assert torch.equal(a, b)
