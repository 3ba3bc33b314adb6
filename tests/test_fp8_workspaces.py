"""The workspaces of the block-scaled FP8 products: none where no product is split."""
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
NONE = [(1, 3584, 7168), (8, 3584, 7168), (9, 512, 640), (256, 3584, 640), (4096, 896, 16), (8, 1, 16)]


def test_sizes():
    import mxfp8_mxfp4_experts_amd as m
    for M, N, K in NONE:
        assert m.moe_fp8_matmul_workspace_size(M, N, K) == 0
        KB, q = ref.blocks(K), (M * 128 * ref.blocks(K) + 255) // 256 * 256
        assert q + 4 * KB * M <= m.moe_fp8_workspace_size(M, N, K) <= q + 4 * KB * (M + 3) + 257
    for M, N, K in ((9, 3584, 656), (256, 3584, 7168), (4096, 896, 1040)):
        assert m.moe_fp8_matmul_workspace_size(M, N, K) > 0
    for N, K in ((3584, 7168), (64, 640), (100, 656)):
        sizes = [m.moe_fp8_matmul_workspace_size(M, N, K) for M in range(0, 600)]
        assert sizes == sorted(sizes)


def test_every_split_has_its_workspace():
    """Whatever is picked, the partial sums fit in what the size names."""
    import mxfp8_mxfp4_experts_amd as m
    probe = ctypes.CDLL(PROBE)
    out = (ctypes.c_int32 * 6)()
    for M in (1, 8, 9, 16, 31, 64, 130, 256, 500, 900, 2000, 4400):
        for N in (1, 65, 152, 448, 896, 3584):
            for K in (16, 640, 656, 768, 1040, 2064, 7168, 10640):
                probe.probe_fp8_pick(M, N, K, out)
                if out[1] > 1:
                    need = 4 * out[1] * M * ((N + 3) // 4 * 4)
                    assert need <= m.moe_fp8_matmul_workspace_size(M, N, K), (M, N, K)


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K", [(1, 300, 7168), (8, 130, 1040), (9, 130, 640), (300, 260, 400)])
def test_products_without_a_workspace(M, N, K):
    import mxfp8_mxfp4_experts_amd as m
    q, xs = (t.cuda() for t in ref.quant(ref.tokens(M, K, 1)))
    w, w_s = (t.cuda() for t in ref.weight(N, K, 2))
    out = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    none = torch.empty(0, dtype=torch.uint8, device="cuda")
    assert m.moe_fp8_matmul(q, xs, w, w_s, out=out, workspace=none) is out
    ref.check(out, *ref.product(q, xs, w, w_s))
