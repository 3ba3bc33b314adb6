"""Workspaces of the 8-bit integer products."""
import os

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "mxfp8_mxfp4_experts_amd", "libmi355moe.so")
pytestmark = pytest.mark.skipif(not os.path.exists(LIB), reason="libmi355moe.so not built")

FAKE = 1 << 20          # aligned, never dereferenced by a failing call
NULL, WORKSPACE = 1, 5


@pytest.fixture(scope="module")
def lib():
    from mxfp8_mxfp4_experts_amd import _binding
    return _binding.load_library(LIB)


@pytest.fixture(scope="module")
def m():
    import mxfp8_mxfp4_experts_amd as mod
    return mod


# ---------------------------------------------------------------------------
# Workspaces.

def test_matmul_workspace_is_the_partial_sums(lib):
    """No room for 8-bit tokens, which the product is given: at most 16 MB, and not more for a
    longer K."""
    size = lib.moe_int8_matmul_workspace_size
    for M, N, K in ((1, 1, 16), (17, 3584, 7168), (8192, 3584, 7168), (4194303, 5, 131056)):
        assert 0 < size(M, N, K) <= 1 << 24
        assert size(M, N, K) == size(M, N, 16) <= lib.moe_int8_workspace_size(M, N, K) - M * K
    assert size(0, 7, 64) == size(-1, 7, 64) == size(4, 0, 64) == size(4, 7, 24) == 0
    for N in (1, 130, 3584):
        sizes = [size(M, N, 1024) for M in range(0, 3000, 7)]
        assert sizes == sorted(sizes)


def test_matmul_refuses_a_small_workspace(lib):
    for M, N, K in ((1, 7, 64), (64, 3584, 7168), (8192, 3584, 7168)):
        need = lib.moe_int8_matmul_workspace_size(M, N, K)

        def call(ws, nb):
            return lib.moe_int8_matmul(FAKE, K, FAKE, FAKE, FAKE, M, N, K, 0, FAKE, N, ws, nb, None)
        assert call(FAKE, need - 1) == WORKSPACE and call(None, need) == NULL


@pytest.mark.gpu
def test_matmul_takes_no_room_for_tokens(m):
    """A call without a workspace allocates its output and the partial sums, not a copy of the
    tokens (59 MB here)."""
    M, N, K = 8192, 64, 7168
    q = torch.ones(M, K, dtype=torch.int8, device="cuda")
    w = torch.ones(N, K, dtype=torch.int8, device="cuda")
    s, sw = torch.ones(M, device="cuda"), torch.ones(N, device="cuda")
    torch.cuda.synchronize()
    torch.cuda.reset_peak_memory_stats()
    before = torch.cuda.memory_allocated()
    out = m.moe_int8_matmul(q, s, w, sw, out_dtype=torch.float32)
    assert (out == K).all()
    # plus what the comparison takes: a truth value for each output
    most = out.numel() * 5 + m.moe_int8_matmul_workspace_size(M, N, K) + (1 << 20)
    assert torch.cuda.max_memory_allocated() - before <= most < M * K
