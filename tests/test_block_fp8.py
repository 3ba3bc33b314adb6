"""MoEBlock with E4M3 weights into the experts' width and back: its calls in order, the buffers
it keeps, its refusals."""
import os

import numpy as np
import pytest
import torch

import block_ref
import fp8_ref as ref
import oracle
from test_block import bits, make, rand
from test_block_buffers import MOST, Calls, cpu_layer

from mxfp8_mxfp4_experts_amd import _binding as B
from mxfp8_mxfp4_experts_amd.block import MoEBlock

pytestmark = pytest.mark.skipif(not os.path.exists(B._LIB_PATH), reason="libmi355moe.so not built")
gpu = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module")
def m():
    import mxfp8_mxfp4_experts_amd as mod
    return mod


def pairs(H, L, dtype=ref.FP8):
    """Empty weights into the width L and back."""
    pair = lambda n, k: (torch.empty(n, k, dtype=torch.uint8).view(dtype),  # noqa: E731
                         torch.empty(ref.blocks(n), ref.blocks(k)))
    return dict(down=pair(L, H), up=pair(H, L))


def cpu_block(H, L, **kw):
    return MoEBlock(cpu_layer(L, 256, 64, 4, MOST), torch.empty(H, dtype=torch.bfloat16),
                    torch.empty(64, H, dtype=torch.bfloat16), max_tokens=MOST, **kw)


def test_buffers_stay(monkeypatch):
    """Each batch up to max_tokens is given the same memory, and enough of it."""
    calls = Calls(monkeypatch)
    monkeypatch.setattr(B, "moe_fp8_linear", calls.noting(
        "moe_fp8_linear", lambda a, k: torch.empty(1) if k["out"] is None else k["out"]))
    H, L = 2048, 512
    block = cpu_block(H, L, **pairs(H, L))
    first = calls.of(block, 1)
    assert [n for n, _ in first].count("moe_fp8_linear") == 2
    for T in (64, 5, MOST, 17, 256):
        assert calls.of(block, T) == first, T
        for shape in ((T, H, L), (T, L, H)):
            assert calls.sizes["moe_fp8_linear"] >= B.moe_fp8_workspace_size(*shape)


def test_refusals():
    H, L = 768, 512
    good = pairs(H, L)
    cpu_block(H, L, **good)
    cpu_block(H, L, **pairs(H, L, torch.uint8))
    int8 = torch.empty(H, L, dtype=torch.int8), torch.empty(H)
    for bad in (dict(good, up=int8), dict(good, down=good["up"]), dict(down=good["down"]),
                dict(good, down=(good["down"][0], torch.empty(L))),
                dict(good, up=(torch.empty(H, L), good["up"][1]))):
        with pytest.raises(ValueError):
            cpu_block(H, L, **bad)


@pytest.mark.parametrize("N,K", [(512, 768), (130, 272), (1, 16)])
def test_quantise_fp8(N, K):
    """Every code is within half a step of its value, every block's largest one is 448."""
    w = rand(N, N, K).to(torch.bfloat16)
    w[0] *= 1e-3
    q, s = MoEBlock.quantise_fp8(w)
    assert q.shape == (N, K) and s.shape == (ref.blocks(N), ref.blocks(K))
    up = lambda t: t.repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)[:, :K].double()  # noqa
    got = q.double() * up(s)
    # Half a step, 2^-4, and the float division's; below 2^-6 steps of 2^-9.
    assert ((got - w.double()).abs() <= 2.0 ** -4 * (1 + 2.0 ** -10) * w.double().abs() +
            2.0 ** -10 * up(s)).all()
    assert q.float().abs().max() == 448
    zero, zs = MoEBlock.quantise_fp8(torch.zeros(N, K, dtype=torch.bfloat16))
    assert (zero.float() == 0).all() and (zs == 2.0 ** -126).all()


def fp8_block(m, T, H, L, seed=1, **kw):
    pair = lambda s, n, k: MoEBlock.quantise_fp8(  # noqa: E731
        rand(s, n, k, scale=k ** -0.5).to(torch.bfloat16).to(DEV))
    block, x, r, w = make(m, T=T, H=H, L=L, I=256, E=32, K=4, seed=seed, n_group=8, topk_group=4)
    fp8 = MoEBlock(block.experts, block.norm_w, block.gate_w, gate_bias=block.gate_bias, n_group=8,
                   topk_group=4, max_tokens=T, down=pair(seed + 3, L, H), up=pair(seed + 4, H, L),
                   **kw)
    return fp8, x, r, w


@gpu
@pytest.mark.parametrize("T,H,L", [(1, 768, 512), (7, 768, 512), (33, 512, 512), (200, 1024, 256)])
@pytest.mark.parametrize("with_residual", [True, False])
def test_block(m, T, H, L, with_residual):
    block, x, r, w = fp8_block(m, T, H, L)
    r = r if with_residual else None
    out, h = block(x, r)
    h2, y, _, _ = m.moe_add_rmsnorm(x, block.norm_w, 1e-6, residual=r)
    assert torch.equal(h, h2) if with_residual else h is x
    logits = m.moe_gate_logits(y, block.gate_w)
    idx, wt = m.moe_route_groups(logits, block.gate_bias, 4, n_group=8, topk_group=4,
                                 routed_scaling=1.5)
    z = m.moe_fp8_linear(y, *block.down)
    ref.check(z, *ref.product(*(t.to(DEV) for t in ref.quant(y)), *block.down))
    lay = block.experts(z, None, None, topk_idx=idx, topk_w=wt)
    assert torch.equal(out, m.moe_fp8_linear(lay, *block.up))
    # Against the experts' oracle and the way up in 64 bits, without the rounding of its input to
    # E4M3 (half a step at most, 2^-4 of a value and about 2% of the rms; with the experts' own
    # requantisation, below 4%, the cosine stays above 0.998).
    w_np = {k: v.cpu().numpy() for k, v in w.items()}
    o = oracle.oracle_layer(bits(z), None, None, w_np["w13"], w_np["w13_s"], w_np["w2"],
                            w_np["w2_s"], top_k=4, topk_idx=idx.cpu().numpy(),
                            topk_w=wt.cpu().numpy())["out"]
    up, s = (t.cpu().double() for t in block.up)
    up = up * s.repeat_interleave(128, 0)[:H].repeat_interleave(128, 1)[:, :L]
    o, got = o @ up.numpy().T, block_ref.f64(out)
    cos = (got * o).sum() / (np.linalg.norm(got) * np.linalg.norm(o))
    assert cos >= 0.998 and np.isfinite(got).all()


@gpu
@pytest.mark.parametrize("T", [1, 24])
def test_graph_beside_other_batches(m, T):
    """A captured block, replayed with other tokens after smaller and larger batches."""
    block, x, r, _ = fp8_block(m, 40, 768, 512)
    a, b = x[:T].clone(), r[:T].clone()
    out, h = torch.empty_like(a), torch.empty_like(a)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        block(a, b, out=out, residual_out=h)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        block(a, b, out=out, residual_out=h)
    for i in range(3):
        a.copy_(x[i:i + T])
        b.copy_(r[i:i + T])
        want, want_h = block(a, b)
        block(x, r)
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(h, want_h)
