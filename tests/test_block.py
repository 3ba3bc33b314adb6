"""MoEBlock: its calls in order, against the same calls one by one and against
the oracle of the expert layer."""
import numpy as np
import pytest
import torch

import block_ref as ref
import oracle
import synth

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


@pytest.fixture(scope="module")
def m():
    import mxfp8_mxfp4_experts_amd as mod
    return mod


def bits(t):
    return t.detach().cpu().contiguous().view(torch.int16).numpy().view(np.uint16)


def rand(seed, *shape, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return scale * torch.randn(*shape, generator=g)


def make(m, T, H, L, I, E, K, seed=1, **kw):
    cfg = synth.custom_config("block", 700 + T, T=T, H=L, I=I, E=E, K=K)
    w = {k: v.to(DEV) for k, v in synth.make_expert_weights(cfg, device="cpu").items()}
    layer = m.MoELayer(w["w13"], w["w13_s"], w["w2"], w["w2_s"], top_k=K, E=E, max_tokens=T,
                       routed_scaling=1.5)
    norm_w = (1 + 0.1 * rand(seed, H)).to(torch.bfloat16).to(DEV)
    gate_w = rand(seed + 1, E, H, scale=H ** -0.5).to(torch.bfloat16).to(DEV)
    bias = 0.1 * rand(seed + 2, E).to(DEV)
    if L != H:
        kw["down"] = m.MoEBlock.quantise(
            rand(seed + 3, L, H, scale=H ** -0.5).to(torch.bfloat16).to(DEV))
        kw["up"] = m.MoEBlock.quantise(
            rand(seed + 4, H, L, scale=L ** -0.5).to(torch.bfloat16).to(DEV))
    block = m.MoEBlock(layer, norm_w, gate_w, gate_bias=bias, max_tokens=T, **kw)
    x = rand(seed + 5, T, H).to(torch.bfloat16).to(DEV)
    r = rand(seed + 6, T, H, scale=2.0).to(torch.bfloat16).to(DEV)
    return block, x, r, w


CASES = [dict(T=1, H=512, L=512, I=256, E=32, K=4), dict(T=33, H=512, L=512, I=256, E=32, K=4),
         dict(T=7, H=768, L=512, I=256, E=32, K=4), dict(T=200, H=1024, L=256, I=128, E=16, K=2)]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "T{T}_H{H}_L{L}".format(**c))
@pytest.mark.parametrize("with_residual", [True, False])
def test_block(m, case, with_residual):
    kw = dict(n_group=8, topk_group=4, score=m.SCORE_SIGMOID)
    block, x, r, w = make(m, **case, **kw)
    T, H, L, K = case["T"], case["H"], case["L"], case["K"]
    r = r if with_residual else None
    out, h = block(x, r)
    # call by call
    q8 = m.Q8_MXFP8 if L == H else m.Q8_INT8
    h2, y, xq, xs = m.moe_add_rmsnorm(x, block.norm_w, 1e-6, residual=r, q8=q8)
    if with_residual:
        assert torch.equal(h, h2)
    else:
        assert h is x and h2 is None
    logits = m.moe_gate_logits(y, block.gate_w)
    assert torch.equal(logits, block.logits[:T])
    idx, wt = m.moe_route_groups(logits, block.gate_bias, K, n_group=8, topk_group=4,
                                 routed_scaling=1.5)
    assert torch.equal(idx, block.topk_idx[:T]) and torch.equal(wt, block.topk_w[:T])
    z = y if L == H else m.moe_int8_matmul(xq, xs, *block.down)
    w_np = {k: v.cpu().numpy() for k, v in w.items()}
    o = oracle.oracle_layer(bits(z), None, None, w_np["w13"], w_np["w13_s"], w_np["w2"],
                            w_np["w2_s"], top_k=K, topk_idx=idx.cpu().numpy(),
                            topk_w=wt.cpu().numpy())["out"]
    if L != H:
        lay = block.experts(z, None, None, topk_idx=idx, topk_w=wt)
        assert torch.equal(out, m.moe_int8_linear(lay, *block.up))
        up = block.up[0].cpu().double().numpy() * block.up[1].cpu().double().numpy()[:, None]
        o = o @ up.T
    # The experts' requantisation may round next to the oracle's in both forms, the MXFP8 of the
    # float y and of its bf16 copy too, and the way up rounds the layer's output to 8 bits (each
    # below 2^-8 of a row's largest value, so about 1% of its rms): the cosine of such an error of
    # up to 4% stays above 0.999.
    got = ref.f64(out)
    cos = (got * o).sum() / (np.linalg.norm(got) * np.linalg.norm(o))
    assert cos >= 0.999 and np.isfinite(got).all()


def test_block_grows_and_shrinks(m):
    """Batches above max_tokens enlarge the buffers; smaller ones afterwards give what they gave."""
    block, x, r, _ = make(m, T=40, H=768, L=512, I=256, E=32, K=4, n_group=4, topk_group=2)
    one, h1 = block(x[:1], r[:1])
    one, h1 = one.clone(), h1.clone()
    big = torch.cat([x] * 8), torch.cat([r] * 8)
    out, h = block(*big)
    assert out.shape == (320, 768) and torch.equal(h[:40], h[40:80])
    again, h2 = block(x[:1], r[:1])
    assert torch.equal(again, one) and torch.equal(h2, h1)


def test_block_chain_in_place(m):
    """Two blocks: the first one's output is the second one's x, the residual stream is updated
    in place."""
    a, x, r, _ = make(m, T=9, H=512, L=512, I=256, E=32, K=4, n_group=4, topk_group=2)
    b, _, _, _ = make(m, T=9, H=512, L=512, I=256, E=32, K=4, seed=40, score=m.SCORE_SOFTMAX)
    o1, h1 = a(x, r)
    o2, h2 = b(o1, h1)
    stream = r.clone()
    p1, s1 = a(x, stream, residual_out=stream)
    p2, s2 = b(p1, s1, residual_out=stream)
    assert s2.data_ptr() == stream.data_ptr()
    assert torch.equal(p2, o2) and torch.equal(stream, h2)


def test_block_refusals(m):
    block, x, r, _ = make(m, T=4, H=512, L=512, I=256, E=32, K=4)
    e, nw, gw = block.experts, block.norm_w, block.gate_w
    q = m.MoEBlock.quantise(torch.zeros(512, 768, dtype=torch.bfloat16, device=DEV))
    for call in (lambda: m.MoEBlock(e, nw[:256], gw), lambda: m.MoEBlock(e, nw, gw[:8]),
                 lambda: m.MoEBlock(e, nw, gw, down=q), lambda: m.MoEBlock(e, nw, gw, down=q, up=q),
                 lambda: block(x[:, :256], r), lambda: block(x, r[:2]),
                 lambda: e.mxfp8(block.xq, block.xs, block.topk_idx[:2], block.topk_w)):
        with pytest.raises(ValueError):
            call()
