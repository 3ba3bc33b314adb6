"""MoEBlock's buffers: one address for every batch up to max_tokens, so a
captured graph stays valid whatever batches run after it."""
import os

import pytest
import torch

from mxfp8_mxfp4_experts_amd import _binding as B
from mxfp8_mxfp4_experts_amd.block import MoEBlock
from mxfp8_mxfp4_experts_amd.layer import MoELayer

pytestmark = pytest.mark.skipif(not os.path.exists(B._LIB_PATH), reason="libmi355moe.so not built")
MOST = 512


class Calls:
    """The library's calls replaced by ones that note which memory they were given."""

    def __init__(self, monkeypatch):
        self.seen = []
        for name, out in (("moe_add_rmsnorm", lambda a, k: (None, k["y"], k["xq"], k["xs"])),
                          ("moe_gate_logits", lambda a, k: k["out"]),
                          ("moe_route_groups", lambda a, k: (k["topk_idx"], k["topk_w"])),
                          ("moe_int8_matmul", lambda a, k: k["out"]),
                          ("moe_int8_linear", lambda a, k: torch.empty(1)),
                          ("moe_quant_permute", lambda a, k: None),
                          ("moe_permute", lambda a, k: None),
                          ("moe_fc1_situ", lambda a, k: None),
                          ("moe_fc2_combine",
                           lambda a, k: torch.empty(1) if a[11] is None else a[11])):
            monkeypatch.setattr(B, name, self.noting(name, out))

    def noting(self, name, out):
        def call(*a, **k):
            # Every buffer that the block and its layer keep: all tensors but the given x.
            kept = [t for t in (*a, *k.values()) if isinstance(t, torch.Tensor) and t is not self.x]
            self.seen.append((name, tuple(t.data_ptr() for t in kept)))
            if "workspace" in k:
                self.sizes[name] = k["workspace"].numel()
            return out(a, k)
        return call

    def of(self, block, T):
        self.seen, self.sizes = [], {}
        self.x = torch.empty(T, block.H, dtype=torch.bfloat16)
        block(self.x)
        return self.seen


def cpu_layer(H, I, E, K, max_tokens):
    """A MoELayer on the CPU: its buffers, without weights."""
    layer = object.__new__(MoELayer)
    layer.E_local, layer.E, layer.H, layer.I, layer.top_k = E, E, H, I, K
    layer.expert_offset, layer.routed_scaling, layer.alpha, layer.beta = 0, 1.0, 4.0, 25.0
    layer.tiled, layer.combine_mode = False, B.COMBINE_DETERMINISTIC
    layer.w13 = layer.w13_s = layer.w2 = layer.w2_s = None
    layer.device = torch.device("cpu")
    layer._alloc(max_tokens)
    return layer


def cpu_block(H, L, E=64, K=4, max_tokens=MOST, layer_tokens=MOST):
    pair = lambda n, k: (torch.empty(n, k, dtype=torch.int8), torch.empty(n))  # noqa: E731
    kw = dict(down=pair(L, H), up=pair(H, L)) if L != H else {}
    return MoEBlock(cpu_layer(L, 256, E, K, layer_tokens), torch.empty(H, dtype=torch.bfloat16),
                    torch.empty(E, H, dtype=torch.bfloat16), max_tokens=max_tokens, **kw)


@pytest.mark.parametrize("H,L", [(1024, 1024), (2048, 512)])
@pytest.mark.parametrize("layer_tokens", [MOST, 1])
def test_buffers_stay_for_every_batch_up_to_max_tokens(monkeypatch, H, L, layer_tokens):
    """Whatever the order of batches, each call is given the same memory, and enough of it."""
    calls = Calls(monkeypatch)
    block = cpu_block(H, L, layer_tokens=layer_tokens)
    first = calls.of(block, 1)
    assert len(first) >= 5
    for T in (64, 5, MOST, 17, 256):
        assert calls.of(block, T) == first, T
        assert calls.sizes["moe_gate_logits"] >= B.moe_gate_workspace_size(T, block.E, H)
        if L != H:
            assert calls.sizes["moe_int8_linear"] >= B.moe_int8_workspace_size(T, H, L)


def test_a_smaller_layer_keeps_its_buffers(monkeypatch):
    """A layer for fewer tokens than the block's is left as it is: graphs of its own stay valid."""
    calls = Calls(monkeypatch)
    layer = cpu_layer(512, 256, 64, 4, 8)
    before = {k: v.data_ptr() for k, v in vars(layer).items() if isinstance(v, torch.Tensor)}
    block = MoEBlock(layer, torch.empty(512, dtype=torch.bfloat16),
                     torch.empty(64, 512, dtype=torch.bfloat16), max_tokens=64)
    calls.of(block, 64)
    calls.of(block, 200)                                   # past max_tokens: the block's grow
    assert block.max_tokens == 200
    after = {k: v.data_ptr() for k, v in vars(layer).items() if isinstance(v, torch.Tensor)}
    assert after == before and layer.max_tokens == 8


@pytest.mark.gpu
@pytest.mark.parametrize("H,L", [(512, 512), (4096, 512)])
@pytest.mark.parametrize("layer_tokens", [MOST, 1])
def test_graph_of_a_block_beside_larger_batches(H, L, layer_tokens):
    """A block captured at 64 tokens, larger batches run eagerly between the replays: every replay
    gives the eager result, and memory taken meanwhile keeps its contents."""
    import synth
    T, E, K = 64, 64, 4
    dev = "cuda:0"
    cfg = synth.custom_config("block_graph", 811, T=T, H=L, I=256, E=E, K=K)
    w = {k: v.to(dev) for k, v in synth.make_expert_weights(cfg, device="cpu").items()}
    layer = MoELayer(w["w13"], w["w13_s"], w["w2"], w["w2_s"], top_k=K, E=E,
                     max_tokens=layer_tokens)
    g = torch.Generator().manual_seed(5)

    def rand(*shape, scale=1.0):
        return (scale * torch.randn(*shape, generator=g)).to(torch.bfloat16).to(dev)

    kw = {}
    if L != H:
        kw = dict(down=MoEBlock.quantise(rand(L, H, scale=H ** -0.5)),
                  up=MoEBlock.quantise(rand(H, L, scale=L ** -0.5)))
    block = MoEBlock(layer, 1 + 0.1 * rand(H), rand(E, H, scale=H ** -0.5), n_group=8,
                     topk_group=4, max_tokens=MOST, **kw)
    x, r, big, more = rand(T, H), rand(T, H), rand(MOST, H), rand(MOST, H)
    out, h = (torch.empty(T, H, dtype=torch.bfloat16, device=dev) for _ in range(2))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        block(x, r, out=out, residual_out=h)
        want = out.clone(), h.clone()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            block(x, r, out=out, residual_out=h)
    torch.cuda.synchronize()
    taken = []
    for rep in range(4):
        eager = block(big, more)[0].clone()                # a batch of max_tokens
        taken += [torch.full((n,), 77, dtype=torch.uint8, device=dev)
                  for n in (1 << 16, 1 << 18, 1 << 20, 1 << 22)]
        out.fill_(3)
        h.fill_(3)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[0]) and torch.equal(h, want[1]), rep
        assert all((t == 77).all() for t in taken), rep
        assert torch.equal(block(big, more)[0], eager), rep
