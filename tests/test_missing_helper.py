"""Without the compiled helper of the argument checks: the grouping needs none, the calls that do
name it."""
import os
import sys

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "mxfp8_mxfp4_experts_amd", "libmi355moe.so")
pytestmark = pytest.mark.skipif(not os.path.exists(LIB), reason="libmi355moe.so not built")


@pytest.fixture
def m(monkeypatch):
    """The binding as it is loaded where _tensor_args.so is not."""
    import mxfp8_mxfp4_experts_amd as mod
    from mxfp8_mxfp4_experts_amd import _binding as B

    def missing(*args):
        return B._load_args()
    monkeypatch.setitem(sys.modules, "mxfp8_mxfp4_experts_amd._tensor_args", None)
    monkeypatch.delattr(mod, "_tensor_args", raising=False)
    monkeypatch.setattr(B, "_call", B._Calls())
    monkeypatch.setattr(B, "_head", missing)
    monkeypatch.setattr(B, "_plain", missing)
    return mod


def ints(dev, *shape):
    return torch.zeros(*shape, dtype=torch.int32, device=dev)


def permute(m, dev, T=5, k=2, E=3):
    idx = (torch.arange(T * k, device=dev) % E).int().view(T, k)
    ws = torch.empty(m.moe_workspace_size(T, k, E, 128, 128), dtype=torch.uint8, device=dev)
    return m.moe_permute(idx, 0, E, ws, ints(dev, E + 1), ints(dev, T * k), ints(dev, T * k))


def test_grouping_checks_its_arguments_itself(m):
    for _ in range(2):
        with pytest.raises(ValueError, match="topk_idx"):
            permute(m, "cpu")


def test_other_calls_name_the_helper(m):
    bf = torch.zeros(2, 128, dtype=torch.bfloat16)
    calls = [lambda: m.moe_quant_fp8(bf, torch.zeros(2, 128, dtype=torch.uint8), torch.zeros(1, 2)),
             lambda: m.moe_quant_fp8(bf), lambda: m.moe_sort_tokens(bf, ints("cpu", 2), 1)]
    for call in calls:
        with pytest.raises(ImportError, match="_tensor_args.so"):
            call()


@pytest.mark.gpu
def test_grouping(m):
    offs, sorted_route, row = permute(m, "cuda")
    assert offs.tolist() == [0, 4, 7, 10]
    assert sorted_route.tolist() == [0, 3, 6, 9, 1, 4, 7, 2, 5, 8]
    assert row.tolist() == [0, 4, 7, 1, 5, 8, 2, 6, 9, 3]
