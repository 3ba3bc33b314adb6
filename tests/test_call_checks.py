"""The compiled check-and-call of the calls beside the experts: what it takes gives what the step by
step checks give, what it does not take is refused as by them, with every buffer given."""
import os

import pytest
import torch

import fp8_ref as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "mxfp8_mxfp4_experts_amd", "libmi355moe.so")
pytestmark = pytest.mark.skipif(not os.path.exists(LIB), reason="libmi355moe.so not built")
gpu = pytest.mark.gpu
DEV = "cuda"
NAMES = ("quant_fp8", "fp8_matmul", "fp8_linear", "fp8_grouped", "sort_tokens", "unsort_tokens",
         "unsort_tokens_grad", "permute")


@pytest.fixture(scope="module")
def m():
    import mxfp8_mxfp4_experts_amd as m
    return m


def test_answers_without_throwing():
    """None for whatever is no plain tensor of the current GPU; the C function is never reached
    (its address here is no function's)."""
    from mxfp8_mxfp4_experts_amd import _tensor_args as ck
    counts = dict(quant_fp8=3, fp8_matmul=6, fp8_linear=5, fp8_grouped=8, sort_tokens=4,
                  unsort_tokens=5, unsort_tokens_grad=6, permute=7)
    bf = torch.bfloat16
    for name in NAMES:
        f = getattr(ck, name)
        for t in (torch.zeros(2, 4, dtype=bf), torch.zeros(2, 4, dtype=bf).to_sparse(), None, 3,
                  torch.zeros(()), torch.zeros(2, 4, dtype=bf, device="meta"), [1.0]):
            assert f(1, None, *[t] * counts[name]) is None, (name, type(t))
        with pytest.raises(TypeError):
            f(1, None)


def buffers(m, seed=0, M=6, N=130, K=272, E=3, k=2):
    """Every call's arguments by name, with every buffer given; M tokens, k routes each."""
    g = torch.Generator().manual_seed(seed)
    NB, KB, R = ref.blocks(N), ref.blocks(K), M * k
    x = ref.tokens(M, K, seed).to(DEV)
    w, w_s = (t.to(DEV) for t in ref.weight(N, K, seed + 1, E))
    idx = torch.rand(M, E, generator=g).argsort(1)[:, :k].int().to(DEV)
    ws = torch.empty(m.moe_workspace_size(M, k, E, 128, 128), dtype=torch.uint8, device=DEV)
    offs, sorted_route, route_row = m.moe_permute(idx, 0, E, ws)
    xq, xs = m.moe_quant_fp8(x)
    bf = dict(dtype=torch.bfloat16, device=DEV)
    ints = lambda *n: torch.zeros(*n, dtype=torch.int32, device=DEV)  # noqa: E731
    wk = torch.empty(m.moe_fp8_workspace_size(M, N, K), dtype=torch.uint8, device=DEV)
    tw = torch.rand(M, k, generator=g).to(DEV)
    rows = torch.randn(R, K, generator=g).to(**bf)
    return dict(
        quant_fp8=dict(x=x, xq=torch.zeros_like(xq), xs=torch.zeros_like(xs)),
        fp8_matmul=dict(xq=xq, xs=xs, w=w[0], w_s=w_s[0], out=torch.zeros(M, N, **bf),
                        workspace=wk),
        fp8_linear=dict(x=x, w=w[1], w_s=w_s[1], out=torch.zeros(M, N, **bf), workspace=wk),
        fp8_grouped=dict(xq=xq, xs=xs, w=w, w_s=w_s, expert_offsets=offs,
                         sorted_route=sorted_route, top_k=k, out=torch.zeros(R, N, **bf)),
        sort_tokens=dict(x=x, route_row=route_row, top_k=k, rows=torch.zeros(R, K, **bf)),
        unsort_tokens=dict(rows=rows, route_row=route_row, topk_w=tw, top_k=k,
                           out=torch.zeros(M, K, **bf)),
        unsort_tokens_grad=dict(dout=x, rows=rows, route_row=route_row, topk_w=tw,
                                drows=torch.zeros(R, K, **bf), dw=torch.zeros(M, k, device=DEV)),
        permute=dict(topk_idx=idx, expert_offset=0, E_local=E, workspace=ws,
                     expert_offsets=ints(E + 1), sorted_route=ints(R), route_row=ints(R)))


def result(r):
    return [t.clone() for t in (r if isinstance(r, tuple) else (r,))]


@gpu
@pytest.mark.parametrize("name", NAMES)
def test_same_results_as_step_by_step(m, name, monkeypatch):
    """Whole tensors, windows of wider ones, FP8 and byte codes, routes in two dimensions: the
    helper takes them and gives what the step by step checks give without it."""
    from mxfp8_mxfp4_experts_amd import _binding as B

    class Off:
        def __getattr__(self, _):
            return lambda *a: None

    took = []
    real = getattr(B._call, name)
    for wide in (False, True):
        kw = buffers(m)[name]
        if wide:
            for key, t in kw.items():
                if key in ("x", "xq", "xs", "out", "rows", "dout", "drows") and t.dim() == 2 and not (
                        name == "quant_fp8" and key == "xq"):
                    big = torch.zeros(t.shape[0], t.shape[1] + 32, dtype=t.dtype, device=DEV)
                    big[:, 16:16 + t.shape[1]] = t
                    kw[key] = big[:, 16:16 + t.shape[1]]
                elif key == "route_row" and "top_k" in kw:
                    kw[key] = t.view(-1, kw["top_k"])
                elif key == "w":
                    kw[key] = t.view(torch.uint8)
            if "sorted_route" in kw and name == "fp8_grouped":
                kw["sorted_route"] = None
                kw["out"] = kw["out"][:kw["xq"].shape[0]]
        with monkeypatch.context() as mp:
            mp.setattr(B._call, name, lambda *a: took.append(real(*a)) or took[-1], raising=False)
            got = result(getattr(m, "moe_" + name)(**kw))
        with monkeypatch.context() as mp:
            mp.setattr(B, "_call", Off())
            want = result(getattr(m, "moe_" + name)(**kw))
        assert all(torch.equal(a, b) for a, b in zip(got, want)) and len(got) == len(want)
    assert took == [0, 0]


def wrong(t):
    """Tensors that are not what `t` is: type, shape, place, layout."""
    yield t.to(torch.float64)
    yield t[:-1] if t.shape[0] > 1 else torch.cat([t, t])
    yield t.cpu()
    yield t.unsqueeze(-1).unsqueeze(-1)
    if t.dim() == 1:
        yield torch.stack([t, t], 1)[:, 0]           # strided
    else:
        yield t.transpose(-1, -2)
        yield torch.stack([t, t], t.dim())[..., 0]   # columns apart
    yield None
    yield 7


@gpu
@pytest.mark.parametrize("name", NAMES)
def test_refusals(m, name):
    """Each tensor of each call replaced in turn: an error before anything is launched, whether a
    missing buffer is made by the call or not."""
    may_be_none = dict(quant_fp8=("xq", "xs"), fp8_matmul=("out", "workspace"),
                       fp8_linear=("out", "workspace"), fp8_grouped=("out", "sorted_route"),
                       sort_tokens=("rows",), unsort_tokens=("out", "topk_w"),
                       unsort_tokens_grad=("drows", "dw"),
                       permute=("expert_offsets", "sorted_route", "route_row"))[name]
    for key, value in buffers(m)[name].items():
        if not isinstance(value, torch.Tensor):
            continue
        for i, bad in enumerate(wrong(value)):
            if bad is None and key in may_be_none:
                continue
            # Fewer rows are taken (routes past them have no part), and a workspace of more bytes
            # than these calls need, in any shape.
            if i == 1 and (name, key) in (("sort_tokens", "rows"), ("unsort_tokens", "rows"),
                                          ("fp8_matmul", "workspace"), ("permute", "workspace")):
                continue
            if i == 3 and key == "workspace":
                continue
            kw = buffers(m)[name]
            kw[key] = bad
            with pytest.raises((ValueError, m.MoEError, AttributeError, TypeError)):
                getattr(m, "moe_" + name)(**kw)
                pytest.fail(f"{key}: wrong({i}) was taken")
    for key in ("top_k", "E_local"):
        kw = buffers(m)[name]
        if key in kw:
            for bad in (0, -1, kw[key] + 1, 1 << 40):
                if name == "fp8_grouped" and bad > 0 and bad < 64:
                    continue                          # routes of other tokens, but routes
                kw[key] = bad
                with pytest.raises((ValueError, m.MoEError)):
                    getattr(m, "moe_" + name)(**kw)
                    pytest.fail(f"{key} = {bad} was taken")
