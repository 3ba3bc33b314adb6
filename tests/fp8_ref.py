"""Plain references of the block-scaled FP8 products, in 64 bits but for the tokens' codes,
whose rule is in float32."""
import torch

FP8 = torch.float8_e4m3fn
BLOCK = 128


def blocks(n):
    return (n + BLOCK - 1) // BLOCK


def quant(x):
    """bf16 [T, H] -> (codes uint8 [T, H], scales float [KB, T]) by the rule of moe_quant_fp8, on
    the CPU in float32."""
    x = x.cpu().float()
    T, H = x.shape
    f = torch.zeros(T, blocks(H) * BLOCK)
    f[:, :H] = x
    f = f.view(T, -1, BLOCK)
    amax = torch.where(torch.isfinite(f), f.abs(), torch.full_like(f, torch.inf)).amax(2)
    odd = torch.isinf(amax)
    s = (amax / torch.tensor(448.0)).clamp_min(2.0 ** -126)
    q = torch.where(odd[..., None], torch.zeros(()), f * (1.0 / s)[..., None])
    q = q.clamp(-448.0, 448.0).to(FP8).view(torch.uint8).reshape(T, -1)[:, :H]
    return q.contiguous(), torch.where(odd, torch.nan, s).t().contiguous()


def weight(N, K, seed, E=None, spread=2.0):
    """Random codes of every magnitude and scales that differ from block to block."""
    g = torch.Generator().manual_seed(seed)
    shape = (N, K) if E is None else (E, N, K)
    w = torch.randn(*shape, generator=g).to(FP8)
    s = torch.exp(spread * torch.randn(*shape[:-2], blocks(N), blocks(K), generator=g)) * 1e-2
    return w, s


def tokens(T, H, seed):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(T, H, generator=g) * torch.exp(2 * torch.randn(T, 1, generator=g))
            ).to(torch.bfloat16)


def product(q, xs, w, w_s):
    """The product and the sum of |products|, in 64 bits: q uint8 [M, K], xs [KB, M], w [N, K] FP8,
    w_s [NB, KB], on one device."""
    a = q.view(FP8).float().double()
    b = w.view(FP8).float().double()
    M, K = a.shape
    N = b.shape[0]
    a = a * xs.double().t().repeat_interleave(BLOCK, 1)[:, :K]
    b = b * w_s.double().repeat_interleave(BLOCK, 0)[:N].repeat_interleave(BLOCK, 1)[:, :K]
    return a @ b.t(), a.abs() @ b.abs().t()


def bound(ref, mag):
    """What a product may be off: half a step of bf16; the matrix unit's accumulation, 2^-15 of the
    sum of |products| (the worst that a block's sum has shown is 2^-16.8 of it); the scales'
    product and the float sum over up to 2^7 blocks, 2^-16 of that sum at most; and bf16's
    smallest steps."""
    return ref.abs() * 2.0 ** -8 * (1 + 2.0 ** -7) + mag * (2.0 ** -15 + 2.0 ** -16) + 1e-38


def check(out, ref, mag, what=""):
    out = out.double().to(ref.device)
    nan = torch.isnan(ref)
    assert torch.equal(torch.isnan(out), nan), what
    worst = ((out - ref).abs() / bound(ref, mag)).nan_to_num(0.0)
    assert worst.max().item() <= 1.0, (what, worst.max().item())
