"""64-bit references of the norm and projection operators (test infrastructure)."""
import numpy as np
import torch


def quantized(seed, N, K):
    """Codes [N][K/2], fp16 scales [N][K/32] of N(0, 0.02) weights, and the weights in fp64 (CPU)."""
    g = torch.Generator().manual_seed(seed)
    w = 0.02 * torch.randn(N, K // 32, 32, generator=g)
    s = (w.abs().amax(-1) / 7).half()
    c = torch.round(w / s.float()[..., None]).clamp(-8, 7)
    u = (c + 8).to(torch.uint8).view(N, K // 2, 2)
    q = u[..., 0] | (u[..., 1] << 4)
    return q.contiguous(), s, (c.double() * s.double()[..., None]).view(N, K)


def product(x64, w64, bias=None):
    y = x64 @ w64.T
    return y if bias is None else y + bias.double()


EXACT_TOKENS, EXACT_WEIGHTS = 8, 1 << 25  # the largest call whose operands are not rounded to fp16


def product_bound(x64, w64, y64, bias=None, tokens=1, bf16=True):
    """Largest error of a bf16 y in a call on `tokens` tokens of bf16 (or 8-bit) x.

    fp32 accumulation: the products of a 32-input block are summed apart, then
    the K/32 block sums; each addition is off by at most 2^-22 of the sum of
    magnitudes (the tensor cores truncate: twice fp32's step 2^-23), a few more
    for the scales: (32 + K/32 + 8) 2^-22 of sum |x||w|.  (One long chain on the
    tensor cores adds 16 products at a time, K/16 additions: K/16 2^-22.)
    One bf16 token: x as multiples of 2^(e - 13), with 2^e at most
    the largest |x| of the block: off by 2^-14 of that at most.
    Above EXACT_TOKENS or EXACT_WEIGHTS the operands may be fp16: each weight is rounded once,
    2^-11 of itself, or, below 2^-14 in units where the row's largest scale is
    at least 2^-9, twice by 2^-25, so 2^-15 of the row's largest scale, which is
    at most its largest |weight| where that block has a code other than 8.
    x loses what lies below 2^-25 of the token's largest |x|.
    Then half a bf16 step of the result."""
    K = x64.shape[1]
    ax, aw = x64.abs(), w64.abs()
    mag = ax @ aw.T + (0 if bias is None else bias.double().abs())
    err = mag * ((32 + K / 16 + 8) * 2.0 ** -22)
    if bf16 and tokens == 1:
        top = ax.view(-1, K // 32, 32).amax(-1).repeat_interleave(32, 1)
        err = err + 2.0 ** -14 * (top @ aw.T)
    if tokens > EXACT_TOKENS or (tokens > 1 and w64.numel() > EXACT_WEIGHTS):
        err = err + 2.0 ** -11 * mag + 2.0 ** -15 * ax.sum(1, keepdim=True) * aw.amax(1)
        err = err + 2.0 ** -25 * ax.amax(1, keepdim=True) * aw.sum(1)
    return err + (y64.abs() + err) * 2.0 ** -8 + 1e-38


def add_rmsnorm(x, r, g, eps):
    """(h as bf16, u in fp64) from the definition."""
    h = x if r is None else (x.double() + r.double()).to(torch.bfloat16)
    h64 = h.double()
    u = h64 / torch.sqrt((h64 * h64).mean(-1, keepdim=True) + eps)
    return h, u if g is None else u * g.double()


def q8_values(q, s):
    T, K = q.shape
    return (q.double().view(T, K // 32, 32) * s.double()[..., None]).view(T, K)


def as_np(t):
    return np.ascontiguousarray(t.cpu().numpy())
