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


def product_bound(x64, w64, y64, bias=None, weight_rounding=0.0):
    """Largest error of a bf16 y.  fp32 accumulation: every one of the K
    additions, in whatever order, is off by at most 2^-22 of the running sum of
    magnitudes (the tensor cores truncate: twice fp32's 2^-23 step), so K 2^-22
    of sum |x||w|, and never more than the 2^-11 that K = 2048 gives because the
    32-input blocks are summed apart: (32 + K/32 + 8) 2^-22.  weight_rounding:
    relative rounding of each weight.  Then half a bf16 step of the result."""
    K = x64.shape[1]
    mag = x64.abs() @ w64.abs().T + (0 if bias is None else bias.double().abs())
    err = mag * ((32 + K / 32 + 8) * 2.0 ** -22 + weight_rounding)
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
