"""Cases of the operators that run around the MoE layer in a model: the norm
that feeds it (with the residual's addition, bf16 or 8-bit output) and the
projections with 4-bit weights in the experts' format.

  norm     h = bf16(x + r), u = h / sqrt(mean(h^2) + eps) * g in bf16
  linear   y = x W^T + b, W in 4-bit codes with one fp16 scale per 32 inputs
  project  the decode form of both in 8 bits: the norm writes u as 8-bit
           codes with one scale per 32 values, the projection reads them

`run` computes them in elementary torch operations in 32 bits, or, where
`own` is true, calls the library.
"""
import math

import torch

own = False

EPS = 1e-6
DEVICE = "cuda"


def listed():
    return [
        # one decode token into an MoE layer of the 35B-shaped stack
        dict(name="norm 1x2048", op="norm", T=1, K=2048, residual=True),
        # a ragged prompt, a wide model, the first norm of a model (no residual)
        dict(name="norm 777x5120 first", op="norm", T=777, K=5120, residual=False),
        # a prefill chunk of the benchmark's size
        dict(name="norm 8192x2048", op="norm", T=8192, K=2048, residual=True),
        # a decode token's square projection, the smallest product of a step
        dict(name="linear 1 2048-2048", op="linear", T=1, K=2048, N=2048, bias=False),
        # the output head on one token; a vocabulary that is no multiple of a tile
        dict(name="linear 1 2048-131073", op="linear", T=1, K=2048, N=131073, bias=False),
        # a batch of 32 requests, one token each
        dict(name="linear 32 4096-8192", op="linear", T=32, K=4096, N=8192, bias=True),
        # the ragged tail of a prompt into an odd number of outputs
        dict(name="linear 200 2080-4111", op="linear", T=200, K=2080, N=4111, bias=True),
        # a short prompt
        dict(name="linear 1024 2048-5120", op="linear", T=1024, K=2048, N=5120, bias=False),
        # a prefill chunk of the benchmark's size
        dict(name="linear 8192 2048-8192", op="linear", T=8192, K=2048, N=8192, bias=False),
        # a decode token and a verify batch of one token and three drafts: norm, then a fused projection
        dict(name="project 1 2048-2560", op="project", T=1, K=2048, N=2560, bias=True, residual=True),
        dict(name="project 4 2048-8192", op="project", T=4, K=2048, N=8192, bias=False, residual=True),
        # a small batch into a wide layer
        dict(name="project 16 5120-10240", op="project", T=16, K=5120, N=10240, bias=False, residual=True),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "linear", "linear", "project"])
    while True:
        K = 32 * _spread(rng, 8, 256)
        if op == "norm":
            T = _spread(rng, 1, 8192)
            if T * K <= 8192 * 2048:
                return dict(op=op, T=T, K=K, residual=rng.random() < 0.75)
            continue
        N = _spread(rng, 64, 131073)
        T = _spread(rng, 1, 32 if op == "project" else 8192)
        if N * K > 131073 * 2048 or T * N * K > 8192 * 2048 * 8192:
            continue
        case = dict(op=op, T=T, K=K, N=N, bias=rng.random() < 0.5)
        if op == "project":
            case["residual"] = rng.random() < 0.75
        return case


def _normal(gen, *shape):
    return torch.randn(*shape, generator=gen, device=DEVICE, dtype=torch.float32)


def _quantized(gen, N, K):
    """Weights N(0, 0.02) as the experts' are: codes [N][K/2] (element 2i in the
    low nibble of byte i), fp16 scales [N][K/32], weight = (code - 8) * scale."""
    q = torch.empty(N, K // 2, device=DEVICE, dtype=torch.uint8)
    s = torch.empty(N, K // 32, device=DEVICE, dtype=torch.float16)
    for r in range(0, N, 32768):
        w = 0.02 * _normal(gen, min(32768, N - r), K // 32, 32)
        sc = (w.abs().amax(-1) / 7).half()
        c = torch.round(w / sc.float()[..., None]).clamp_(-8, 7).add_(8).to(torch.uint8).view(-1, K // 2, 2)
        q[r:r + 32768] = c[..., 0] | (c[..., 1] << 4)
        s[r:r + 32768] = sc
    return q, s


def prepare(case, seed):
    gen = torch.Generator(device=DEVICE)
    gen.manual_seed(seed)
    T, K, op = case["T"], case["K"], case["op"]
    st = dict(case)
    st["x"] = _normal(gen, T, K).bfloat16()
    if op != "linear":
        # the residual stream's rows differ in size, and a few channels stand out
        st["r"] = None
        if case["residual"]:
            r = _normal(gen, T, K) * torch.exp(_normal(gen, T, 1))
            r[:, :: 97] *= 12
            st["r"] = r.bfloat16()
        st["g"] = 1 + 0.2 * _normal(gen, K)
        st["h"] = torch.empty_like(st["x"])
        st["u"] = torch.empty_like(st["x"])
    if op != "norm":
        N = case["N"]
        st["q"], st["s"] = _quantized(gen, N, K)
        st["b"] = 0.1 * _normal(gen, N) if case["bias"] else None
        st["y"] = torch.empty(T, N, device=DEVICE, dtype=torch.bfloat16)
    if op == "project":
        st["u8"] = torch.empty(T, K, device=DEVICE, dtype=torch.int8)
        st["us"] = torch.empty(T, K // 32, device=DEVICE, dtype=torch.float32)
    if own:
        import quantized_expert_ffn_softmax_gb300 as moe

        st["moe"] = moe
        if op != "norm":
            st["linear"] = moe.MoELinear(dict(in_features=K, out_features=case["N"], max_tokens=T),
                                         dict(q=st["q"], s=st["s"], bias=st["b"]), weights_on_device=True)
    return st


def _norm32(st):
    h = st["x"]
    if st["r"] is not None:
        h = (h.float() + st["r"].float()).bfloat16()
    hf = h.float()
    u = hf * torch.rsqrt((hf * hf).mean(-1, keepdim=True) + EPS) * st["g"]
    return h, u


def _weights32(st):
    q = st["q"]
    N, K = st["N"], st["K"]
    c = torch.stack((q & 15, q >> 4), -1).view(N, K // 32, 32).float() - 8
    return (c * st["s"].float()[..., None]).view(N, K)


def _product32(st, x):
    y = x @ _weights32(st).t()
    if st["b"] is not None:
        y = y + st["b"]
    return y.bfloat16()


def run(st):
    op, T, K = st["op"], st["T"], st["K"]
    if own:
        moe = st["moe"]
        if op == "norm":
            moe.moe_add_rmsnorm(st["x"], st["r"], st["g"], EPS, T, K, st["h"], st["u"])
            return dict(h=st["h"], u=st["u"])
        if op == "linear":
            moe.moe_linear_forward(st["linear"].handle, st["x"], T, st["y"])
            return st["y"]
        moe.moe_add_rmsnorm_q8(st["x"], st["r"], st["g"], EPS, T, K, st["h"], st["u8"], st["us"])
        moe.moe_linear_forward_q8(st["linear"].handle, st["u8"], st["us"], T, st["y"])
        return dict(h=st["h"], y=st["y"])
    if op == "norm":
        h, u = _norm32(st)
        return dict(h=h, u=u.bfloat16())
    if op == "linear":
        return _product32(st, st["x"].float())
    h, u = _norm32(st)
    b = u.view(T, K // 32, 32)
    s = b.abs().amax(-1, keepdim=True) / 127
    q = torch.where(s > 0, torch.round(b / s), torch.zeros_like(b)).clamp(-127, 127)
    return dict(h=h, y=_product32(st, (q * s).view(T, K)))


def work(case):
    T, K, op = case["T"], case["K"], case["op"]
    nbytes = flops = 0
    if op != "linear":
        rows = 3 if case["residual"] else 2  # x, h and the residual
        nbytes += 2 * T * K * rows + 4 * K + (2 * T * K if op == "norm" else 0)
        flops += 5 * T * K
    if op != "norm":
        N = case["N"]
        nbytes += N * K // 2 + 2 * N * (K // 32) + 2 * T * N + (4 * N if case["bias"] else 0)
        nbytes += 2 * T * K if op == "linear" else 0
        flops += 2 * T * N * K
    return dict(bytes=nbytes, flops=flops)


def exact(case, seed):
    """The definitions in 64 bits, row by row of W and without the plain form's steps."""
    st = prepare(case, seed)
    op, T, K = case["op"], case["T"], case["K"]
    x = st["x"].double()
    out = {}
    if op != "linear":
        h = x if st["r"] is None else (x + st["r"].double()).bfloat16().double()
        norm = torch.linalg.vector_norm(h, dim=1, keepdim=True)
        u = h / torch.sqrt(norm.square() / K + EPS) * st["g"].double()[None]
        out["h"] = h
        if op == "norm":
            out["u"] = u
            return out
        top = u.unflatten(1, (K // 32, 32)).abs().max(2).values.repeat_interleave(32, 1)
        x = torch.round(torch.nan_to_num(u * 127 / top)) * top / 127
    N = case["N"]
    y = torch.empty(T, N, device=DEVICE, dtype=torch.float64)
    low = torch.arange(0, 16, device=DEVICE, dtype=torch.float64) - 8
    for n in range(0, N, 8192):
        q = st["q"][n:n + 8192].long()
        w = torch.empty(q.shape[0], K, device=DEVICE, dtype=torch.float64)
        w[:, 0::2] = low[q % 16]
        w[:, 1::2] = low[q // 16]
        w *= st["s"][n:n + 8192].double().repeat_interleave(32, 1)
        y[:, n:n + 8192] = torch.matmul(x, w.T)
    if st["b"] is not None:
        y += st["b"].double()
    if op == "linear":
        return y
    out["y"] = y
    return out
