"""The operators as a model runs them around an MoE layer: norm, 4-bit
projection, residual norm, MoE layer, final 8-bit norm and output head."""
import numpy as np
import pytest
import torch

import oracle
import quantized_expert_ffn_softmax_gb300 as moe
import workload as W
import operators_ref as R

pytestmark = pytest.mark.gpu

WEIGHTS = ("router_w", "slot_of_expert", "gate_q", "gate_s", "up_q", "up_s", "down_q", "down_s", "sh_gate_q",
           "sh_gate_s", "sh_up_q", "sh_up_s", "sh_down_q", "sh_down_s")


@pytest.fixture(scope="module")
def model():
    cfg = W.CONFIGS["tiny"]
    L = W.layer(cfg, 0)
    w = {n: L[n] for n in WEIGHTS}
    w["router_bias"] = L["router_b"]
    layer = moe.MoELayer(dict(hidden=cfg.hidden, n_experts=cfg.n_experts, top_k=cfg.top_k, ffn=cfg.ffn,
                              shared_ffn=cfg.shared_ffn, max_tokens=64), w, weights_on_device=False)
    H, V = cfg.hidden, 1003
    q0, s0, w0 = R.quantized(1, H, H)
    q1, s1, w1 = R.quantized(2, V, H)
    proj = moe.MoELinear(dict(in_features=H, out_features=H, max_tokens=64), dict(q=q0, s=s0), False)
    head = moe.MoELinear(dict(in_features=H, out_features=V, max_tokens=64), dict(q=q1, s=s1), False)
    gains = [1 + 0.2 * torch.randn(H, generator=torch.Generator().manual_seed(i)) for i in range(3)]
    return cfg, L, layer, proj, w0, head, w1, gains


def bits(t):
    return np.ascontiguousarray(t.cpu().view(torch.int16).numpy().view(np.uint16))


def run(model, h, gains, bufs=None):
    cfg, _, layer, proj, _, head, _, _ = model
    _, u0 = moe.add_rmsnorm(h, None, gains[0])
    a = proj.forward(u0)
    h1, u1 = moe.add_rmsnorm(a, h, gains[1])
    m = layer.forward(u1)
    if h.shape[0] <= 32:
        h2, q, s = moe.add_rmsnorm(m, h1, gains[2], q8=True)
        return u0, a, h1, u1, m, h2, (q, s), head.forward_q8(q, s)
    h2, u2 = moe.add_rmsnorm(m, h1, gains[2])
    return u0, a, h1, u1, m, h2, u2, head.forward(u2)


@pytest.mark.parametrize("T", [1, 4, 9, 40])
def test_block(cuda_device, model, T):
    cfg, L, layer, _, w0, _, w1, gains = model
    gd = [g.to(cuda_device) for g in gains]
    h = torch.randn(T, cfg.hidden, generator=torch.Generator().manual_seed(T)).bfloat16()
    u0, a, h1, u1, m, h2, u2, logits = run(model, h.to(cuda_device), gd)
    rtol = 2.0 ** -8 + 2.0 ** -12
    # every step against the definition on the GPU's own input of that step
    want = R.add_rmsnorm(h, None, gains[0], 1e-6)[1]
    assert ((u0.cpu().double() - want).abs() <= rtol * want.abs()).all()
    x64 = u0.cpu().double()
    y64 = R.product(x64, w0)
    assert ((a.cpu().double() - y64).abs() <= R.product_bound(x64, w0, y64, None, T)).all()
    hr, want = R.add_rmsnorm(a.cpu(), h, gains[1], 1e-6)
    assert torch.allclose(h1.cpu().double(), hr.double(), rtol=2 ** -7, atol=0)
    want = R.add_rmsnorm(h1.cpu(), None, gains[1], 1e-6)[1]
    assert ((u1.cpu().double() - want).abs() <= rtol * want.abs()).all()
    y_ref, _, _, margin = oracle.moe_forward(L, cfg.top_k, bits(u1))
    if margin.min() >= 1e-4:
        y_ref = torch.from_numpy(y_ref)
        assert ((m.cpu().double() - y_ref).abs().amax(1) <= 1e-2 * y_ref.abs().amax(1) + 1e-3).all()
    assert torch.allclose(h2.cpu().double(), R.add_rmsnorm(m.cpu(), h1.cpu(), None, 1e-6)[0].double(), rtol=2 ** -7,
                          atol=0)
    x64 = R.q8_values(u2[0].cpu(), u2[1].cpu()) if T <= 32 else u2.cpu().double()
    y64 = R.product(x64, w1)
    assert ((logits.cpu().double() - y64).abs() <= R.product_bound(x64, w1, y64, None, T, T > 32)).all()


@pytest.mark.parametrize("T", [1, 40])
def test_block_in_a_graph(cuda_device, model, T):
    """Captured once, replayed on new inputs, equal to the eager run up to the
    MoE layer's documented one-rounding freedom."""
    cfg, layer, proj, head = model[0], model[2], model[3], model[5]
    H, V = cfg.hidden, 1003
    gd = [g.to(cuda_device) for g in model[7]]
    h = torch.zeros(T, H, dtype=torch.bfloat16, device=cuda_device)
    u, a, m = (torch.zeros_like(h) for _ in range(3))
    h1 = torch.zeros_like(h)
    logits = torch.zeros(T, V, dtype=torch.bfloat16, device=cuda_device)
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        moe.moe_add_rmsnorm(h, None, gd[0], 1e-6, T, H, None, u)
        moe.moe_linear_forward(proj.handle, u, T, a)
        moe.moe_add_rmsnorm(a, h, gd[1], 1e-6, T, H, h1, u)
        moe.moe_forward(layer.handle, u, T, m)
        moe.moe_add_rmsnorm(m, h1, gd[2], 1e-6, T, H, h1, u)
        moe.moe_linear_forward(head.handle, u, T, logits)
    for seed in range(3):
        h.copy_(torch.randn(T, H, generator=torch.Generator().manual_seed(seed)).bfloat16())
        g.replay()
        # the captured chain's last steps on the graph's own m and the eager chain's first ones
        _, u0 = moe.add_rmsnorm(h, None, gd[0])
        a0 = proj.forward(u0)
        h10, u10 = moe.add_rmsnorm(a0, h, gd[1])
        m0 = layer.forward(u10)
        assert torch.equal(a, a0)
        assert torch.allclose(m.float(), m0.float(), rtol=2 ** -6, atol=1e-3)
        h2, u2 = moe.add_rmsnorm(m, h10, gd[2])
        assert torch.equal(h1, h2) and torch.equal(u, u2)
        assert torch.equal(logits, head.forward(u2))
    assert moe.moe_status_sync(layer.handle) == moe.MOE_OK
