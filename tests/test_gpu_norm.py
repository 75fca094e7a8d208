"""moe_add_rmsnorm against the definition in 64 bits.

Tolerances.  h: the fp32 sum of two bf16 values rounded to bf16 equals the
64-bit sum rounded to bf16 except where the fp32 rounding lands on a bf16 tie
(double rounding): then one bf16 step, 2^-7 relative.  u: fp32 sum of squares
(relative 2^-24 per addition, at most H/8 + 40 of them in a chain: below
2^-12 at H = 32768, halved by the square root), rsqrtf and two products (a few
2^-23), then half a bf16 step, 2^-8: rtol 2^-8 + 2^-12.  8-bit u: half a code
step of the block's scale, (max|u| / 127) / 2, plus the same 2^-12 of the value
for the fp32 part and of the scale."""
import pytest
import torch

import quantized_expert_ffn_softmax_gb300 as moe
import operators_ref as R

pytestmark = pytest.mark.gpu

SHAPES = [(1, 32), (1, 2048), (2, 64), (3, 8192), (5, 8224), (7, 2080), (33, 256), (64, 5120), (129, 96), (1, 32768),
          (2, 16416), (1000, 512), (4097, 128), (700, 2048), (800, 4096), (600, 1056), (1025, 32),
          (1100, 288), (1030, 544), (300, 16416), (257, 8224)]


def inputs(T, H, residual, gain, seed=0):
    g = torch.Generator().manual_seed(seed * 7919 + T * 31 + H)
    x = torch.randn(T, H, generator=g).bfloat16()
    r = (torch.randn(T, H, generator=g) * torch.exp(torch.randn(T, 1, generator=g))).bfloat16() if residual else None
    w = 1 + 0.3 * torch.randn(H, generator=g) if gain else None
    return x, r, w


def dev(t, d):
    return None if t is None else t.to(d)


def close(got, want, rtol, atol=0.0):
    got, want = got.double().cpu(), want.double()
    bad = (got - want).abs() > rtol * want.abs() + atol
    assert not bad.any(), (bad.sum().item(), (got - want).abs().max().item())


@pytest.mark.parametrize("T,H", SHAPES)
@pytest.mark.parametrize("residual,gain", [(True, True), (False, False), (True, False), (False, True)])
def test_bf16(cuda_device, T, H, residual, gain):
    x, r, w = inputs(T, H, residual, gain)
    h, u = moe.add_rmsnorm(dev(x, cuda_device), dev(r, cuda_device), dev(w, cuda_device), 1e-6)
    h_ref, _ = R.add_rmsnorm(x, r, w, 1e-6)
    close(h, h_ref, 2.0 ** -7)
    _, u_ref = R.add_rmsnorm(h.cpu(), None, w, 1e-6)
    close(u, u_ref, 2.0 ** -8 + 2.0 ** -12)


@pytest.mark.parametrize("T,H", SHAPES)
@pytest.mark.parametrize("residual,gain", [(True, True), (False, False)])
def test_q8(cuda_device, T, H, residual, gain):
    x, r, w = inputs(T, H, residual, gain, 1)
    h, q, s = moe.add_rmsnorm(dev(x, cuda_device), dev(r, cuda_device), dev(w, cuda_device), 1e-6, q8=True)
    _, u = R.add_rmsnorm(h.cpu(), None, w, 1e-6)
    top = u.view(T, H // 32, 32).abs().amax(-1)
    close(s, top / 127, 2.0 ** -12)
    assert int(q.max()) <= 127 and int(q.min()) >= -127
    step = (top / 127).repeat_interleave(32, 1)
    off = (R.q8_values(q.cpu(), s.cpu()) - u).abs()
    assert (off <= 0.5 * step * (1 + 2.0 ** -10) + 2.0 ** -11 * u.abs()).all()


def test_rows_do_not_depend_on_the_batch(cuda_device):
    x, r, w = (dev(t, cuda_device) for t in inputs(700, 2048, True, True))
    h, u = moe.add_rmsnorm(x, r, w)
    for t in (0, 1, 350, 699):
        h1, u1 = moe.add_rmsnorm(x[t:t + 1].contiguous(), r[t:t + 1].contiguous(), w)
        assert torch.equal(h1[0], h[t]) and torch.allclose(u1[0].float(), u[t].float(), rtol=2 ** -7, atol=0)


@pytest.mark.parametrize("T,H", [(3, 512), (900, 2048), (2, 16416)])
def test_in_place(cuda_device, T, H):
    x, r, w = (dev(t, cuda_device) for t in inputs(T, H, True, True))
    h0, u0 = moe.add_rmsnorm(x, r, w)
    x1, r1 = x.clone(), r.clone()
    moe.moe_add_rmsnorm(x1, r1, w, 1e-6, T, H, r1, x1)  # h over the residual, u over x
    assert torch.equal(r1, h0) and torch.equal(x1, u0)
    x2 = x.clone()
    moe.moe_add_rmsnorm(x2, r, w, 1e-6, T, H, x2, r.clone())
    assert torch.equal(x2, h0)


@pytest.mark.parametrize("H,T", [(128, 2), (2048, 600), (16416, 2)])
def test_extreme_rows(cuda_device, H, T):
    """Zeros, the smallest and the largest finite values, infinities and NaN."""
    x = torch.randn(T, H, generator=torch.Generator().manual_seed(4)).bfloat16()
    x[0] = 0
    x[1] = (x[1].float() * 1e37).bfloat16()  # squares overflow fp32
    xd = x.to(cuda_device)
    _, u = moe.add_rmsnorm(xd, None, None, 1e-6)
    assert (u[0] == 0).all()
    close(u, R.add_rmsnorm(x, None, None, 1e-6)[1], 2.0 ** -8 + 2.0 ** -12)
    _, q, s = moe.add_rmsnorm(xd, None, None, 1e-6, q8=True)
    assert (q[0] == 0).all() and (s[0] == 0).all()
    x[0] = 1e-30
    x[0, 5] = float("inf")
    x[1, 7] = float("nan")
    _, u = moe.add_rmsnorm(x.to(cuda_device))
    assert torch.isnan(u[0, 5]) and (u[0, 6:] == 0).all() and torch.isnan(u[1]).all()
    _, q, s = moe.add_rmsnorm(x.to(cuda_device), q8=True)
    assert torch.isnan(s[0, 0]) and (s[0, 1:] == 0).all() and torch.isnan(s[1]).all()
    assert (q[:2] == 0).all() and torch.isfinite(s[2:]).all()


def test_guard_rows_stay(cuda_device):
    """Nothing is written past the last row."""
    T, H = 3, 2080
    x, r, w = (dev(t, cuda_device) for t in inputs(T, H, True, True))
    h, u = (torch.full((T + 1, H), 7.0, dtype=torch.bfloat16, device=cuda_device) for _ in range(2))
    moe.moe_add_rmsnorm(x, r, w, 1e-6, T, H, h, u)
    assert (h[T] == 7).all() and (u[T] == 7).all()
    q = torch.full((T + 1, H), 9, dtype=torch.int8, device=cuda_device)
    s = torch.full((T + 1, H // 32), 7.0, device=cuda_device)
    moe.moe_add_rmsnorm_q8(x, r, w, 1e-6, T, H, h, q, s)
    assert (q[T] == 9).all() and (s[T] == 7).all()


def test_offsets_past_32_bits(cuda_device):
    """Rows of a 4.3 GB input against calls on those rows alone."""
    T, H = 65536, 32768
    x = torch.randn(1024, H, device=cuda_device).bfloat16().repeat(T // 1024, 1)
    x[T - 1] = 3
    h, u = torch.empty_like(x), torch.empty_like(x)
    moe.moe_add_rmsnorm(x, x, None, 1e-6, T, H, h, u)
    for t in (0, 40000, T - 1):
        row = x[t:t + 1].contiguous()
        h1, u1 = moe.add_rmsnorm(row, row)
        assert torch.equal(h[t], h1[0]) and torch.equal(u[t], u1[0])
    del h, u
    q = torch.empty(T, H, dtype=torch.int8, device=cuda_device)
    s = torch.empty(T, H // 32, device=cuda_device)
    moe.moe_add_rmsnorm_q8(x, None, None, 1e-6, T, H, None, q, s)
    for t in (0, 40000, T - 1):
        _, q1, s1 = moe.add_rmsnorm(x[t:t + 1].contiguous(), q8=True)
        assert torch.equal(q[t], q1[0]) and torch.equal(s[t], s1[0])


def test_refusals(cuda_device):
    T, H = 4, 64
    x, r, w = (dev(t, cuda_device) for t in inputs(T, H, True, True))
    u = torch.empty_like(x)
    flat = torch.zeros(4 * T * H, dtype=torch.bfloat16, device=cuda_device)

    def refuse(*a):
        with pytest.raises(moe.MoeError) as ei:
            moe.moe_add_rmsnorm(*a)
        assert ei.value.status == moe.MOE_ERR_INVALID
        return moe.moe_last_error()

    assert "NULL" in refuse(None, r, w, 1e-6, T, H, None, u)
    assert "NULL" in refuse(x, r, w, 1e-6, T, H, None, None)
    assert "x" in refuse(x.cpu(), r, w, 1e-6, T, H, None, u)
    assert "aligned" in refuse(flat[1:1 + T * H], None, None, 1e-6, T, H, None, u)
    assert "overlaps" in refuse(x, r, w, 1e-6, T, H, u, u)
    assert "overlaps" in refuse(flat[:T * H], None, None, 1e-6, T, H, None, flat[8:8 + T * H])
    q = torch.empty(2 * T * H, dtype=torch.int8, device=cuda_device)
    s = torch.empty(T * H // 32, device=cuda_device)
    with pytest.raises(moe.MoeError):
        moe.moe_add_rmsnorm_q8(x, r, w, 1e-6, T, H, None, x, s)
    with pytest.raises(moe.MoeError):
        moe.moe_add_rmsnorm_q8(x, r, w, 1e-6, T, H, None, q, None)
    with pytest.raises(ValueError):
        moe.add_rmsnorm(x.float())
    with pytest.raises(ValueError):
        moe.add_rmsnorm(x, r[:2])
    with pytest.raises(ValueError):
        moe.add_rmsnorm(x, r, w.bfloat16())
    with pytest.raises(ValueError):
        moe.add_rmsnorm(x.t())  # not contiguous


def test_side_stream_and_graph(cuda_device):
    T, H = 4, 2048
    x, r, w = (dev(t, cuda_device) for t in inputs(T, H, True, True))
    h0, u0 = moe.add_rmsnorm(x, r, w)
    h, u = torch.zeros_like(x), torch.zeros_like(x)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    moe.moe_add_rmsnorm(x, r, w, 1e-6, T, H, h, u, st)
    st.synchronize()
    assert torch.equal(h, h0) and torch.equal(u, u0)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        moe.moe_add_rmsnorm(x, r, w, 1e-6, T, H, h, u)
        moe.moe_add_rmsnorm(u, h, w, 1e-6, T, H, None, r)  # reads what the first wrote, over its input
    r0 = r.clone()
    for _ in range(3):
        r.copy_(r0)
        g.replay()
    want = moe.add_rmsnorm(u0, h0, w)[1]
    assert torch.equal(u, u0) and torch.equal(r, want)
