"""moe_linear against the product in 64 bits (bounds: operators_ref.product_bound)."""
import pytest
import torch

import quantized_expert_ffn_softmax_gb300 as moe
import operators_ref as R

pytestmark = pytest.mark.gpu


def make(N, K, T, bias, device, seed=0):
    q, s, w = R.quantized(seed + N + K, N, K)
    b = 0.3 * torch.randn(N, generator=torch.Generator().manual_seed(seed + 5)) if bias else None
    lin = moe.MoELinear(dict(in_features=K, out_features=N, max_tokens=T), dict(q=q, s=s, bias=b), False)
    return lin, w, b


def acts(T, K, seed=0):
    g = torch.Generator().manual_seed(1000 + seed + T * 17 + K)
    return (torch.randn(T, K, generator=g) * torch.exp(torch.randn(T, 1, generator=g))).bfloat16()


def check(y, x64, w64, bias, tokens=None, bf16=True):
    y64 = R.product(x64, w64, bias)
    off = (y.double().cpu() - y64).abs()
    bound = R.product_bound(x64, w64, y64, bias, tokens or x64.shape[0], bf16)
    assert (off <= bound).all(), (off / bound).max().item()


SMALL = [(1, 16, 32), (2, 16, 32), (4, 30, 32), (1, 50, 16384), (1, 30, 32768), (2, 3000, 10272), (2, 90000, 512), (5, 45000, 2048), (1, 40, 12288), (3, 700, 2048), (1, 1, 32), (1, 17, 64), (1, 2048, 2048), (2, 100, 96), (3, 2049, 160), (4, 33, 8192), (5, 640, 1056),
         (8, 257, 2080), (9, 1000, 256), (16, 4099, 512), (17, 48, 2048), (31, 515, 1024), (32, 1024, 4096),
         (1, 40000, 256), (8, 5000, 4128), (32, 16, 32768), (24, 9000, 128)]


@pytest.mark.parametrize("T,N,K", SMALL)
@pytest.mark.parametrize("bias", [False, True])
def test_small_batches(cuda_device, T, N, K, bias):
    lin, w, b = make(N, K, T, bias, cuda_device)
    x = acts(T, K)
    y = lin.forward(x.to(cuda_device))
    check(y, x.double(), w, b)
    assert moe.moe_linear_status_sync(lin.handle) == moe.MOE_OK


@pytest.mark.parametrize("T,N,K", SMALL + [(9, 4000, 2080), (16, 5000, 2048), (3, 18000, 2048), (2, 18000, 2048), (2, 60, 16384), (33, 100, 64), (100, 4111, 2080), (300, 777, 1056), (40, 70, 16416)])
def test_q8(cuda_device, T, N, K):
    lin, w, b = make(N, K, T, True, cuda_device)
    g = torch.Generator().manual_seed(T + N + K)
    q = torch.randint(-127, 128, (T, K), generator=g).to(torch.int8)
    s = torch.rand(T, K // 32, generator=g) + 0.01
    y = lin.forward_q8(q.to(cuda_device), s.to(cuda_device))
    check(y, R.q8_values(q, s), w, b, bf16=False)


LARGE = [(9, 30000, 2048), (17, 30, 64), (16, 24000, 2080), (33, 100, 64), (40, 2048, 2048), (64, 300, 96), (65, 1, 32), (100, 4111, 2080), (128, 128, 128),
         (129, 513, 1056), (200, 777, 4096), (256, 256, 256), (257, 1025, 544), (511, 48, 8192), (700, 2560, 2048),
         (1025, 640, 160), (2050, 2050, 320), (65, 20000, 64), (40, 70000, 32), (48, 130, 32768), (5000, 1300, 96)]


@pytest.mark.parametrize("T,N,K", LARGE)
@pytest.mark.parametrize("bias", [False, True])
def test_large_batches(cuda_device, T, N, K, bias):
    lin, w, b = make(N, K, T, bias, cuda_device)
    x = acts(T, K)
    y = lin.forward(x.to(cuda_device))
    check(y, x.double(), w, b)
    assert moe.moe_linear_status_sync(lin.handle) == moe.MOE_OK


# either side of the sizes where the GEMM takes over from the small-batch kernels,
# on handles made for just that batch
@pytest.mark.parametrize("T,N,K,q8", [(2, 9380, 5120, False), (8, 9370, 5120, False), (3, 16400, 2080, True), (8, 16100, 2080, True),
                                      (9, 1960, 2048, True), (16, 1940, 2048, True), (9, 7820, 2048, False), (16, 7800, 2048, False)])
def test_path_borders(cuda_device, T, N, K, q8):
    lin, w, b = make(N, K, T, True, cuda_device)
    if q8:
        g = torch.Generator().manual_seed(T + N + K)
        q = torch.randint(-127, 128, (T, K), generator=g).to(torch.int8)
        s = torch.rand(T, K // 32, generator=g) + 0.01
        check(lin.forward_q8(q.to(cuda_device), s.to(cuda_device)), R.q8_values(q, s), w, b, bf16=False)
    else:
        x = acts(T, K)
        check(lin.forward(x.to(cuda_device)), x.double(), w, b)
    assert moe.moe_linear_status_sync(lin.handle) == moe.MOE_OK


# one token, many rows: two row tiles per unit (an odd number of tiles, a last one
# with one row), with x small, large and larger than what they are used for
@pytest.mark.parametrize("N,K", [(4897, 96), (4897, 2080), (4900, 7200), (4897, 8224), (5020, 12288), (4897, 12320), (40000, 512)])
@pytest.mark.parametrize("q8", [False, True])
def test_one_token_many_rows(cuda_device, N, K, q8):
    lin, w, b = make(N, K, 1, True, cuda_device)
    y = torch.full((2, N), 7.0, dtype=torch.bfloat16, device=cuda_device)
    if q8:
        g = torch.Generator().manual_seed(N + K)
        q = torch.randint(-127, 128, (1, K), generator=g).to(torch.int8)
        s = torch.rand(1, K // 32, generator=g) + 0.01
        moe.moe_linear_forward_q8(lin.handle, q.to(cuda_device), s.to(cuda_device), 1, y[:1])
        check(y[:1], R.q8_values(q, s), w, b, bf16=False)
    else:
        x = acts(1, K)
        moe.moe_linear_forward(lin.handle, x.to(cuda_device), 1, y[:1])
        check(y[:1], x.double(), w, b)
    assert (y[1] == 7.0).all()


# one tile per SM and few row blocks: tiles of more than 160 tokens, whole and
# shared by the CTAs of a cluster, with rows and tokens left over
@pytest.mark.parametrize("T,N,K", [(322, 7700, 352), (161, 1600, 6752), (700, 2044, 8192), (213, 1500, 6784)])
def test_large_tiles(cuda_device, T, N, K):
    lin, w, b = make(N, K, T, True, cuda_device)
    x = acts(T, K)
    y = torch.full(((T + 1) * N,), 7.0, dtype=torch.bfloat16, device=cuda_device)
    moe.moe_linear_forward(lin.handle, x.to(cuda_device), T, y[:T * N])
    check(y[:T * N].view(T, N), x.double(), w, b)
    assert (y[T * N:] == 7.0).all()
    assert moe.moe_linear_status_sync(lin.handle) == moe.MOE_OK


@pytest.mark.parametrize("T", [1, 5, 32, 33, 300])
def test_device_and_host_weights_agree(cuda_device, T):
    N, K = 1030, 608
    q, s, _ = R.quantized(3, N, K)
    b = torch.randn(N)
    cfg = dict(in_features=K, out_features=N, max_tokens=T)
    a = moe.MoELinear(cfg, dict(q=q, s=s, bias=b), False)
    qd, sd, bd = q.to(cuda_device), s.to(cuda_device), b.to(cuda_device)
    d = moe.MoELinear(cfg, dict(q=qd, s=sd, bias=bd), True)
    qd.zero_(), sd.zero_(), bd.zero_()  # the handle keeps its own copy
    x = acts(T, K).to(cuda_device)
    assert torch.equal(a.forward(x), d.forward(x))


@pytest.mark.parametrize("T,N,K", [(1, 3000, 2048), (4, 8192, 2048), (32, 515, 4096), (200, 4111, 2080), (1100, 1030, 544)])
def test_repeats_are_bit_identical_and_guards_stay(cuda_device, T, N, K):
    lin, _, _ = make(N, K, T, True, cuda_device)
    x = acts(T, K).to(cuda_device)
    first = lin.forward(x)
    y = torch.full(((T + 1) * N + 8,), 7.0, dtype=torch.bfloat16, device=cuda_device)
    for _ in range(20):
        moe.moe_linear_forward(lin.handle, x, T, y[:T * N])
        assert torch.equal(y[:T * N].view(T, N), first)
    assert (y[T * N:] == 7).all()
    # an output that starts 2 bytes past a 16-byte boundary
    z = torch.full((T * N + 9,), 7.0, dtype=torch.bfloat16, device=cuda_device)
    moe.moe_linear_forward(lin.handle, x, T, z[1:1 + T * N])
    assert torch.equal(z[1:1 + T * N].view(T, N), first) and z[0] == 7 and (z[1 + T * N:] == 7).all()


@pytest.mark.parametrize("T,N,K", [(1, 600, 2048), (8, 600, 96), (20, 600, 544), (300, 600, 544)])
def test_non_finite_tokens_stay_apart(cuda_device, T, N, K):
    lin, w, b = make(N, K, T, True, cuda_device)
    x = acts(T, K)
    bad = [t for t in (0, T // 2, T - 1)][:max(1, min(3, T))]
    x[0, 3] = float("inf")
    x[T // 2, K - 1] = float("nan")
    x[T - 1, K // 2] = float("-inf")
    y = lin.forward(x.to(cuda_device)).cpu()
    assert not torch.isfinite(y[sorted(set(bad))]).any()
    rest = [t for t in range(T) if t not in bad]
    if rest:
        check(y[rest], x[rest].double(), w, b, T)


@pytest.mark.parametrize("T", [1, 33, 600])
def test_extreme_scales(cuda_device, T):
    """Scales from the smallest subnormal to the largest fp16 value, zeros, every code."""
    N, K = 64, 256
    g = torch.Generator().manual_seed(9)
    q = torch.randint(0, 256, (N, K // 2), generator=g).to(torch.uint8)
    s = torch.exp2(torch.randint(-24, 16, (N, K // 32), generator=g).float()).half()
    s[0] = 0
    s[1] = 65504.0
    s[2] = 6e-8
    lin = moe.MoELinear(dict(in_features=K, out_features=N, max_tokens=T), dict(q=q, s=s), False)
    c = torch.stack((q & 15, q >> 4), -1).view(N, K // 32, 32).double() - 8
    w = (c * s.double()[..., None]).view(N, K)
    x = acts(T, K)
    check(lin.forward(x.to(cuda_device)), x.double(), w, None)


@pytest.mark.parametrize("T", [1, 3, 12, 100])
def test_bad_rows_of_weights_stay_apart(cuda_device, T):
    """Negative, infinite and NaN scales: only their own rows feel them."""
    N, K = 200, 288
    q, s, w = R.quantized(11, N, K)
    sign = 1 - 2 * torch.randint(0, 2, s.shape, generator=torch.Generator().manual_seed(3)).half()
    s = s * sign
    w = w * sign.double().repeat_interleave(32, 1)
    x = acts(T, K)
    lin = moe.MoELinear(dict(in_features=K, out_features=N, max_tokens=T), dict(q=q, s=s), False)
    y = lin.forward(x.to(cuda_device))
    check(y, x.double(), w, None)
    s[17, 3], s[150, 0] = float("inf"), float("nan")
    lin = moe.MoELinear(dict(in_features=K, out_features=N, max_tokens=T), dict(q=q, s=s), False)
    z = lin.forward(x.to(cuda_device))
    good = [n for n in range(N) if n not in (17, 150)]
    assert torch.equal(z[:, good], y[:, good])
    assert torch.isnan(z[:, 150]).all() and not torch.isfinite(z[:, 17]).any()


def test_output_past_32_bits(cuda_device):
    """An output of 5.2 GB: the last rows against a call on those tokens alone."""
    T, N, K = 65536, 40003, 64
    lin, w, b = make(N, K, T, True, cuda_device)
    x = torch.randn(T, K, device=cuda_device).bfloat16()
    y = lin.forward(x)
    assert y.numel() * 2 > 1 << 32
    for t in (0, 32768, T - 40):
        assert torch.equal(y[t:t + 40], lin.forward(x[t:t + 40].contiguous()))
    check(y[T - 3:], x[T - 3:].cpu().double(), w, b, T)
    assert moe.moe_linear_status_sync(lin.handle) == moe.MOE_OK


@pytest.mark.parametrize("T", [1, 5, 40])
def test_weights_past_32_bits(cuda_device, T):
    """5.5 GB of packed weights: the last rows against the definition."""
    N, K = 600001, 16384
    g = torch.Generator(device=cuda_device).manual_seed(1)
    q = torch.randint(0, 256, (N, K // 2), generator=g, device=cuda_device, dtype=torch.uint8)
    s = (torch.rand(N, K // 32, generator=g, device=cuda_device) * 0.02).half()
    lin = moe.MoELinear(dict(in_features=K, out_features=N, max_tokens=T), dict(q=q, s=s), True)
    qt, st = q[-50:].cpu(), s[-50:].cpu()
    del q, s
    torch.cuda.empty_cache()
    x = acts(T, K)
    y = lin.forward(x.to(cuda_device))[:, -50:]
    c = torch.stack((qt & 15, qt >> 4), -1).view(50, K // 32, 32).double() - 8
    w = (c * st.double()[..., None]).view(50, K)
    check(y, x.double(), w, None, max(T, 9) if T > 1 else 1)


@pytest.mark.parametrize("Ta,Tb", [(100, 300), (1, 64), (8, 700)])
def test_two_handles_on_two_streams(cuda_device, Ta, Tb):
    a, _, _ = make(1500, 2048, Ta, True, cuda_device)
    b, _, _ = make(2048, 1056, Tb, False, cuda_device, seed=4)
    xa, xb = acts(Ta, 2048).to(cuda_device), acts(Tb, 1056).to(cuda_device)
    ya, yb = a.forward(xa), b.forward(xb)
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    za, zb = (torch.zeros((20,) + tuple(y.shape), dtype=y.dtype, device=cuda_device) for y in (ya, yb))
    torch.cuda.synchronize()
    for i in range(20):
        moe.moe_linear_forward(a.handle, xa, Ta, za[i], sa)
        moe.moe_linear_forward(b.handle, xb, Tb, zb[i], sb)
    torch.cuda.synchronize()
    assert all(torch.equal(z, ya) for z in za) and all(torch.equal(z, yb) for z in zb)
    assert moe.moe_linear_status_sync(a.handle) == moe.MOE_OK == moe.moe_linear_status_sync(b.handle)


def test_profile_names_the_kernels(cuda_device):
    lin, _, _ = make(512, 512, 64, False, cuda_device)
    moe.moe_profile_read()
    moe.moe_profile_enable(True)
    try:
        for T in (1, 8, 64):
            lin.forward(acts(T, 512).to(cuda_device))
        moe.add_rmsnorm(acts(3, 512).to(cuda_device))
    finally:
        moe.moe_profile_enable(False)
    got = moe.moe_profile_read()
    assert {k: v[0] for k, v in got.items()} == {"linear_dot": 1, "linear_small": 1, "linear_prep": 1, "linear_gemm": 1,
                                                 "add_rmsnorm": 1}


def test_refusals(cuda_device):
    N, K, T = 64, 128, 40
    lin, _, _ = make(N, K, T, False, cuda_device)
    x = acts(T, K).to(cuda_device)
    y = torch.empty(T, N, dtype=torch.bfloat16, device=cuda_device)
    big = torch.empty(T * K + 8, dtype=torch.bfloat16, device=cuda_device)
    for args, status in (((x, 0, y), moe.MOE_ERR_CAPACITY), ((x, T + 1, y), moe.MOE_ERR_CAPACITY),
                         ((None, T, y), moe.MOE_ERR_INVALID), ((x, T, None), moe.MOE_ERR_INVALID),
                         ((x.cpu(), T, y), moe.MOE_ERR_INVALID), ((x, T, y.cpu()), moe.MOE_ERR_INVALID),
                         ((big[1:1 + T * K], T, y), moe.MOE_ERR_INVALID), ((x, T, x), moe.MOE_ERR_INVALID)):
        with pytest.raises(moe.MoeError) as ei:
            moe.moe_linear_forward(lin.handle, *args)
        assert ei.value.status == status
    q = torch.zeros(T, K, dtype=torch.int8, device=cuda_device)
    s = torch.zeros(T, K // 32, device=cuda_device)
    with pytest.raises(moe.MoeError) as ei:
        moe.moe_linear_forward_q8(lin.handle, q, s, T + 1, y)
    assert ei.value.status == moe.MOE_ERR_CAPACITY
    for args in ((None, s, 4, y), (q, None, 4, y), (q, s, 4, None), (q.cpu(), s, 4, y), (q, s, 4, q)):
        with pytest.raises(moe.MoeError) as ei:
            moe.moe_linear_forward_q8(lin.handle, *args)
        assert ei.value.status == moe.MOE_ERR_INVALID
    with pytest.raises(ValueError):
        lin.forward(x.float())
    with pytest.raises(ValueError):
        lin.forward(x[:, :64])
    with pytest.raises(ValueError):
        lin.forward_q8(q, s[:3])


def test_create_refuses_what_the_gpu_cannot_read(cuda_device):
    N, K = 32, 64
    q, s, _ = R.quantized(0, N, K)
    cfg = dict(in_features=K, out_features=N, max_tokens=1)
    qd, sd = q.to(cuda_device), s.to(cuda_device)
    odd = torch.zeros(2 * s.numel() + 2, dtype=torch.uint8, device=cuda_device)[1:1 + 2 * s.numel()]
    for w in (dict(q=q, s=sd), dict(q=qd, s=s), dict(q=qd, s=sd, bias=torch.zeros(N)), dict(q=qd, s=odd)):
        with pytest.raises(moe.MoeError) as ei:
            moe.moe_linear_create(cfg, w, True)
        assert ei.value.status == moe.MOE_ERR_INVALID


@pytest.mark.parametrize("T", [1, 3, 8, 12, 40])
def test_q8_special_values(cuda_device, T):
    """Zero and NaN scales, the codes' ends; other tokens stay as they are."""
    N, K = 100, 160
    lin, w, b = make(N, K, T, True, cuda_device)
    g = torch.Generator().manual_seed(T)
    q = torch.randint(-128, 128, (T, K), generator=g).to(torch.int8)
    q[:, 0], q[:, 1] = -128, 127
    s = torch.rand(T, K // 32, generator=g) + 0.01
    s[:, 1] = 0
    y = lin.forward_q8(q.to(cuda_device), s.to(cuda_device))
    check(y, R.q8_values(q, s), w, b, bf16=False)
    s[T - 1, 2] = float("nan")
    z = lin.forward_q8(q.to(cuda_device), s.to(cuda_device))
    assert torch.isnan(z[T - 1]).all() and torch.equal(z[:T - 1], y[:T - 1])


@pytest.mark.parametrize("T,N,K", [(1, 300, 2048), (2, 300, 2048), (8, 300, 2048), (12, 300, 2048), (40, 300, 2048)])
@pytest.mark.parametrize("size", [1e-37, 1e-30, 1e30])
def test_tiny_and_huge_activations(cuda_device, T, N, K, size):
    lin, w, _ = make(N, K, T, False, cuda_device)
    x = (acts(T, K).float() * size).bfloat16()
    y = lin.forward(x.to(cuda_device))
    # at 1e-37 the result nears fp32's smallest normal number: 2^-126 K absolute
    y64 = R.product(x.double(), w)
    bound = R.product_bound(x.double(), w, y64, None, T) + K * 2.0 ** -126
    assert ((y.double().cpu() - y64).abs() <= bound).all()


@pytest.mark.parametrize("T", [1, 40])
def test_captured_after_a_join_of_streams(cuda_device, T):
    """The input comes from a kernel of another stream, inside one capture."""
    N, K = 2048, 2048
    lin, _, _ = make(N, K, T, False, cuda_device)
    src = acts(T, K).to(cuda_device)
    x, y, other = torch.zeros_like(src), torch.zeros(T, N, dtype=torch.bfloat16, device=cuda_device), torch.zeros(1 << 22, device=cuda_device)
    side = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        main = torch.cuda.current_stream()
        side.wait_stream(main)
        with torch.cuda.stream(side):
            for _ in range(8):
                other.add_(1)
            x.copy_(src)
            x.mul_(2)
        main.wait_stream(side)
        moe.moe_linear_forward(lin.handle, x, T, y)
    want = lin.forward(src * 2)
    for _ in range(5):
        x.zero_()
        y.zero_()
        g.replay()
        assert torch.equal(y, want)
    # the same without a capture
    for _ in range(5):
        x.zero_()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            for _ in range(8):
                other.add_(1)
            torch.mul(src, 2, out=x)
        torch.cuda.current_stream().wait_stream(side)
        moe.moe_linear_forward(lin.handle, x, T, y)
        assert torch.equal(y, want)


@pytest.mark.parametrize("T,N,K", [(100, 4111, 2080), (300, 256, 2048), (2000, 3000, 256)])
def test_bounded_waits_report_a_timeout(cuda_device, monkeypatch, T, N, K):
    """A barrier that one arrival never reaches: the waits run out, the call
    reports MOE_ERR_TIMEOUT and the next one is right again."""
    lin, w, b = make(N, K, T, True, cuda_device)
    x = acts(T, K)
    xd = x.to(cuda_device)
    monkeypatch.setenv("MOE_DEBUG_UNREACHABLE_BARRIER", "1")
    monkeypatch.setenv("MOE_WAIT_TIMEOUT_US", "20000")
    lin.forward(xd)
    assert moe.moe_linear_status_sync(lin.handle) == moe.MOE_ERR_TIMEOUT
    monkeypatch.delenv("MOE_DEBUG_UNREACHABLE_BARRIER")
    monkeypatch.delenv("MOE_WAIT_TIMEOUT_US")
    assert moe.moe_linear_status_sync(lin.handle) == moe.MOE_OK  # cleared
    check(lin.forward(xd), x.double(), w, b)
    assert moe.moe_linear_status_sync(lin.handle) == moe.MOE_OK


@pytest.mark.parametrize("T,N,K", [(32, 1030, 4096), (40, 1000, 512), (700, 2044, 8192)])
def test_bounded_waits_in_clusters(cuda_device, monkeypatch, T, N, K):
    """The same where the CTAs of a cluster share a tile: all of them end."""
    test_bounded_waits_report_a_timeout(cuda_device, monkeypatch, T, N, K)


@pytest.mark.parametrize("T,N,K", [(20, 500, 512), (64, 2000, 256), (33, 900, 1056), (50, 300, 768)])
def test_few_stages_back_to_back(cuda_device, T, N, K):
    """More groups of producers than stages; every call reads the output of the
    one before it and overwrites what the one before that read."""
    a, wa, ba = make(N, K, T, True, cuda_device)
    b, wb, bb = make(K, N // 32 * 32, T, True, cuda_device, seed=1)
    x0 = acts(T, K).to(cuda_device)
    x = x0.clone()
    y = torch.empty(T, N, dtype=torch.bfloat16, device=cuda_device)
    cut = torch.empty(T, N // 32 * 32, dtype=torch.bfloat16, device=cuda_device)
    want, w = [], x0
    for _ in range(3):
        w = b.forward(a.forward(w)[:, :cut.shape[1]].contiguous())
        torch.cuda.synchronize()
        want.append(w)
    for r in range(20):
        x.copy_(x0)
        for i in range(3):
            moe.moe_linear_forward(a.handle, x, T, y)
            cut.copy_(y[:, :cut.shape[1]])
            moe.moe_linear_forward(b.handle, cut, T, x)
            assert r < 19 or torch.equal(x, want[i])
    check(y, want[1].double().cpu(), wa, ba)


@pytest.mark.parametrize("T", [1, 4, 32, 200])
def test_side_stream_and_graph(cuda_device, T):
    N, K = 1536, 2048
    lin, _, _ = make(N, K, T, True, cuda_device)
    back, _, _ = make(K, N, T, False, cuda_device, seed=1)
    x = acts(T, K).to(cuda_device)
    y0 = lin.forward(x)
    z0 = back.forward(y0)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    y = torch.zeros_like(y0)
    moe.moe_linear_forward(lin.handle, x, T, y, st)
    st.synchronize()
    assert torch.equal(y, y0)
    x1, z = x.clone(), torch.zeros_like(z0)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        moe.moe_linear_forward(lin.handle, x1, T, y)
        moe.moe_linear_forward(back.handle, y, T, z)
    for k in range(3):
        x1.copy_(x if k != 1 else -x)
        g.replay()
        assert torch.equal(z, z0 if k != 1 else back.forward(lin.forward(-x)))
