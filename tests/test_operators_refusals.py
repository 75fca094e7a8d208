"""Refusals of the norm and projection entry points that need no GPU: bad
sizes, missing pointers, host memory."""
import ctypes

import pytest

import quantized_expert_ffn_softmax_gb300 as moe
from quantized_expert_ffn_softmax_gb300 import _build


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return moe.lib()


@pytest.mark.parametrize("bad", [dict(in_features=0), dict(in_features=48), dict(in_features=-32),
                                 dict(in_features=32800), dict(out_features=0),
                                 dict(out_features=(1 << 20) + 1), dict(max_tokens=0),
                                 dict(max_tokens=65537)])
def test_linear_create_rejects_bad_configs(lib, bad):
    cfg = dict(in_features=256, out_features=100, max_tokens=8)
    cfg.update(bad)
    with pytest.raises(moe.MoeError) as ei:
        moe.moe_linear_create(cfg, dict(q=16, s=16), False)
    assert ei.value.status == moe.MOE_ERR_INVALID
    assert next(iter(bad)) in moe.moe_last_error()


@pytest.mark.parametrize("missing", ["q", "s"])
def test_linear_create_rejects_missing_weights(lib, missing):
    w = dict(q=16, s=16)
    del w[missing]
    with pytest.raises(moe.MoeError) as ei:
        moe.moe_linear_create(dict(in_features=64, out_features=8, max_tokens=1), w, True)
    assert ei.value.status == moe.MOE_ERR_INVALID
    assert "NULL" in moe.moe_last_error()


def test_linear_create_reports_a_failed_allocation(lib, monkeypatch):
    monkeypatch.setenv("MOE_FAULT_ALLOC", "1")
    out = ctypes.c_void_p(1)
    cfg = moe.moe_linear_config(64, 8, 1)
    w = moe.moe_linear_weights(16, 16, None)
    assert lib.moe_linear_create(ctypes.byref(cfg), ctypes.byref(w), 0, ctypes.byref(out)) == moe.MOE_ERR_OOM
    assert out.value is None


def test_calls_reject_null_handles(lib):
    assert lib.moe_linear_create(None, None, 0, None) == moe.MOE_ERR_INVALID
    out = ctypes.c_void_p(1)
    assert lib.moe_linear_create(None, None, 0, ctypes.byref(out)) == moe.MOE_ERR_INVALID
    assert out.value is None
    assert lib.moe_linear_forward(None, None, 1, None, None) == moe.MOE_ERR_INVALID
    assert lib.moe_linear_forward_q8(None, None, None, 1, None, None) == moe.MOE_ERR_INVALID
    assert lib.moe_linear_status_sync(None, None) == moe.MOE_ERR_INVALID
    lib.moe_linear_destroy(None)


@pytest.mark.parametrize("kw,status", [(dict(n_tokens=0), moe.MOE_ERR_CAPACITY),
                                       (dict(n_tokens=65537), moe.MOE_ERR_CAPACITY),
                                       (dict(hidden=0), moe.MOE_ERR_INVALID),
                                       (dict(hidden=40), moe.MOE_ERR_INVALID),
                                       (dict(hidden=32800), moe.MOE_ERR_INVALID),
                                       (dict(eps=-1.0), moe.MOE_ERR_INVALID),
                                       (dict(eps=float("nan")), moe.MOE_ERR_INVALID),
                                       (dict(eps=float("inf")), moe.MOE_ERR_INVALID)])
def test_norm_rejects_bad_sizes(lib, kw, status):
    a = dict(eps=1e-6, n_tokens=1, hidden=64)
    a.update(kw)
    for f, outs in ((moe.moe_add_rmsnorm, (16, 16)), (moe.moe_add_rmsnorm_q8, (16, 16, 16))):
        with pytest.raises(moe.MoeError) as ei:
            f(16, None, None, a["eps"], a["n_tokens"], a["hidden"], *outs, stream=0)
        assert ei.value.status == status


def test_new_symbols_are_exported(lib):
    raw = ctypes.CDLL(moe.LIB_PATH)
    for n in ("moe_add_rmsnorm", "moe_add_rmsnorm_q8", "moe_linear_create", "moe_linear_destroy",
              "moe_linear_forward", "moe_linear_forward_q8", "moe_linear_status_sync"):
        assert hasattr(raw, n), n
