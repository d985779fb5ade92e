"""CPU tests of the few-token layer's host side: workspace, refusals before anything is
enqueued (no GPU is touched)."""
import ctypes

import pytest

from top_routing_expert_fp32_b200 import configs


@pytest.fixture(scope="module")
def abi():
    from top_routing_expert_fp32_b200 import build
    build.build()
    from top_routing_expert_fp32_b200 import abi as a
    return a


def _p(abi, **kw):
    base = dict(N=4, D=64, F=128, E=4, k=2, dtype=configs.DTYPE_BF16, activation=0, renormalize=1)
    return abi.problem(configs.MoEConfig("few", **{**base, **kw}))


def _call(abi, p, ws_bytes=None, w8=False, **over):
    names = (["X", "W_r", "bias", "W1q", "S1", "W2q", "S2", "W3q", "S3", "out"] if w8 else
             ["X", "W_r", "bias", "W1", "W2", "W3", "out"])
    args = [over.get(n, 4096) for n in names] + [None] * 8
    need = abi.workspace_size(p) if ws_bytes is None else ws_bytes
    fn = abi.lib.moe_forward_few_w8 if w8 else abi.lib.moe_forward_few
    return fn(ctypes.byref(p), *args, over.get("ws", 4096), need, None)


def test_workspace_holds_the_intermediates(abi):
    assert abi.FEW_MAX_TOKENS == 64
    # H of 64 x 2 records in two bf16 terms.
    assert abi.workspace_size(_p(abi, N=64)) >= 64 * 2 * 128 * 4


@pytest.mark.parametrize("kw", [dict(), dict(dtype=configs.DTYPE_F32), dict(E=64, k=8),
                                dict(D=4096, F=14336, E=8)])
def test_a_workspace_serves_every_smaller_batch(abi, kw):
    lib, b = abi.lib, ctypes.c_size_t()
    for size in (lib.moe_workspace_size, lib.moe_workspace_size_host):
        sizes = []
        for n in (0, 1, 2, 7, 8, 9, 16, 17, 33, 63, 64, 65, 66, 100, 128, 500, 4096):
            p = _p(abi, N=n, **kw)
            assert size(ctypes.byref(p), ctypes.byref(b)) == 0
            sizes.append(b.value)
        assert sizes == sorted(sizes)


@pytest.mark.parametrize("w8", [False, True])
def test_refusals(abi, w8):
    p = _p(abi)
    need = abi.workspace_size(p)
    assert _call(abi, p, ws_bytes=need - 1, w8=w8) == abi.MOE_ERR_INVALID_ARG
    assert b"too small" in abi.lib.moe_last_error()
    for name in (["W1q", "S3", "W2q"] if w8 else ["W1", "W2", "W3"]) + ["X", "W_r", "out"]:
        assert _call(abi, p, w8=w8, **{name: None}) == abi.MOE_ERR_INVALID_ARG
        assert name.encode() in abi.lib.moe_last_error()
        assert _call(abi, p, w8=w8, **{name: 4104}) == abi.MOE_ERR_INVALID_ARG
        assert b"aligned" in abi.lib.moe_last_error()
    assert _call(abi, p, w8=w8, ws=None) == abi.MOE_ERR_INVALID_ARG
    big = _p(abi, N=65)
    assert _call(abi, big, w8=w8) == abi.MOE_ERR_UNSUPPORTED
    assert b"64 tokens" in abi.lib.moe_last_error()
    noisy = _p(abi, routing_mode=configs.ROUTE_NOISY_TOPK)
    assert _call(abi, noisy, w8=w8) == abi.MOE_ERR_INVALID_ARG


def test_w8_shape_rules(abi):
    assert _call(abi, _p(abi, D=72), w8=True) == abi.MOE_ERR_UNSUPPORTED
    assert _call(abi, _p(abi, dtype=configs.DTYPE_F32), w8=True) == abi.MOE_ERR_UNSUPPORTED
