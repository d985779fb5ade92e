"""CPU tests of moe_lora_forward's host side: workspace sizes and refusals before anything is
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
    base = dict(M=4, K=64, N=128, adapters=2, rank=16, dtype=configs.DTYPE_BF16)
    return abi.lora_problem(**{**base, **kw})


def _size(abi, p):
    b = ctypes.c_size_t()
    return abi.lib.moe_lora_workspace_size(ctypes.byref(p), ctypes.byref(b)), b.value


def _call(abi, p, ws_bytes=1 << 30, **over):
    names = ["X", "W", "A", "B", "adapter", "scale", "addend", "Y"]
    args = [over.get(n, 4096) for n in names]
    return abi.lib.moe_lora_forward(ctypes.byref(p), *args, over.get("ws", 4096), ws_bytes, None)


@pytest.mark.parametrize("kw,status", [
    (dict(M=-1), 1), (dict(K=0), 1), (dict(N=0), 1), (dict(adapters=0), 1), (dict(rank=0), 1),
    (dict(dtype=7), 1), (dict(rank=136), 2), (dict(rank=12), 2), (dict(K=68), 2), (dict(N=4), 2),
    (dict(K=66, dtype=configs.DTYPE_F32), 2), (dict(rank=2, dtype=configs.DTYPE_F32), 2),
    (dict(M=(1 << 30) + 1), 2), (dict(K=(1 << 24) + 8), 2)])
def test_problem_refusals(abi, kw, status):
    p = _p(abi, **kw)
    assert _size(abi, p)[0] == status
    assert _call(abi, p) == status


def test_reserved_and_null(abi):
    p = _p(abi)
    p.reserved = 1
    assert _size(abi, p)[0] == abi.MOE_ERR_INVALID_ARG
    assert abi.lib.moe_lora_workspace_size(None, None) == abi.MOE_ERR_INVALID_ARG
    assert abi.lib.moe_lora_workspace_size(ctypes.byref(_p(abi)), None) == abi.MOE_ERR_INVALID_ARG


@pytest.mark.parametrize("M", [4, 300])
def test_call_refusals(abi, M):
    p = _p(abi, M=M)
    st, need = _size(abi, p)
    assert st == 0
    assert _call(abi, p, ws_bytes=need - 1) == abi.MOE_ERR_INVALID_ARG
    assert b"too small" in abi.lib.moe_last_error()
    for name in ("X", "W", "A", "B", "adapter", "Y", "ws"):
        assert _call(abi, p, **{name: None}) == abi.MOE_ERR_INVALID_ARG, name
        assert name.encode() in abi.lib.moe_last_error()
    for name, ptr in (("X", 4104), ("Y", 4104), ("addend", 4104), ("adapter", 4098),
                      ("scale", 4098), ("ws", 4112)):
        assert _call(abi, p, **{name: ptr}) == abi.MOE_ERR_INVALID_ARG, name
        assert b"aligned" in abi.lib.moe_last_error()


def test_no_rows_is_a_no_op(abi):
    p = _p(abi, M=0)
    assert _size(abi, p) == (0, 256)
    assert _call(abi, p, X=None, Y=None) == 0


def test_workspace_grows_with_the_rows(abi):
    for dtype in (configs.DTYPE_BF16, configs.DTYPE_F32):
        sizes = [_size(abi, _p(abi, M=m, dtype=dtype, K=4096))[1] for m in (65, 128, 700, 4096)]
        assert sizes == sorted(sizes)


@pytest.mark.parametrize("kw", [dict(), dict(dtype=configs.DTYPE_F32), dict(K=14336, rank=128),
                                dict(N=4096)])
def test_a_workspace_serves_every_smaller_batch(abi, kw):
    sizes = [_size(abi, _p(abi, M=m, **kw))[1]
             for m in (0, 1, 3, 4, 5, 8, 9, 31, 32, 37, 63, 64, 65, 127, 128, 129, 256, 511, 512,
                       1000, 2304, 2305, 2560, 4096, 18432, 18433, 20000)]
    assert sizes == sorted(sizes)
