"""CPU tests: which workspace sizes the entry points accept (no GPU is touched: a call whose
workspace is large enough is refused for its missing X)."""
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
    base = dict(N=512, D=256, F=512, E=8, k=2, dtype=configs.DTYPE_BF16, activation=0,
                renormalize=1)
    return abi.problem(configs.MoEConfig("ws", **{**base, **kw}))


def _calls(abi, p, ws_bytes):
    """(name, status, message) of entry points called without X."""
    lib, r = abi.lib, ctypes.byref(p)
    a = 4096
    for name, args in (
            ("moe_route", [None, a, None, None, a, a, None]),
            ("moe_forward", [None, a, None, a, a, a, a] + [None] * 8),
            ("moe_forward_host", [None, a, None, a, a, a, a])):
        status = getattr(lib, name)(r, *args, a, ws_bytes, None)
        yield name, status, lib.moe_last_error()


# Sizes that the layer's own regions take (router sums, counters, routing, X_perm, H, Y).
@pytest.mark.parametrize("kw,own", [
    (dict(), 2158336), (dict(N=65, D=64, F=64), None), (dict(N=4096, D=64, F=64, E=64, k=8), None),
    (dict(N=200, D=64, F=128, E=4, dtype=configs.DTYPE_F32), None)])
def test_large_batches_need_no_room_for_the_few_token_form(abi, kw, own):
    p = _p(abi, **kw)
    es = 4 if p.dtype == configs.DTYPE_F32 else 2
    R = p.N * p.k
    rows = R * (2 * p.D + p.F) * es
    if own is None:  # routing: 17 bytes a record; the rest: counters and partial sums, below 1 MB
        own = rows + 17 * R + (1 << 20)
    for name, status, message in _calls(abi, p, own + 4 * p.N * p.D * es):
        assert status == abi.MOE_ERR_INVALID_ARG
        assert b"too small" not in message and b"X" in message, (name, message)
    for name, status, message in _calls(abi, p, rows):
        assert status == abi.MOE_ERR_INVALID_ARG and b"too small" in message, name
    # The size functions' answer serves fewer tokens too, the few-token form among them.
    few = _p(abi, **{**kw, "N": 64})
    for host in (False, True):
        assert abi.workspace_size(p, host) >= abi.workspace_size(few, host)
    assert abi.workspace_size(p) > own
