"""MOE_DROP_RENORM_KEPT where a token keeps only experts whose gates are 0 in fp32: the kept slots
share the whole weight equally, in moe_combine, moe_forward and moe_forward_few.

The router's weights pick the experts by hand: all tokens choose expert 0, whose capacity the first
half takes; the others keep what they chose next, whose logits lie `gap` below the largest."""
import numpy as np
import pytest
import torch

import oracle
from top_routing_expert_fp32_b200 import configs, inputs
from gpu_helpers import TOL_BF16, normwise_rel_err, np_host, oracle_dtype, to_f64, tol

pytestmark = pytest.mark.gpu

BF16, F32 = configs.DTYPE_BF16, configs.DTYPE_F32


@pytest.fixture(scope="module")
def abi():
    from top_routing_expert_fp32_b200 import abi as a
    return a


def _case(dtype, k, gap, renorm, N=8):
    E = 4 if k == 2 else 5
    cfg = configs.MoEConfig("gates", N=N, D=64, F=128, E=E, k=k, dtype=dtype, activation=0,
                            renormalize=renorm, capacity_factor=0.5 * E / k,  # N / 2 rows
                            drop_policy=configs.DROP_RENORM_KEPT)
    inp = inputs.make_inputs(cfg, "cuda")
    W_r = torch.zeros((cfg.D, E), device="cuda")
    sign = torch.where(torch.arange(N, device="cuda") % 2 == 0, 1.0, -1.0).to(inp.X.dtype)
    inp.X[:, 0] = sign
    # Even tokens take experts 1 .. k-1 next, odd ones the experts from the other end.
    W_r[0, 1:] = torch.linspace(1.0, -1.0, E - 1, device="cuda")
    bias = torch.full((E,), -float(gap), device="cuda")
    bias[0] = 0.0
    return cfg, inputs.MoEInputs(inp.X, W_r, bias, inp.W1, inp.W2, inp.W3)


def _expected(cfg, inp, idx, dropped):
    """Expected rows: the kept experts' mean where the first choice was dropped (their gates are
    all 0), expert 0's output where it was kept (gate 1)."""
    N, k = idx.shape
    t = np.repeat(np.arange(N, dtype=np.int32), k)
    Y = oracle.expert_ffn(t, idx.reshape(-1).astype(np.int32), np_host(inp.X), np_host(inp.W1),
                          np_host(inp.W2), np_host(inp.W3), oracle_dtype(cfg), cfg.activation)
    Y = Y.reshape(N, k, -1)
    ref = np.zeros((N, cfg.D))
    for i in range(N):
        keep = dropped[i] == 0
        ref[i] = Y[i, keep].mean(0) if dropped[i, 0] else Y[i, 0]
    return ref


def _check(cfg, out, ref, few):
    # moe_forward: the suite's bound on a row (H, Y and the output are rounded). moe_forward_few:
    # one rounding, of half a step, and 1e-4 (fp32: 1e-5) of the row's largest value for the two
    # terms of H and the fp32 sums.
    got = to_f64(out)
    assert np.isfinite(got).all()
    if not few:
        assert normwise_rel_err(got, ref).max() <= tol(cfg)
        return
    half, sums = (2.0 ** -8, 1e-4) if cfg.dtype == BF16 else (2.0 ** -24, 1e-5)
    bound = half * np.abs(ref) + sums * np.abs(ref).max(axis=1, keepdims=True)
    assert (np.abs(got - ref) <= bound).all()


CASES = [(BF16, 2, 200.0, 1), (BF16, 2, 1e4, 0), (F32, 2, 1e4, 1), (BF16, 3, 1e4, 1),
         (F32, 3, 300.0, 0)]


@pytest.mark.parametrize("dtype,k,gap,renorm", CASES)
@pytest.mark.parametrize("few", [True, False], ids=["few", "forward"])
def test_kept_gates_that_underflow_share_the_weight(abi, dtype, k, gap, renorm, few):
    cfg, inp = _case(dtype, k, gap, renorm)
    p = abi.problem(cfg)
    ws = abi.workspace(p)
    idx = torch.empty((cfg.N, k), dtype=torch.int32, device="cuda")
    gate = torch.empty((cfg.N, k), device="cuda")
    dropped = torch.empty((cfg.N, k), dtype=torch.uint8, device="cuda")
    out = torch.empty_like(inp.X)
    call = abi.forward_few if few else abi.forward
    call(p, inp.X, inp.W_r, inp.bias, inp.W1, inp.W2, inp.W3, out, ws, topk_idx=idx,
         topk_gate=gate, dropped=dropped)
    torch.cuda.synchronize()
    assert abi.device_error(ws) == 0
    idx, gate, dropped = (v.cpu().numpy() for v in (idx, gate, dropped))
    assert (idx[:, 0] == 0).all() and (gate[:, 0] == 1).all() and (gate[:, 1:] == 0).all()
    half = cfg.N // 2
    assert (dropped[:half, 0] == 0).all() and (dropped[half:, 0] == 1).all()
    assert (dropped[half:, 1:] == 0).any(1).all()
    # (The first half's rows, where other slots may be dropped, have gates 1, 0, ...)
    _check(cfg, out, _expected(cfg, inp, idx, dropped), few)


def test_kept_gates_that_underflow_8_bit(abi):
    cfg, inp = _case(BF16, 2, 1e4, 1)
    w8 = inputs.make_w8_weights(cfg, "cuda")
    p = abi.problem(cfg)
    ws = abi.workspace(p)
    outs = [torch.empty_like(inp.X) for _ in range(2)]
    abi.forward_few_w8(p, inp.X, inp.W_r, inp.bias, w8, outs[0], ws)
    abi.forward_w8(p, inp.X, inp.W_r, inp.bias, w8, outs[1], ws)
    torch.cuda.synchronize()
    a, b = to_f64(outs[0]), to_f64(outs[1])
    assert np.isfinite(a).all() and np.isfinite(b).all() and (np.abs(b).max(1) > 0).all()
    assert normwise_rel_err(a, b).max() <= TOL_BF16


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_combine_of_zero_gates(abi, dtype):
    # moe_combine alone: token 0 keeps two of three slots, both with gate 0; token 1 one of them
    # with the smallest fp32 number; token 2 keeps all three (no renormalisation: zeros); token 3
    # none.
    N, k, E, D = 4, 3, 3, 64
    cfg = configs.MoEConfig("c", N=N, D=D, F=64, E=E, k=k, dtype=dtype, activation=0,
                            renormalize=0, capacity_factor=0.75,
                            drop_policy=configs.DROP_RENORM_KEPT)
    t = torch.bfloat16 if dtype == BF16 else torch.float32
    idx = torch.tensor([[0, 1, 2]] * N, dtype=torch.int32, device="cuda")
    dropped = torch.tensor([[1, 0, 0], [1, 1, 0], [0, 0, 0], [1, 1, 1]], dtype=torch.uint8,
                           device="cuda")
    gate = torch.zeros((N, k), device="cuda")
    gate[1, 2] = 2.0 ** -149
    pos = torch.zeros((N, k), dtype=torch.int32, device="cuda")
    counts = [0] * E
    for i in range(N):
        for j in range(k):
            if not dropped[i, j]:
                pos[i, j] = counts[j]
                counts[j] += 1
    offsets = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32,
                           device="cuda")
    Y = torch.randn((sum(counts), D), device="cuda").to(t)
    out = torch.full((N, D), 7.0, dtype=t, device="cuda")
    abi.combine(abi.problem(cfg), Y, idx, gate, offsets, pos, dropped, out)
    torch.cuda.synchronize()
    y = lambda i, j: Y[int(offsets[j]) + int(pos[i, j])].float()
    assert torch.equal(out[0], (0.5 * y(0, 1) + 0.5 * y(0, 2)).to(t))  # exact halves
    assert torch.equal(out[1], y(1, 2).to(t))
    assert (out[2] == 0).all() and (out[3] == 0).all()
