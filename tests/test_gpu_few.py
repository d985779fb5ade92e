"""GPU parity of the few-token layer (moe_forward_few, moe_forward_few_w8) against the oracle's
fp64 layer, its refusals, and its behaviour under graphs, streams and used workspaces.

Tolerances. The output is rounded once: at most half a step, 2^-8 (bf16) or 2^-24 (fp32) of the
value. Before that come fp32 sums of n <= 2^15 terms, whose errors grow like sqrt(n) 2^-24 of the
terms' 2-norm when they are independent and at most a few times that on the tensor cores, which
truncate: sqrt(2^15) * 2^-23 = 2.2e-5 per product, two products in a row; the second bf16 term
of H leaves 2^-17 = 7.6e-6 and the activation 7.6e-6 (gelu_erf's far tail). 1e-4 of the row's
largest value covers their sum. The fp32 layer's products are shorter here (n <= 512): 1e-5."""
import numpy as np
import pytest
import torch

import oracle
from top_routing_expert_fp32_b200 import configs, inputs
from gpu_helpers import (alloc_dispatch_out, alloc_route_out, check_routing, np_host,
                         oracle_dtype, to_f64)

pytestmark = pytest.mark.gpu

BF16, F32 = configs.DTYPE_BF16, configs.DTYPE_F32


@pytest.fixture(scope="module")
def abi():
    from top_routing_expert_fp32_b200 import abi as a
    return a


def _cfg(name, N, D, F, E, k, dtype=BF16, act=configs.ACT_SILU, renorm=1, **kw):
    return configs.MoEConfig(name, N=N, D=D, F=F, E=E, k=k, dtype=dtype, activation=act,
                             renormalize=renorm, **kw)


def _run(abi, cfg, inp, w8=None, ws=None, exports=True):
    p = abi.problem(cfg)
    ws = abi.workspace(p) if ws is None else ws
    r = alloc_route_out(cfg.N, cfg.E, cfg.k)
    d = alloc_dispatch_out(cfg.N, cfg.E, cfg.k)
    # One row behind the last token, which must stay as it is.
    buf = torch.full((cfg.N + 1, cfg.D), 7.5, dtype=inp.X.dtype, device="cuda")
    out = buf[:cfg.N]
    more = dict(logits=r["logits"], topk_idx=r["idx"], topk_gate=r["gate"], load=d["load"],
                offsets=d["offsets"], pos=d["pos"], dropped=d["dropped"],
                prob_colsum=r["colsum"]) if exports else {}
    if w8 is None:
        abi.forward_few(p, inp.X, inp.W_r, inp.bias, inp.W1, inp.W2, inp.W3, out, ws, **more)
    else:
        abi.forward_few_w8(p, inp.X, inp.W_r, inp.bias, w8, out, ws, **more)
    torch.cuda.synchronize()
    assert abi.device_error(ws) == 0
    assert (buf[cfg.N] == 7.5).all()
    assert ws[:256].view(torch.int32).abs().sum().item() == 0  # header words at rest
    return out, {key: v.cpu().numpy() for key, v in {**r, **d}.items()}


def _reference(cfg, inp, ex, w8=None):
    """fp64 output from the GPU's own routing (checked on its own by check_routing)."""
    dg, gate, _ = check_routing(cfg, inp, ex)
    keep = dg["dropped"] == 0
    rec_t, slot = np.nonzero(keep)
    rec_e = ex["idx"][rec_t, slot].astype(np.int32)
    rec_t = rec_t.astype(np.int32)
    ref = np.zeros((cfg.N, cfg.D))
    if len(rec_t) == 0:
        return ref, dg
    if w8 is None:
        Y = oracle.expert_ffn(rec_t, rec_e, np_host(inp.X), np_host(inp.W1), np_host(inp.W2),
                              np_host(inp.W3), oracle_dtype(cfg), cfg.activation)
    else:
        Y = oracle.expert_ffn_w8(rec_t, rec_e, np_host(inp.X), oracle.BF16,
                                 *(getattr(w8, n).cpu().numpy() for n in
                                   ("W1q", "S1", "W2q", "S2", "W3q", "S3")), cfg.activation)
    g = gate.copy()
    if cfg.drop_policy == configs.DROP_RENORM_KEPT:
        part = keep.any(1) & ~keep.all(1)
        g[part] = gate[part] / (gate * keep).sum(1)[part, None]
    for t, j, y in zip(rec_t, slot, Y):
        ref[t] += g[t, j] * y
    return ref, dg


def _check(cfg, out, ref):
    got = to_f64(out)
    half, sums = (2.0 ** -8, 1e-4) if cfg.dtype == BF16 else (2.0 ** -24, 1e-5)
    bound = half * np.abs(ref) + sums * np.abs(ref).max(axis=1, keepdims=True)
    assert np.isfinite(got).all()
    worst = np.max(np.abs(got - ref) - bound)
    assert worst <= 0, f"over the bound by {worst:.3g} (largest |ref| {np.abs(ref).max():.3g})"


CASES = [
    _cfg("one_by_one", 1, 8, 8, 1, 1),
    _cfg("one_token", 1, 64, 128, 4, 2),
    _cfg("wide_k", 1, 4096, 256, 8, 2, act=configs.ACT_GELU_ERF, renorm=0),
    _cfg("wide_f", 2, 256, 8192, 3, 2),
    _cfg("odd_small", 3, 72, 136, 5, 3, act=configs.ACT_GELU_ERF, renorm=0),
    _cfg("half_step_tail", 8, 104, 200, 6, 2, act=configs.ACT_GELU_TANH),
    _cfg("nine_tokens_k8", 9, 200, 328, 64, 8, router_bias_var=1.0),
    _cfg("drops_token_major", 17, 1000, 2728, 13, 3, act=configs.ACT_GELU_TANH,
         capacity_factor=1.0, router_bias_var=1.0, capacity_order=configs.ORDER_TOKEN_MAJOR,
         drop_policy=configs.DROP_RENORM_KEPT),
    _cfg("drops_slot_major", 33, 136, 72, 5, 2, capacity_factor=0.7, router_bias_var=2.0,
         drop_policy=configs.DROP_RENORM_KEPT),
    _cfg("most_dropped", 64, 128, 64, 2, 1, capacity_factor=0.1),
    _cfg("min_capacity", 40, 64, 64, 16, 2, capacity_factor=0.2, min_capacity=3,
         router_bias_var=2.0),
    _cfg("one_expert_64_rows", 64, 264, 520, 1, 1),
    _cfg("two_experts_all_rows", 57, 512, 320, 2, 2, renorm=0),
    _cfg("decode_narrow", 64, 1024, 768, 8, 2),
    _cfg("many_experts", 64, 128, 192, 64, 4, router_bias_var=2.0),
    _cfg("most_records", 64, 72, 136, 64, 8, router_bias_var=1.0),
    _cfg("f32_smallest", 2, 4, 4, 3, 3, dtype=F32),
    _cfg("f32_tiny", 64, 64, 128, 4, 2, dtype=F32),
    _cfg("f32_odd", 5, 100, 516, 7, 2, dtype=F32, act=configs.ACT_GELU_ERF, renorm=0),
    _cfg("f32_drops", 50, 68, 36, 5, 3, dtype=F32, act=configs.ACT_GELU_TANH,
         capacity_factor=0.6, capacity_order=configs.ORDER_TOKEN_MAJOR),
]


@pytest.mark.parametrize("cfg", CASES, ids=[c.name for c in CASES])
def test_few_matches_oracle(abi, cfg):
    inp = inputs.make_inputs(cfg, "cuda")
    out, ex = _run(abi, cfg, inp)
    ref, dg = _reference(cfg, inp, ex)
    _check(cfg, out, ref)
    assert (to_f64(out)[dg["dropped"].all(1)] == 0).all()


W8_CASES = [
    _cfg("w8_smallest", 1, 16, 16, 1, 1),
    _cfg("w8_one_token", 1, 256, 512, 8, 2, act=configs.ACT_GELU_ERF, renorm=0),
    _cfg("w8_odd", 11, 144, 336, 5, 3, capacity_factor=1.0, router_bias_var=1.0),
    _cfg("w8_tail", 8, 2064, 1040, 8, 2, act=configs.ACT_GELU_TANH),
    _cfg("w8_all_rows", 64, 272, 400, 2, 2),
    _cfg("w8_24_rows", 24, 128, 128, 1, 1),
]


@pytest.mark.parametrize("cfg", W8_CASES, ids=[c.name for c in W8_CASES])
def test_few_w8_matches_oracle(abi, cfg):
    inp = inputs.make_inputs(cfg, "cuda", weights=False)
    w8 = inputs.make_w8_weights(cfg, "cuda")
    w8.W1q[0, 0, :3] = torch.tensor([-128, 127, -1], dtype=torch.int8, device="cuda")
    out, ex = _run(abi, cfg, inp, w8)
    ref, _ = _reference(cfg, inp, ex, w8)
    _check(cfg, out, ref)


def test_equal_logits_take_the_lower_expert(abi):
    cfg = _cfg("ties", 5, 64, 64, 40, 4)
    inp = inputs.make_inputs(cfg, "cuda")
    inp.W_r.zero_()
    _, ex = _run(abi, cfg, inp)
    assert (ex["idx"] == np.arange(4)).all() and (ex["gate"] == 0.25).all()
    # -0 and +0 are equal.
    inp.X.zero_()
    inp.W_r.fill_(-1.0)
    _, ex = _run(abi, cfg, inp)
    assert (ex["idx"] == np.arange(4)).all()


def test_capacity_of_zero_gives_zeros(abi):
    # An infinite capacity factor overflows the capacity formula to zero, as in moe_forward.
    cfg = _cfg("none", 9, 72, 64, 4, 2, capacity_factor=float("inf"))
    inp = inputs.make_inputs(cfg, "cuda")
    if abi.capacity(abi.problem(cfg)) != 0:
        pytest.skip("this capacity is not zero here")
    out, ex = _run(abi, cfg, inp)
    assert (out == 0).all() and (ex["dropped"] == 1).all()


def test_repeated_calls_and_dirty_workspace_give_equal_bits(abi):
    cfg = _cfg("again", 13, 520, 776, 8, 2)
    inp = inputs.make_inputs(cfg, "cuda")
    p = abi.problem(cfg)
    ws = abi.workspace(p)
    first, _ = _run(abi, cfg, inp, ws=ws)
    for fill in (0x00, 0xFF, 0x7F):
        ws[256:] = fill  # whatever an earlier call left behind the header
        out, _ = _run(abi, cfg, inp, ws=ws, exports=False)
        assert torch.equal(out.view(torch.int16), first.view(torch.int16))


def test_graph_replay_and_other_stream(abi):
    cfg = _cfg("graph", 6, 256, 384, 8, 2)
    inp = inputs.make_inputs(cfg, "cuda")
    other = inputs.make_inputs(cfg, "cuda", seed=5)
    want, _ = _run(abi, cfg, inp)
    want2, _ = _run(abi, cfg.with_(seed=5), inp.__class__(other.X, inp.W_r, inp.bias, inp.W1,
                                                          inp.W2, inp.W3))
    p = abi.problem(cfg)
    ws = abi.workspace(p)
    X = inp.X.clone()
    out = torch.empty_like(X)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        abi.forward_few(p, X, inp.W_r, inp.bias, inp.W1, inp.W2, inp.W3, out, ws)
    side.synchronize()
    assert torch.equal(out, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for _ in range(3):  # calls in a row on one workspace
            abi.forward_few(p, X, inp.W_r, inp.bias, inp.W1, inp.W2, inp.W3, out, ws)
    for x, w in ((other.X, want2), (inp.X, want), (other.X, want2)):
        X.copy_(x)
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, w)
    assert abi.device_error(ws) == 0


def _guarded(nbytes, n=4096):
    """A workspace of nbytes inside a larger buffer whose other bytes are known."""
    buf = torch.full((nbytes + 2 * n,), 0x5A, dtype=torch.uint8, device="cuda")
    buf[n:n + 256] = 0  # the header
    return buf, buf[n:n + nbytes], lambda: bool((buf[:n] == 0x5A).all() and (buf[-n:] == 0x5A).all())


@pytest.mark.parametrize("name", ["one_by_one", "drops_token_major", "one_expert_64_rows",
                                  "two_experts_all_rows", "most_records", "f32_tiny", "f32_drops"])
def test_writes_stay_in_the_workspace(abi, name):
    cfg = next(c for c in CASES if c.name == name)
    inp = inputs.make_inputs(cfg, "cuda")
    buf, ws, intact = _guarded(abi.workspace_size(abi.problem(cfg)))
    _run(abi, cfg, inp, ws=ws)
    assert intact()


def test_two_streams_at_once(abi):
    # Calls on two streams, one of high priority, with a workspace each and other kernels beside
    # them: every call's own result, no wait that runs out.
    cfg = _cfg("pair", 5, 512, 1024, 8, 2)
    inp = inputs.make_inputs(cfg, "cuda")
    want, _ = _run(abi, cfg, inp)
    p = abi.problem(cfg)
    streams = [torch.cuda.Stream(), torch.cuda.Stream(priority=-1)]
    ws = [abi.workspace(p) for _ in streams]
    outs = [[torch.empty_like(inp.X) for _ in range(20)] for _ in streams]
    big = [torch.randn((2048, 2048), device="cuda") for _ in streams]
    torch.cuda.synchronize()
    for i in range(20):
        for s, w, out, b in zip(streams, ws, outs, big):
            with torch.cuda.stream(s):
                b.mul_(0.5)
                abi.forward_few(p, inp.X, inp.W_r, inp.bias, inp.W1, inp.W2, inp.W3, out[i], w)
    torch.cuda.synchronize()
    assert all(abi.device_error(w) == 0 for w in ws)
    assert all(torch.equal(o, want) for out in outs for o in out)


def test_a_larger_batch_s_workspace(abi):
    # One workspace for a server's largest batch, used by both forms of the layer in turn.
    cfg = _cfg("largest", 200, 128, 256, 8, 2)
    small = cfg.with_(N=20)
    ws = abi.workspace(abi.problem(cfg))
    inp, few = inputs.make_inputs(cfg, "cuda"), inputs.make_inputs(small, "cuda")
    want, _ = _run(abi, small, few)
    p = abi.problem(cfg)
    alone, out = torch.empty_like(inp.X), torch.empty_like(inp.X)
    abi.forward(p, inp.X, inp.W_r, inp.bias, inp.W1, inp.W2, inp.W3, alone, ws)
    for _ in range(2):
        got, _ = _run(abi, small, few, ws=ws)
        assert torch.equal(got, want)
        abi.forward(p, inp.X, inp.W_r, inp.bias, inp.W1, inp.W2, inp.W3, out, ws)
        torch.cuda.synchronize()
        assert torch.equal(out, alone)


def test_activations_past_the_bf16_range(abi):
    # h = 3.394e38 lies between the largest bf16 (3.3895e38) and the largest fp32 value, and rounds
    # to an infinite bf16 term: infinity, not NaN. GELU of a large value is the value itself.
    cfg = _cfg("edge", 1, 8, 8, 1, 1, act=configs.ACT_GELU_ERF)
    X = torch.zeros((1, 8), dtype=torch.bfloat16, device="cuda")
    X[0, 0] = 1.0
    X[0, 1] = 2.0 ** -10
    W1 = torch.zeros((1, 8, 8), dtype=torch.bfloat16, device="cuda")
    W2, W3 = torch.zeros_like(W1), torch.zeros_like(W1)
    W1[0, 0, 0] = 2.0 ** 64
    # x W2 = 2^64 (1 - 2^-9 + 2^-12), exact in fp32.
    W2[0, 0, 0] = 255.0 / 256 * 2.0 ** 64
    W2[0, 1, 0] = (2.0 ** -9 + 2.0 ** -12) * 2.0 ** 74
    W3[0, 0] = 1.0
    h = 2.0 ** 64 * float(W2[0, 0, 0].float() + W2[0, 1, 0].float() * 2.0 ** -10)
    assert torch.finfo(torch.bfloat16).max < h < torch.finfo(torch.float32).max
    W_r = torch.zeros((8, 1), device="cuda")
    out, _ = _run(abi, cfg, inputs.MoEInputs(X, W_r, None, W1, W2, W3))
    assert (out == float("inf")).all()


def test_a_nan_token_leaves_the_others_alone(abi):
    # Non-finite inputs are unsupported, but a bad token must not reach the other rows.
    cfg = _cfg("nan", 12, 72, 104, 2, 1)
    inp = inputs.make_inputs(cfg, "cuda")
    want, _ = _run(abi, cfg, inp)
    inp.X[7] = float("nan")
    p = abi.problem(cfg)
    ws = abi.workspace(p)
    out = torch.empty_like(inp.X)
    abi.forward_few(p, inp.X, inp.W_r, inp.bias, inp.W1, inp.W2, inp.W3, out, ws)
    torch.cuda.synchronize()
    keep = [t for t in range(cfg.N) if t != 7]
    assert torch.equal(out[keep], want[keep])


def test_no_tokens(abi):
    cfg = _cfg("none", 0, 64, 64, 4, 2)
    one = inputs.make_inputs(cfg.with_(N=1), "cuda")
    p = abi.problem(cfg)
    ws = abi.workspace(p)
    load = torch.full((4,), 9, dtype=torch.int32, device="cuda")
    offsets = torch.full((5,), 9, dtype=torch.int32, device="cuda")
    out = torch.full((1, 64), 3.0, dtype=torch.bfloat16, device="cuda")
    abi.forward_few(p, one.X, one.W_r, None, one.W1, one.W2, one.W3, out, ws, load=load,
                    offsets=offsets)
    torch.cuda.synchronize()
    assert (load == 0).all() and (offsets == 0).all() and (out == 3.0).all()


def test_agrees_with_the_whole_layer_call(abi):
    # The same layer through moe_forward, which rounds H and Y to bf16 on the way: one rounding
    # of 2^-8 for each of H, Y and the output, relative to the row's scale.
    cfg = _cfg("both", 48, 512, 1024, 8, 2, capacity_factor=1.0, router_bias_var=1.0)
    inp = inputs.make_inputs(cfg, "cuda")
    out, ex = _run(abi, cfg, inp)
    layer = abi.Layer(cfg)
    idx = torch.empty((cfg.N, cfg.k), dtype=torch.int32, device="cuda")
    ref = layer.forward(inp.X, inp.W_r, inp.bias, inp.W1, inp.W2, inp.W3, topk_idx=idx)
    same = layer.forward_few(inp.X, inp.W_r, inp.bias, inp.W1, inp.W2, inp.W3)
    torch.cuda.synchronize()
    assert torch.equal(same, out)
    assert np.array_equal(idx.cpu().numpy(), ex["idx"])
    a, b = to_f64(out), to_f64(ref)
    assert (np.abs(a - b).max(1) <= 3 * 2.0 ** -8 * np.abs(b).max(1) + 1e-6).all()


def test_an_expert_past_32_bit_offsets(abi):
    # The last of 64 experts lies past 2^31 elements: the same bits as a layer of it alone.
    D, F, E = 4096, 8448, 64
    assert (E - 1) * D * F > 2 ** 31
    one = inputs.make_inputs(_cfg("one", 3, D, F, 1, 1), "cuda")
    far = [torch.zeros((E,) + tuple(w.shape[1:]), dtype=w.dtype, device="cuda")
           for w in (one.W1, one.W2, one.W3)]
    for w, o in zip(far, (one.W1, one.W2, one.W3)):
        w[E - 1] = o[0]
    bias = torch.zeros(E, device="cuda")
    bias[E - 1] = 1e4
    W_r = torch.zeros((D, E), device="cuda")
    cfg = _cfg("far", 3, D, F, E, 1)
    want, _ = _run(abi, cfg.with_(E=1), one)
    inp = inputs.MoEInputs(one.X, W_r, bias, *far)
    out, ex = _run(abi, cfg, inp)
    assert (ex["idx"] == E - 1).all() and torch.equal(out, want)
