"""The serving operators for small batches and per-request adapters: what is computed, in which
sizes, and what each pass has to read and write.

Two operators:

* ``few``  -- the whole mixture-of-experts layer for a few tokens (1 to 64): fp32 router, softmax,
  top-k, capacity, gated expert FFNs and the gate-weighted sum, ``abi.forward_few`` (bf16 or fp32
  weights) and ``abi.forward_few_w8`` (8-bit expert weights with one scale per output column).
* ``lora`` -- a projection that every row takes, X W, beside the low-rank adapter of the row's own
  request, scale[a] (X A[a]) B[a], and an optional addend, ``abi.lora_forward``.

``run`` computes them in their plain form from elementary torch operations, or, with ``own`` set,
through the package's entry points. ``exact`` is the definition in 64 bits.
"""
import math
from types import SimpleNamespace

import torch

own = False

F32, BF16, W8 = "f32", "bf16", "w8"
SILU, GELU_ERF, GELU_TANH = 0, 1, 2


def _few(name, N, D, F, E, k, dtype=BF16, act=SILU, renorm=1, cf=0.0, min_cap=0, token_major=0,
         renorm_kept=0, bias_var=0.0):
    return dict(name=name, op="few", N=N, D=D, F=F, E=E, k=k, dtype=dtype, act=act, renorm=renorm,
                cf=cf, min_cap=min_cap, token_major=token_major, renorm_kept=renorm_kept,
                bias_var=bias_var)


def _lora(name, M, K, N, L, r, dtype=BF16, run_rows=1, none=0.0, addend=False):
    return dict(name=name, op="lora", M=M, K=K, N=N, L=L, r=r, dtype=dtype, run_rows=run_rows,
                none=none, addend=addend)


def listed():
    return [
        # One user generating on the Mixtral-shaped layer: two experts' weights are all there is.
        _few("few_1_mixtral", 1, 4096, 14336, 8, 2),
        # The decode workload's batch: nearly every expert is read, 16 rows each on average.
        _few("few_64_decode", 64, 4096, 14336, 8, 2),
        # Eight users on the same layer with 8-bit expert weights.
        _few("few_8_mixtral_w8", 8, 4096, 14336, 8, 2, dtype=W8),
        # Four users on a layer of many small experts, with a capacity and a router bias.
        _few("few_4_experts64", 4, 2048, 8192, 64, 2, cf=1.25, min_cap=2, bias_var=2.0),
        # Sixteen users on the Grok-1-shaped layer: the largest weights, erf GELU, no renorm.
        _few("few_16_grok1", 16, 6144, 32768, 8, 2, act=GELU_ERF, renorm=0),
        # Odd widths, an odd number of experts, three per token, and a capacity that drops.
        _few("few_17_odd", 17, 1000, 2728, 13, 3, act=GELU_TANH, cf=1.0, token_major=1,
             renorm_kept=1, bias_var=1.0),
        # The fp32 test layer for one token: nothing but latency.
        _few("few_1_tiny_f32", 1, 64, 128, 4, 2, dtype=F32),
        # One request with its adapter beside a square projection of the model width.
        _lora("lora_1_square", 1, 4096, 4096, 8, 16),
        # A decode batch: every row another request's adapter, a few rows without one, beside an
        # up-projection, added to a residual.
        _lora("lora_48_mixed", 48, 4096, 14336, 64, 16, none=0.1, addend=True),
        # Odd rows, widths and rank; short prompts of a few requests.
        _lora("lora_200_odd", 200, 2040, 5000, 5, 24, run_rows=33, none=0.2),
        # Prompts of eight requests, 512 tokens each: one large product.
        _lora("lora_4096_prompts", 4096, 4096, 14336, 8, 64, run_rows=512),
        # The fp32 test layer's widths.
        _lora("lora_64_f32", 64, 64, 128, 4, 8, dtype=F32, addend=True),
    ]


def _log_int(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(step, int(round(v / step)) * step)


def draw(rng):
    if rng.random() < 0.5:
        dtype = rng.choice([BF16, BF16, BF16, W8, F32])
        step = {BF16: 8, W8: 16, F32: 4}[dtype]
        E = _log_int(rng, 2, 64)
        k = rng.randint(1, min(E, 4))
        D = _log_int(rng, 64, 6144, step)
        # The experts' weights stay under a quarter of the largest listed layer's.
        cap = 2.4e9 / (3.0 * E * D * (4 if dtype == F32 else 2))
        F = _log_int(rng, 64, max(65.0, min(32768.0, cap)), step)
        cf = rng.choice([0.0, 0.0, 1.0, 1.25])
        return _few(None, _log_int(rng, 1, 64), D, F, E, k, dtype=dtype, act=rng.randint(0, 2),
                    renorm=rng.randint(0, 1), cf=cf, min_cap=rng.choice([0, 2]),
                    token_major=rng.randint(0, 1), renorm_kept=rng.randint(0, 1),
                    bias_var=rng.choice([0.0, 1.0, 2.0]))
    dtype = rng.choice([BF16, BF16, BF16, BF16, F32])
    M = _log_int(rng, 1, 4096 if dtype == BF16 else 256)
    r = rng.choice([8, 16, 16, 24, 32, 64])
    return _lora(None, M, _log_int(rng, 64, 4096, 8), _log_int(rng, 64, 14336, 8),
                 _log_int(rng, 1, 64 if r <= 32 else 16), r, dtype=dtype,
                 run_rows=min(M, _log_int(rng, 1, 512)) if M > 64 else rng.choice([1, 1, 3]),
                 none=rng.choice([0.0, 0.1, 0.5]), addend=rng.random() < 0.5)


def work(case):
    c = SimpleNamespace(**case)
    if c.op == "few":
        # Experts that N tokens with k of E each are expected to reach, each read once.
        used = min(c.E * (1.0 - (1.0 - c.k / c.E) ** c.N), float(c.N * c.k))
        el = {F32: 4, BF16: 2, W8: 1}[c.dtype]
        act = 4 if c.dtype == F32 else 2
        weights = used * 3 * c.D * c.F * el
        if c.dtype == W8:
            weights += used * 4 * (2 * c.F + c.D)
        data = c.D * c.E * 4 + 2 * c.N * c.D * act + c.N * c.k * 9
        return {"bytes": weights + data,
                "flops": 6.0 * c.N * c.k * c.D * c.F + 2.0 * c.N * c.D * c.E}
    el = 4 if c.dtype == F32 else 2
    requests = -(-c.M // c.run_rows)
    used = c.L * (1.0 - (1.0 - (1.0 - c.none) / c.L) ** requests)
    b = el * (c.M * c.K + c.K * c.N + c.M * c.N * (2 if c.addend else 1) + used * c.r * (c.K + c.N))
    return {"bytes": b + 4 * c.M,
            "flops": 2.0 * c.M * c.K * c.N + 2.0 * c.M * (1.0 - c.none) * c.r * (c.K + c.N)}


# ---------------------------------------------------------------------------- inputs


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _normal(g, shape, std, dtype):
    return torch.randn(shape, generator=g, device="cuda", dtype=dtype).mul_(std)


def prepare(case, seed):
    c = SimpleNamespace(**case)
    g = _gen(seed)
    t = torch.float32 if c.dtype == F32 else torch.bfloat16
    s = {"case": dict(case)}
    if c.op == "few":
        s["X"] = _normal(g, (c.N, c.D), 1.0, t)
        s["W_r"] = _normal(g, (c.D, c.E), c.D ** -0.5, torch.float32)
        s["bias"] = _normal(g, (c.E,), c.bias_var ** 0.5, torch.float32) if c.bias_var > 0 else None
        for name, rows, cols in (("1", c.D, c.F), ("2", c.D, c.F), ("3", c.F, c.D)):
            if c.dtype == W8:
                # Quantised normal weights: 127 stands for about four standard deviations.
                q = torch.empty((c.E, rows, cols), dtype=torch.int8, device="cuda")
                for e in range(c.E):
                    q[e] = _normal(g, (rows, cols), 32.0, torch.float32).round_().clamp_(-127, 127)
                s["W" + name + "q"] = q
                s["S" + name] = (torch.rand((c.E, cols), generator=g, device="cuda") + 0.5) * (
                    rows ** -0.5 / 32.0)
            else:
                s["W" + name] = _normal(g, (c.E, rows, cols), rows ** -0.5, t)
        s["out"] = torch.empty_like(s["X"])
        s["idx"] = torch.empty((c.N, c.k), dtype=torch.int32, device="cuda")
        s["gate"] = torch.empty((c.N, c.k), dtype=torch.float32, device="cuda")
        s["dropped"] = torch.empty((c.N, c.k), dtype=torch.uint8, device="cuda")
        return s
    s["X"] = _normal(g, (c.M, c.K), 1.0, t)
    s["W"] = _normal(g, (c.K, c.N), c.K ** -0.5, t)
    s["A"] = _normal(g, (c.L, c.K, c.r), c.K ** -0.5, t)
    s["B"] = _normal(g, (c.L, c.r, c.N), c.r ** -0.5, t)
    s["scale"] = torch.rand((c.L,), generator=g, device="cuda") + 0.5
    # Requests of run_rows rows each, a random adapter for each (-1: the request has none).
    requests = -(-c.M // c.run_rows)
    a = torch.randint(0, c.L, (requests,), generator=g, device="cuda", dtype=torch.int32)
    a[torch.rand((requests,), generator=g, device="cuda") < c.none] = -1
    s["adapter"] = a.repeat_interleave(c.run_rows)[:c.M].contiguous()
    s["addend"] = _normal(g, (c.M, c.N), 1.0, t) if c.addend else None
    s["Y"] = torch.empty((c.M, c.N), dtype=t, device="cuda")
    return s


# ---------------------------------------------------------------------------- plain forms


def _act(kind, v):
    if kind == SILU:
        return v * torch.sigmoid(v)
    if kind == GELU_ERF:
        return v * 0.5 * (1.0 + torch.erf(v * 0.5 ** 0.5))
    return 0.5 * v * (1.0 + torch.tanh((2.0 / math.pi) ** 0.5 * (v + 0.044715 * v * v * v)))


def _expert_weight(s, name, pick):
    """The picked experts' matrix in fp32 (8-bit weights: value times its column's scale)."""
    if "W1q" in s:
        return s["W" + name + "q"][pick].float() * s["S" + name][pick].unsqueeze(-2)
    return s["W" + name][pick].float()


def _capacity(c):
    if c.cf <= 0:
        return c.N * c.k
    return max(math.ceil(c.cf * float(c.N) * float(c.k) / float(c.E)), c.min_cap)


def _plain_few(s):
    c = SimpleNamespace(**s["case"])
    z = s["X"].double() @ s["W_r"].double()  # 64 bits: a choice between experts hangs on it
    if s["bias"] is not None:
        z = z + s["bias"].double()
    idx = torch.sort(z, dim=1, descending=True, stable=True).indices[:, :c.k]
    zs = torch.gather(z, 1, idx)
    gate = torch.softmax(zs, 1) if c.renorm else torch.gather(torch.softmax(z, 1), 1, idx)
    # Position of each record among its expert's, in the order that records take capacity.
    order = idx if c.token_major else idx.t()
    hot = torch.nn.functional.one_hot(order.reshape(-1), c.E)
    pos = ((hot.cumsum(0) - 1) * hot).sum(1).reshape(order.shape)
    dropped = (pos if c.token_major else pos.t()) >= _capacity(c)
    g = torch.where(dropped, 0.0, gate)
    if c.renorm_kept:
        mend = dropped.any(1, keepdim=True) & ~dropped.all(1, keepdim=True)
        g = torch.where(mend, g / g.sum(1, keepdim=True).clamp_min(1e-300), g)
    X, g = s["X"].float(), g.float()
    if c.N * c.k <= c.E:  # fewer records than experts: each record's own matrices
        pick = idx.reshape(-1)
        x = X.repeat_interleave(c.k, 0).unsqueeze(1)
        h = _act(c.act, x @ _expert_weight(s, "1", pick)) * (x @ _expert_weight(s, "2", pick))
        y = (h @ _expert_weight(s, "3", pick)).reshape(c.N, c.k, c.D)
        out = (y * g.unsqueeze(-1)).sum(1)
    else:  # every expert on every token, weighted by the gates (zero where not chosen)
        every = slice(None)
        w = torch.zeros((c.N, c.E), device=X.device).scatter_(1, idx, g).t().unsqueeze(-1)
        h = _act(c.act, X @ _expert_weight(s, "1", every)) * (X @ _expert_weight(s, "2", every))
        out = ((h @ _expert_weight(s, "3", every)) * w).sum(0)
    return {"out": out.to(s["X"].dtype), "topk_idx": idx.int(), "topk_gate": gate.float(),
            "dropped": dropped.to(torch.uint8)}


def _plain_lora(s):
    c = SimpleNamespace(**s["case"])
    X = s["X"].float()
    a = s["adapter"].long()
    mine = (a.unsqueeze(1) == torch.arange(c.L, device=X.device)).float() * s["scale"]
    xa = (X @ s["A"].float().transpose(0, 1).reshape(c.K, c.L * c.r)).reshape(c.M, c.L, c.r)
    y = X @ s["W"].float() + (xa * mine.unsqueeze(-1)).reshape(c.M, c.L * c.r) @ s[
        "B"].float().reshape(c.L * c.r, c.N)
    if s["addend"] is not None:
        y = y + s["addend"].float()
    return {"Y": y.to(s["X"].dtype)}


# ---------------------------------------------------------------------------- the package's calls


def _own_few(s):
    from top_routing_expert_fp32_b200 import abi, configs
    c = SimpleNamespace(**s["case"])
    if "layer" not in s:  # the problem and its workspace, kept as a serving loop keeps them
        cfg = configs.MoEConfig(
            "few", N=c.N, D=c.D, F=c.F, E=c.E, k=c.k,
            dtype=configs.DTYPE_F32 if c.dtype == F32 else configs.DTYPE_BF16, activation=c.act,
            renormalize=c.renorm, capacity_factor=c.cf, capacity_order=c.token_major,
            drop_policy=c.renorm_kept, min_capacity=c.min_cap)
        s["layer"] = abi.Layer(cfg)
        s["w8"] = SimpleNamespace(**{n: s[n] for n in ("W1q", "S1", "W2q", "S2", "W3q", "S3")}
                                  ) if c.dtype == W8 else None
    layer = s["layer"]
    more = dict(topk_idx=s["idx"], topk_gate=s["gate"], dropped=s["dropped"])
    if c.dtype == W8:
        abi.forward_few_w8(layer.p, s["X"], s["W_r"], s["bias"], s["w8"], s["out"], layer.ws,
                           **more)
    else:
        abi.forward_few(layer.p, s["X"], s["W_r"], s["bias"], s["W1"], s["W2"], s["W3"], s["out"],
                        layer.ws, **more)
    return {"out": s["out"], "topk_idx": s["idx"], "topk_gate": s["gate"],
            "dropped": s["dropped"]}


def _own_lora(s):
    from top_routing_expert_fp32_b200 import abi, configs
    c = SimpleNamespace(**s["case"])
    if "lora" not in s:
        p = abi.lora_problem(M=c.M, K=c.K, N=c.N, adapters=c.L, rank=c.r,
                             dtype=configs.DTYPE_F32 if c.dtype == F32 else configs.DTYPE_BF16)
        s["lora"] = (p, abi.lora_workspace(p))
    p, ws = s["lora"]
    abi.lora_forward(p, s["X"], s["W"], s["A"], s["B"], s["adapter"], s["Y"], ws,
                     scale=s["scale"], addend=s["addend"])
    return {"Y": s["Y"]}


def run(state):
    if state["case"]["op"] == "few":
        return _own_few(state) if own else _plain_few(state)
    return _own_lora(state) if own else _plain_lora(state)


# ---------------------------------------------------------------------------- 64 bits


def exact(case, seed):
    c = SimpleNamespace(**case)
    s = prepare(case, seed)
    if c.op == "lora":
        x = s["X"].double()
        y = x @ s["W"].double()
        ids = s["adapter"].tolist()
        for a in sorted(set(ids) - {-1}):
            rows = torch.tensor([m for m, v in enumerate(ids) if v == a], device=x.device)
            y[rows] += s["scale"][a].double() * (
                (x[rows] @ s["A"][a].double()) @ s["B"][a].double())
        if s["addend"] is not None:
            y += s["addend"].double()
        return {"Y": y}
    x = s["X"].double()
    logits = x @ s["W_r"].double()
    if s["bias"] is not None:
        logits += s["bias"].double()
    rows = logits.tolist()
    chosen = [sorted(range(c.E), key=lambda e: (-z[e], e))[:c.k] for z in rows]
    gates = []
    for z, sel in zip(rows, chosen):
        top = max(z)
        total = sum(math.exp(z[e] - top) for e in (sel if c.renorm else range(c.E)))
        gates.append([math.exp(z[e] - top) / total for e in sel])
    room = [c.N * c.k if c.cf <= 0 else max(math.ceil(c.cf * c.N * c.k / c.E), c.min_cap)] * c.E
    drop = [[0] * c.k for _ in range(c.N)]
    records = ([(t, j) for t in range(c.N) for j in range(c.k)] if c.token_major else
               [(t, j) for j in range(c.k) for t in range(c.N)])
    for t, j in records:
        e = chosen[t][j]
        if room[e] > 0:
            room[e] -= 1
        else:
            drop[t][j] = 1
    out = torch.zeros((c.N, c.D), dtype=torch.float64, device=x.device)
    for e in range(c.E):
        mine = [(t, j) for t in range(c.N) for j in range(c.k) if chosen[t][j] == e
                and not drop[t][j]]
        if not mine:
            continue
        mats = []
        for n in "123":
            if c.dtype == W8:
                mats.append(s["W" + n + "q"][e].double() * s["S" + n][e].double())
            else:
                mats.append(s["W" + n][e].double())
        tok = torch.tensor([t for t, _ in mine], device=x.device)
        u = x[tok] @ mats[0]
        if c.act == SILU:
            u = u / (1.0 + torch.exp(-u))
        elif c.act == GELU_ERF:
            u = 0.5 * u * torch.special.erfc(-u / math.sqrt(2.0))
        else:
            u = u / (1.0 + torch.exp(-2.0 * math.sqrt(2.0 / math.pi) * (u + 0.044715 * u ** 3)))
        y = (u * (x[tok] @ mats[1])) @ mats[2]
        w = []
        for t, j in mine:
            kept = sum(gates[t][i] for i in range(c.k) if not drop[t][i])
            w.append(gates[t][j] / kept if c.renorm_kept and any(drop[t]) else gates[t][j])
        out.index_add_(0, tok, y * torch.tensor(w, dtype=torch.float64,
                                                device=x.device).unsqueeze(1))
    return {"out": out, "topk_idx": torch.tensor(chosen, dtype=torch.int32),
            "topk_gate": torch.tensor(gates, dtype=torch.float64),
            "dropped": torch.tensor(drop, dtype=torch.uint8)}
