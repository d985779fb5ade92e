"""GPU parity of the shared projection with per-row adapters (moe_lora_forward) against the
formula in 64 bits, its refusals, and its behaviour under graphs, streams and used workspaces.

Tolerances. The output is rounded once: at most 2^-8 (bf16) or 2^-24 (fp32) of the value. The
fp32 sums of n <= 2^13 terms before it err by at most a few sqrt(n) 2^-23 of the terms' 2-norm
(tensor cores truncate): 1e-4 of the row's largest value covers them with room (fp32 kernels keep
runs of at most 64 terms: 1e-5). More than 64 bf16 rows round S = scale X A to bf16: at most 2^-8
of every term S_r B_rn, so 2^-8 sum_r |S_r| |B_rn|."""
import pytest
import torch

from top_routing_expert_fp32_b200 import configs

pytestmark = pytest.mark.gpu

BF16, F32 = configs.DTYPE_BF16, configs.DTYPE_F32


@pytest.fixture(scope="module")
def abi():
    from top_routing_expert_fp32_b200 import abi as a
    return a


class Case:
    def __init__(self, M, K, N, L, r, dtype=BF16, rows=1, none=0.0, addend=False, scale=True,
                 seed=0):
        g = torch.Generator(device="cuda")
        g.manual_seed(1000 + seed)
        t = torch.bfloat16 if dtype == BF16 else torch.float32
        rnd = lambda shape, std: (torch.randn(shape, generator=g, device="cuda") * std).to(t)
        self.M, self.K, self.N, self.L, self.r, self.dtype = M, K, N, L, r, dtype
        self.X, self.W = rnd((M, K), 1.0), rnd((K, N), K ** -0.5)
        self.A, self.B = rnd((L, K, r), K ** -0.5), rnd((L, r, N), r ** -0.5)
        n = -(-M // rows) if M else 0
        ids = torch.randint(0, L, (n,), generator=g, device="cuda", dtype=torch.int32)
        ids[torch.rand((n,), generator=g, device="cuda") < none] = -1
        self.adapter = ids.repeat_interleave(rows)[:M].contiguous()
        self.scale = torch.rand((L,), generator=g, device="cuda") + 0.5 if scale else None
        self.addend = rnd((M, N), 1.0) if addend else None

    def run(self, abi, ws=None, adapter=None, Y=None, err=0):
        p = abi.lora_problem(self.M, self.K, self.N, self.L, self.r, self.dtype)
        ws = abi.lora_workspace(p) if ws is None else ws
        buf = None
        if Y is None:  # a row behind the last one, which must stay as it is
            buf = torch.full((self.M + 1, self.N), 7.5, dtype=self.X.dtype, device="cuda")
            Y = buf[:self.M]
        abi.lora_forward(p, self.X, self.W, self.A, self.B,
                         self.adapter if adapter is None else adapter, Y, ws, scale=self.scale,
                         addend=self.addend)
        torch.cuda.synchronize()
        assert abi.device_error(ws) == err
        assert buf is None or (buf[self.M] == 7.5).all()
        assert ws[:256].view(torch.int32).abs().sum().item() == 0
        return Y

    def reference(self, adapter=None):
        """(Y, sum_r |S_r| |B_rn|) in 64 bits."""
        x = self.X.double()
        y, spread = x @ self.W.double(), torch.zeros((self.M, self.N), device="cuda").double()
        ids = (self.adapter if adapter is None else adapter).tolist()
        for a in sorted(set(ids)):
            if not 0 <= a < self.L:
                continue
            rows = torch.tensor([m for m, v in enumerate(ids) if v == a], device="cuda")
            s = x[rows] @ self.A[a].double()
            if self.scale is not None:
                s = s * self.scale[a].double()
            y[rows] += s @ self.B[a].double()
            spread[rows] = s.abs() @ self.B[a].double().abs()
        if self.addend is not None:
            y += self.addend.double()
        return y, spread

    def check(self, Y, adapter=None):
        ref, spread = self.reference(adapter)
        half, sums = (2.0 ** -8, 1e-4) if self.dtype == BF16 else (2.0 ** -24, 1e-5)
        bound = half * ref.abs() + sums * ref.abs().amax(1, keepdim=True)
        if self.dtype == BF16 and self.M > 64:
            bound += 2.0 ** -8 * spread
        got = Y.double()
        assert torch.isfinite(got).all()
        worst = ((got - ref).abs() - bound).max().item()
        assert worst <= 0, f"over the bound by {worst:.3g} (largest {ref.abs().max().item():.3g})"


FEW = [
    dict(M=1, K=8, N=8, L=1, r=8),
    dict(M=1, K=4096, N=4096, L=8, r=16),
    dict(M=2, K=136, N=264, L=3, r=128, addend=True),
    dict(M=7, K=2040, N=520, L=5, r=24, none=0.3),
    dict(M=8, K=64, N=72, L=2, r=8, scale=False),
    dict(M=17, K=200, N=5000, L=40, r=40),
    dict(M=31, K=1032, N=1000, L=4, r=64, rows=5, addend=True),
    dict(M=33, K=512, N=136, L=64, r=16),
    dict(M=48, K=1024, N=3584, L=64, r=16, none=0.1, addend=True),
    dict(M=64, K=2048, N=2048, L=64, r=16),
    dict(M=64, K=72, N=520, L=6, r=128, none=1.0),
    dict(M=1, K=4, N=4, L=1, r=4, dtype=F32),
    dict(M=5, K=100, N=516, L=3, r=12, dtype=F32, addend=True),
    dict(M=30, K=512, N=68, L=9, r=128, dtype=F32, none=0.2),
    dict(M=64, K=64, N=128, L=4, r=8, dtype=F32, addend=True),
    dict(M=12, K=4096, N=40, L=3, r=16, addend=True),                # a tile shared by many blocks
    dict(M=40, K=1000, N=136, L=30, r=24, addend=True),              # pairs of warps
    dict(M=50, K=256, N=20480, L=50, r=16, addend=True),             # and whole tiles
    dict(M=63, K=4096, N=4096, L=5, r=96, none=0.2),
    dict(M=12, K=260, N=1000, L=3, r=20, dtype=F32, addend=True),
    dict(M=41, K=1284, N=252, L=20, r=36, dtype=F32, none=0.3),
    dict(M=10, K=132, N=16384, L=2, r=64, dtype=F32, addend=True),
    dict(M=64, K=4096, N=512, L=64, r=16, dtype=F32, scale=False),
]

MANY = [
    dict(M=65, K=8, N=8, L=1, r=8),
    dict(M=65, K=256, N=512, L=70, r=16),
    dict(M=100, K=1000, N=264, L=3, r=24, rows=33, none=0.3, addend=True),
    dict(M=128, K=512, N=1024, L=200, r=16, scale=False),
    dict(M=129, K=136, N=72, L=2, r=128),
    dict(M=200, K=2040, N=5000, L=5, r=24, rows=33, none=0.2),
    dict(M=257, K=384, N=520, L=64, r=64, none=0.1),
    dict(M=512, K=512, N=256, L=4, r=40, rows=100, addend=True),
    dict(M=513, K=512, N=2056, L=16, r=8, rows=7),
    dict(M=600, K=320, N=4096, L=300, r=16),
    dict(M=1100, K=264, N=9216, L=6, r=80, rows=90),          # 9 x 36 tiles of 256 columns
    dict(M=2500, K=456, N=4104, L=8, r=64, rows=313, addend=True),   # pairs, ragged edges
    dict(M=2560, K=512, N=4096, L=300, r=16),                 # pairs, all rows different
    dict(M=4000, K=128, N=3000, L=5, r=128, rows=64, none=0.5),      # pairs, half tiles
    dict(M=3000, K=256, N=4096, L=3, r=32, none=1.0),         # no row has an adapter
    dict(M=65, K=100, N=132, L=7, r=12, dtype=F32, addend=True),
    dict(M=130, K=1028, N=260, L=3, r=128, dtype=F32, rows=20, none=0.3),
    dict(M=70, K=4, N=4, L=2, r=4, dtype=F32),
    dict(M=300, K=4100, N=68, L=5, r=4, dtype=F32, addend=True),     # K over eight blocks
    dict(M=257, K=260, N=1028, L=9, r=64, dtype=F32, none=0.1),
]


@pytest.mark.parametrize("kw", FEW + MANY, ids=lambda k: "-".join(str(v) for v in k.values()))
def test_lora_matches_the_formula(abi, kw):
    c = Case(**kw)
    c.check(c.run(abi))


@pytest.mark.parametrize("M", [3, 64, 65, 300, 2560])
def test_bad_adapter_index_is_reported_and_ignored(abi, M):
    c = Case(M, 256, 4096 if M > 2000 else 512, 4, 16)
    bad = c.adapter.clone()
    bad[0], bad[M // 2], bad[M - 1] = 4, -2, 2 ** 31 - 1
    c.check(c.run(abi, adapter=bad, err=abi.DEVERR_BAD_INDEX), bad)


@pytest.mark.parametrize("M", [5, 64, 130, 2560])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_bad_adapter_or_row_stays_with_its_rows(abi, M, bad):
    # One request's adapter or activations may hold anything: the other rows do not see it.
    c = Case(M, 128, 4096 if M > 2000 else 256, 6, 16, rows=2, none=0.2)
    want = c.run(abi)
    c.A[2] = bad
    c.B[2, 3] = bad
    c.X[M - 1] = bad
    got = c.run(abi)
    keep = c.adapter != 2
    keep[M - 1] = False
    assert keep.any() and torch.equal(got[keep], want[keep])


@pytest.mark.parametrize("M,dtype", [(9, BF16), (64, F32), (200, BF16), (2560, BF16), (70, F32)])
def test_in_place_residual_and_repeats(abi, M, dtype):
    c = Case(M, 264, 4096 if M > 2000 else 392, 5, 16, dtype=dtype, rows=3, addend=True)
    want = c.run(abi)
    p = abi.lora_problem(c.M, c.K, c.N, c.L, c.r, c.dtype)
    ws = abi.lora_workspace(p)
    for fill in (0x00, 0xFF, 0x7F):
        ws[256:] = fill  # whatever an earlier call left behind the header
        assert torch.equal(c.run(abi, ws=ws), want)
    Y = c.addend.clone()
    c.addend = Y  # Y += ...
    c.run(abi, ws=ws, Y=Y)
    assert torch.equal(Y, want)


@pytest.mark.parametrize("M", [4, 200, 2560])
def test_graph_replay_and_other_stream(abi, M):
    c = Case(M, 256, 4096 if M > 2000 else 640, 5, 16)
    d = Case(M, 256, 4096 if M > 2000 else 640, 5, 16, seed=1)
    d.W, d.A, d.B, d.scale = c.W, c.A, c.B, c.scale
    want, want2 = c.run(abi), d.run(abi)
    p = abi.lora_problem(c.M, c.K, c.N, c.L, c.r, c.dtype)
    ws = abi.lora_workspace(p)
    X, ids, Y = c.X.clone(), c.adapter.clone(), torch.empty_like(want)
    call = lambda: abi.lora_forward(p, X, c.W, c.A, c.B, ids, Y, ws, scale=c.scale)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    side.synchronize()
    assert torch.equal(Y, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for _ in range(3):
            call()
    for x, w in ((d, want2), (c, want), (d, want2)):
        X.copy_(x.X)
        ids.copy_(x.adapter)
        Y.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(Y, w)
    assert abi.device_error(ws) == 0


@pytest.mark.parametrize("kw", [FEW[0], FEW[1], FEW[7], FEW[9], FEW[14], FEW[17], FEW[20],
                                MANY[1], MANY[4], MANY[12], MANY[16], MANY[18]],
                         ids=lambda k: "-".join(str(v) for v in k.values()))
def test_writes_stay_in_the_workspace(abi, kw):
    import ctypes
    c = Case(**kw)
    p = abi.lora_problem(c.M, c.K, c.N, c.L, c.r, c.dtype)
    size = ctypes.c_size_t()
    assert abi.lib.moe_lora_workspace_size(ctypes.byref(p), ctypes.byref(size)) == 0
    n, pad = size.value, 4096
    buf = torch.full((n + 2 * pad,), 0x5A, dtype=torch.uint8, device="cuda")
    buf[pad:pad + 256] = 0  # the header
    c.check(c.run(abi, ws=buf[pad:pad + n]))
    assert (buf[:pad] == 0x5A).all() and (buf[-pad:] == 0x5A).all()


@pytest.mark.parametrize("M", [4, 200])
def test_two_streams_at_once(abi, M):
    # Calls on two streams, one of high priority, with a workspace each: every call's own result.
    c = Case(M, 1024, 2048, 5, 16)
    want = c.run(abi)
    p = abi.lora_problem(c.M, c.K, c.N, c.L, c.r, c.dtype)
    streams = [torch.cuda.Stream(), torch.cuda.Stream(priority=-1)]
    ws = [abi.lora_workspace(p) for _ in streams]
    outs = [[torch.empty_like(want) for _ in range(20)] for _ in streams]
    torch.cuda.synchronize()
    for i in range(20):
        for s, w, out in zip(streams, ws, outs):
            with torch.cuda.stream(s):
                abi.lora_forward(p, c.X, c.W, c.A, c.B, c.adapter, out[i], w, scale=c.scale)
    torch.cuda.synchronize()
    assert all(abi.device_error(w) == 0 for w in ws)
    assert all(torch.equal(o, want) for out in outs for o in out)


def test_a_larger_batch_s_workspace(abi):
    # One workspace for a server's largest batch, whatever path a batch takes.
    big, small = Case(300, 256, 384, 3, 16), Case(20, 256, 384, 3, 16, seed=1)
    want, want_small = big.run(abi), small.run(abi)
    ws = abi.lora_workspace(abi.lora_problem(300, 256, 384, 3, 16, BF16))
    for _ in range(2):
        assert torch.equal(small.run(abi, ws=ws), want_small)
        assert torch.equal(big.run(abi, ws=ws), want)


def test_no_rows(abi):
    c = Case(0, 64, 64, 2, 8)
    assert c.run(abi, Y=torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")).numel() == 0


def test_layer_and_projection_together(abi):
    # A decode step as a server runs it: the few-token layer, and beside it a projection of the
    # same activations with each request's adapter, added to the layer's output in place.
    from top_routing_expert_fp32_b200 import inputs
    cfg = configs.MoEConfig("together", N=24, D=512, F=1024, E=8, k=2, dtype=BF16, activation=0,
                            renormalize=1)
    inp = inputs.make_inputs(cfg, "cuda")
    layer = abi.Layer(cfg)
    c = Case(cfg.N, cfg.D, cfg.D, 6, 16, none=0.2)
    c.X = inp.X
    out = layer.forward_few(inp.X, inp.W_r, inp.bias, inp.W1, inp.W2, inp.W3)
    c.addend = out.clone()
    p = abi.lora_problem(c.M, c.K, c.N, c.L, c.r, c.dtype)
    ws = abi.lora_workspace(p)
    abi.lora_forward(p, c.X, c.W, c.A, c.B, c.adapter, out, ws, scale=c.scale, addend=out)
    torch.cuda.synchronize()
    assert abi.device_error(ws) == 0 and abi.device_error(layer.ws) == 0
    c.check(out)


@pytest.mark.parametrize("M", [4, 200])
def test_an_adapter_past_32_bit_offsets(abi, M):
    # The last adapter lies past 2^31 elements: the same bits as that adapter alone.
    K, N, L, r = 14336, 256, 1216, 128
    assert (L - 1) * K * r > 2 ** 31
    one = Case(M, K, N, 1, r, scale=False)
    want = one.run(abi)
    A = torch.zeros((L, K, r), dtype=torch.bfloat16, device="cuda")
    B = torch.zeros((L, r, N), dtype=torch.bfloat16, device="cuda")
    A[L - 1], B[L - 1] = one.A[0], one.B[0]
    one.A, one.B, one.L = A, B, L
    one.adapter = torch.full_like(one.adapter, L - 1)
    assert torch.equal(one.run(abi), want)
