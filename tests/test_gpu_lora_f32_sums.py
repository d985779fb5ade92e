"""fp32 sums of moe_lora_forward: runs of at most 64 terms whose sums are added up, whatever K and
the rank. Tolerances: beside the output's own rounding (2^-24 of it), a chain of n additions of
terms of one sign errs by at most n 2^-24 of the sum; terms of random signs by about sqrt(n) 2^-24
of their 2-norm, which 1e-5 of a row's largest value covers with room."""
import pytest
import torch

from top_routing_expert_fp32_b200 import configs

pytestmark = pytest.mark.gpu

F32 = configs.DTYPE_F32


@pytest.fixture(scope="module")
def abi():
    from top_routing_expert_fp32_b200 import abi as a
    return a


def _call(abi, X, W, A, B, adapter):
    M, K = X.shape
    p = abi.lora_problem(M, K, W.shape[1], A.shape[0], A.shape[2], F32)
    ws = abi.lora_workspace(p)
    Y = torch.empty((M, W.shape[1]), device="cuda")
    abi.lora_forward(p, X, W, A, B, adapter, Y, ws)
    torch.cuda.synchronize()
    assert abi.device_error(ws) == 0
    return Y


@pytest.mark.parametrize("M", [64, 33, 1, 65, 130])
def test_fp32_shrink_in_short_runs(abi, M):
    # S = X A of K equal terms, whose fp32 sum in one run drifts: 3584 terms of 0.1 by 3.5e-5. In
    # runs of 64 whose sums are added up (at most 56 of them per thread here, then a few partial
    # sums): (64 + 56 + 64) 2^-24 = 1.1e-5 at the very most. B is the identity and W is zero, so
    # that Y is S itself.
    K, r = 14336, 128
    X = torch.ones((M, K), device="cuda")
    A = torch.full((1, K, r), 0.1, device="cuda")
    B = torch.eye(r, device="cuda").reshape(1, r, r).contiguous()
    W = torch.zeros((K, r), device="cuda")
    adapter = torch.zeros(M, dtype=torch.int32, device="cuda")
    Y = _call(abi, X, W, A, B, adapter).double()
    ref = K * A[0, 0, 0].double().item()
    assert ((Y - ref).abs() <= (64 + 56 + 64) * 2.0 ** -24 * ref).all()


@pytest.mark.parametrize("M", [64, 130])
def test_fp32_many_terms_and_ranks(abi, M):
    # K and the rank both large, in the terms of the formula: 1e-5 of a row's largest value.
    K, N, L, r = 14336, 132, 3, 128
    g = torch.Generator(device="cuda")
    g.manual_seed(M)
    rnd = lambda shape, std: torch.randn(shape, generator=g, device="cuda") * std
    X, W, A, B = rnd((M, K), 1.0), rnd((K, N), K ** -0.5), rnd((L, K, r), K ** -0.5), \
        rnd((L, r, N), r ** -0.5)
    adapter = torch.randint(0, L, (M,), generator=g, device="cuda", dtype=torch.int32)
    Y = _call(abi, X, W, A, B, adapter).double()
    ref = X.double() @ W.double()
    for a in range(L):
        rows = (adapter == a).nonzero()[:, 0]
        ref[rows] += X[rows].double() @ A[a].double() @ B[a].double()
    assert ((Y - ref).abs() <= 2.0 ** -24 * ref.abs()
            + 1e-5 * ref.abs().amax(1, keepdim=True)).all()
