"""How many bits moe_lora_forward keeps of the adapters' part: the same above 64 rows as up to them.

Tolerances. The output is rounded once: 2^-8 of the value. scale X A enters the product with
B as two bf16 terms: the first is off by at most 2^-8 of it, the second by at most 2^-8 of that, so
2^-16 sum_r |S_r| |B_rn|. The fp32 sums of n <= 2^11 terms err by a few sqrt(n) 2^-23 of the terms'
2-norm (tensor cores truncate), 1e-5 at most of a row's largest value per sum: 5e-5 covers the
three in a row (X A, X W, S B) with room."""
import pytest
import torch

from top_routing_expert_fp32_b200 import configs

pytestmark = pytest.mark.gpu

BF16 = configs.DTYPE_BF16


@pytest.fixture(scope="module")
def abi():
    from top_routing_expert_fp32_b200 import abi as a
    return a


def _call(abi, X, W, A, B, adapter, dtype, scale=None):
    M, K = X.shape
    p = abi.lora_problem(M, K, W.shape[1], A.shape[0], A.shape[2], dtype)
    ws = abi.lora_workspace(p)
    Y = torch.empty((M, W.shape[1]), dtype=X.dtype, device="cuda")
    abi.lora_forward(p, X, W, A, B, adapter, Y, ws, scale=scale)
    torch.cuda.synchronize()
    assert abi.device_error(ws) == 0
    return Y


@pytest.mark.parametrize("M,K,N,L,r,run", [
    (64, 512, 512, 9, 16, 1), (65, 512, 512, 9, 16, 1), (65, 64, 72, 3, 8, 1),
    (130, 264, 520, 70, 24, 1), (300, 512, 1000, 5, 32, 7), (97, 328, 264, 4, 40, 3),
    (520, 256, 392, 40, 48, 1), (200, 1024, 264, 5, 64, 33), (129, 136, 520, 20, 72, 1),
    (600, 264, 1032, 7, 128, 50), (2560, 512, 4096, 300, 16, 1), (2500, 264, 4104, 8, 56, 313),
    (4000, 128, 3000, 5, 104, 64), (1100, 136, 9216, 6, 80, 90)])
def test_the_adapters_part_keeps_16_bits(abi, M, K, N, L, r, run):
    g = torch.Generator(device="cuda")
    g.manual_seed(M * 131 + r)
    rnd = lambda shape, std: (torch.randn(shape, generator=g, device="cuda") * std).bfloat16()
    X, W = rnd((M, K), 1.0), rnd((K, N), 0.1 * K ** -0.5)
    A, B = rnd((L, K, r), K ** -0.5), rnd((L, r, N), r ** -0.5)  # most of the result
    scale = torch.rand((L,), generator=g, device="cuda") + 0.5
    ids = torch.randint(-1, L, (-(-M // run),), generator=g, device="cuda", dtype=torch.int32)
    adapter = ids.repeat_interleave(run)[:M].contiguous()
    Y = _call(abi, X, W, A, B, adapter, BF16, scale).double()

    x = X.double()
    ref, spread = x @ W.double(), torch.zeros((M, N), device="cuda", dtype=torch.float64)
    for a in range(L):
        rows = (adapter == a).nonzero()[:, 0]
        s = (x[rows] @ A[a].double()) * scale[a].double()
        ref[rows] += s @ B[a].double()
        spread[rows] = s.abs() @ B[a].double().abs()
    bound = 2.0 ** -8 * ref.abs() + 2.0 ** -16 * spread + 5e-5 * ref.abs().amax(1, keepdim=True)
    worst = ((Y - ref).abs() - bound).max().item()
    assert worst <= 0, f"over the bound by {worst:.3g} (largest {ref.abs().max().item():.3g})"
