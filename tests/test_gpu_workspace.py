"""GPU: batches that the few-token form does not take run within a workspace that has no room for
it, and write nowhere else."""
import pytest
import torch

from top_routing_expert_fp32_b200 import configs, inputs

pytestmark = pytest.mark.gpu


def test_a_large_batch_in_its_own_regions():
    from top_routing_expert_fp32_b200 import abi
    cfg = configs.MoEConfig("own", N=512, D=256, F=512, E=8, k=2, dtype=configs.DTYPE_BF16,
                            activation=0, renormalize=1)
    p = abi.problem(cfg)
    inp = inputs.make_inputs(cfg, "cuda")
    want = abi.Layer(cfg).forward(inp.X, inp.W_r, inp.bias, inp.W1, inp.W2, inp.W3)
    own, x = 2158336, cfg.N * cfg.D * 2  # router, dispatch, X_perm, H, Y; one buffer of X or out
    assert own + 4 * x < abi.workspace_size(p)
    pad = 4096
    for size in (own, own + 4 * x):
        buf = torch.full((size + 2 * pad,), 0x5A, dtype=torch.uint8, device="cuda")
        buf[pad:pad + 256] = 0  # the header
        ws = buf[pad:pad + size]
        if size == own:
            out = torch.empty_like(inp.X)
            abi.forward(p, inp.X, inp.W_r, inp.bias, inp.W1, inp.W2, inp.W3, out, ws)
        else:
            host = torch.empty(inp.X.shape, dtype=inp.X.dtype, pin_memory=True)
            abi.forward_host(p, inp.X.cpu().pin_memory(), inp.W_r, inp.bias, inp.W1, inp.W2,
                             inp.W3, host, ws)
            torch.cuda.synchronize()
            out = host.cuda()
        torch.cuda.synchronize()
        assert abi.device_error(ws) == 0
        assert torch.equal(out, want)
        assert (buf[:pad] == 0x5A).all() and (buf[-pad:] == 0x5A).all()
