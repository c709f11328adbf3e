"""The gradient of the balance loss at padding tokens, on the GPU."""
import math

import pytest
import torch

from gpu_util import DEV
from ring_allreduce_reduction_02_amd import ccgpu
from test_gpu_balance import forward
from test_gpu_model import draw_logits, gen, ranks, say

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("up", [math.inf, -math.inf, math.nan], ids=str)
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("E", [3, 16, 64, 100, 1024])
def test_padding_rows_are_base_at_any_dloss(E, dtype, up):
    """A token without a logit has no gradient, also where the loss's own is not finite: 0, or the base's bits."""
    N, T = 2, 19
    say("padding rows", E, dtype, up)
    z = draw_logits(N, T, E, dtype, 5, False)
    z[:, 3], z[1, 11:] = -math.inf, -math.inf
    logits = ranks(N, T * E, dtype, 3, 1, z)
    dead = torch.zeros(N, T, dtype=torch.bool, device=DEV)
    dead[:, 3], dead[1, 11:] = True, True
    total, _, _ = forward(logits, torch.ones(N, E, dtype=torch.int32, device=DEV), N, T, E, False)
    dloss = torch.tensor([[1.0], [up]], device=DEV)
    out = ranks(N, T * E, dtype, 5, 1)
    ccgpu.moe_balance_loss_grad(logits, total, dloss, out)
    torch.cuda.synchronize()
    assert not out.reshape(N, T, E)[dead].any()
    assert not torch.isnan(out[0]).any()
    base = ranks(N, T * E, dtype, 2, 1, torch.randn((N, T, E), generator=gen(1), device=DEV))
    base[0, 3 * E], base[1, 3 * E] = math.inf, math.nan              # a base is passed on whatever it holds
    was = base.clone().reshape(N, T, E)
    ccgpu.moe_balance_loss_grad(logits, total, dloss, out, base=base)
    ccgpu.moe_balance_loss_grad(logits, total, dloss, base, base=base)
    torch.cuda.synchronize()
    for got in (out, base):
        bits = torch.int16 if dtype == "bf16" else torch.int32
        assert torch.equal(got.reshape(N, T, E)[dead].view(bits), was[dead].view(bits))
