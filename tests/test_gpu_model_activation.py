"""SiLU and its derivative inside the float32 feed-forward block, element by
element over [-87, 87], against 64-bit values.  With x = [g, 1, 0 ..], gate rows
[1, 0 ..], up rows [0, 1, 0 ..] and an identity behind them every product is
exact, so y holds silu(g) and dx = [silu'(g), silu(g), 0 ..] as the block
computed them.

Relative error, U half a step of float32: with e = exp(-|g|) (one step, 2 U),
r = 1 / (1 + e) is off by 2 U e / (1 + e) <= U of e, U of the sum and U of the
quotient; e r by 2 U + 3 U + U.  So the sigmoid s and its complement c are off
by at most 6 U, g s by 7 U, and s (1 + g c) by s (7 U |g c| + U |1 + g c|)
before a product that adds 6 U + U."""
import pytest
import torch

from gpu_util import DEV
from ring_allreduce_reduction_02_amd import ccgpu
from test_gpu_model import U, near, say

pytestmark = pytest.mark.gpu


def sweep():
    """g on a grid, dense at 0, and next to the values where exp changes its reduced argument."""
    g = torch.linspace(-87.0, 87.0, 8192, dtype=torch.float64)
    k = torch.arange(-125, 126, dtype=torch.float64) * 0.6931471805599453
    return torch.cat([g, k, k + 1e-5, k - 1e-5, g / 87, g * 1e-6, torch.tensor([0.0, -44.866, 44.866])]).clamp(-87, 87).float().to(DEV)


@pytest.mark.parametrize("width", [2, 4], ids=["any rows", "whole vectors"])
def test_silu_float32(width):
    say("silu", width)
    g = sweep()
    R, W, F = len(g), width, width // 2 if width == 2 else 4
    x = torch.zeros(R, W, device=DEV)
    x[:, 0], x[:, 1] = g, 1.0
    w_in = torch.zeros(2 * F, W, device=DEV)
    w_in[:F, 0], w_in[F:, 1] = 1.0, 1.0
    w_out = torch.eye(W, F, device=DEV)
    dy = torch.zeros(R, W, device=DEV)
    dy[:, 0] = 1.0
    x, dy, w_in, w_out = (t.reshape(1, -1) for t in (x, dy, w_in, w_out))
    pre, y, dx = torch.empty(1, R * 2 * F, device=DEV), torch.empty_like(x), torch.empty_like(x)
    counts = [[R]]
    ccgpu.moe_ffn(x, w_in, w_out, y, counts, R, W, pre=pre, act="silu",
                  workspace=ccgpu.make_moe_ffn_workspace(counts, R, W, F, "f32"))
    ccgpu.moe_ffn_grad(x, w_in, w_out, pre, dy, dx, torch.empty_like(w_in), torch.empty_like(w_out), counts, R, W, act="silu",
                       workspace=ccgpu.make_moe_ffn_workspace(counts, R, W, F, "f32", grad=True))
    torch.cuda.synchronize()
    assert torch.equal(pre.view(R, 2 * F)[:, 0], g)
    z = g.double()
    s, c = torch.sigmoid(z), torch.sigmoid(-z)
    a, d = z * s, s * (1 + z * c)
    near(y.view(R, W)[:, 0], a, 7.1 * U * a.abs(), "silu")
    near(dx.view(R, W)[:, 1], a, 7.1 * U * a.abs(), "silu of the gradient")
    near(dx.view(R, W)[:, 0], d, U * 1.01 * (7 * s * (z * c).abs() + 8 * d.abs()), "derivative")
