"""8-bit products with many large weights for few rows, on the GPU."""
import pytest
import torch

from gpu_util import DEV
from ring_allreduce_reduction_02_amd import ccgpu
from test_gpu_model import HALF, TORCH_DT, U, gen, near, say

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("W", [3, 16])
def test_many_experts_of_many_columns(W, dtype):
    """8192 experts of 65536 columns, of which four have rows: 4096 tiles, where their weights' gradients would be 2^24."""
    E, C, live = 8192, 65536, {0: 1, 17: 1, 4097: 1, 8191: 1}
    say("8-bit product of many experts", W, dtype)
    counts = [[live.get(e, 0) for e in range(E)]]
    g = gen(W)
    w = torch.zeros(1, E * C * W, dtype=torch.int8, device=DEV)
    x = torch.randint(-127, 128, (1, E * W), generator=g, device=DEV, dtype=torch.int8)
    sx, sw = torch.rand(1, E, generator=g, device=DEV), torch.zeros(1, E * C, device=DEV)
    for e in live:
        w.view(E, C, W)[e] = torch.randint(-127, 128, (C, W), generator=g, device=DEV, dtype=torch.int8)
        sw.view(E, C)[e] = torch.rand(C, generator=g, device=DEV)
    y = torch.full((1, E * C), 7.0, dtype=TORCH_DT[dtype], device=DEV)
    ccgpu.moe_matmul_int8(x, sx, w, sw, y, counts, 1, W, workspace=ccgpu.make_moe_matmul_int8_workspace(counts, 1, W, C))
    torch.cuda.synchronize()
    for e in live:
        want = (w.view(E, C, W)[e].double() @ x.view(E, W)[e].double()) * sx[0, e].double() * sw.view(E, C)[e].double()
        near(y.view(E, C)[e], want, (3.01 * U + HALF[dtype] * 1.01) * want.abs() + 1e-38, f"y of expert {e}")
        y.view(E, C)[e] = 7.0
    assert (y == 7.0).all()
