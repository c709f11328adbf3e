"""The embedding's gradients on small tables, whose rows and columns go to more
workgroups: widths on both sides of a wave's columns, runs of every length
that ends a batch of rows, words without tokens."""
import pytest
import torch

from gpu_util import DEV
from ring_allreduce_reduction_02_amd import ccgpu
from test_gpu_model import HALF, U, draw_ids, gen, grad_reference, ints, near, ranks, say

pytestmark = pytest.mark.gpu

# (ranks, tokens, vocab, width, ids)
TABLES = [(3, 740, 74, 192, "zipf"), (1, 700, 60, 2048, "zipf"), (2, 3000, 100, 1500, "zipf"), (2, 1000, 500, 1001, "random"),
          (8, 257, 300, 513, "zipf"), (1, 50, 2, 257, "random"), (4, 300, 700, 1025, "zipf"), (1, 2000, 1100, 520, "zipf")]


def runs_of(N, V):
    """Word v has v tokens on every rank, in an order that mixes the words."""
    ids = torch.repeat_interleave(torch.arange(V), torch.arange(V)).int()
    mix = torch.randperm(len(ids), generator=torch.Generator().manual_seed(3))
    return ids[mix].to(DEV).repeat(N, 1)


def check(ids, V, D, dtype, summed, seed):
    N, T = ids.shape
    grad = ranks(N, T * D, dtype, 8, 0, torch.randn((N, T, D), generator=gen(seed), device=DEV))
    out = ranks(N, V * D, dtype, 16)
    ws = ccgpu.make_embedding_grad_workspace(N, V, T, D)
    ws.fill_(0xFF)
    f = ccgpu.all_reduce_embedding_grad if summed else ccgpu.embedding_grad
    f(grad, ids, out, D, scale=0.75, workspace=ws)
    torch.cuda.synchronize()
    d, a, n = grad_reference(grad, ids, V, D, 0.75, summed)
    # n - 1 additions and one product in float32 (each off by at most U of the magnitudes' sum), one rounding
    near(out.reshape(N, V, D), d, (n + 1) * U * 1.01 * a + HALF[dtype] * (d.abs() + (n + 1) * U * a) * 1.01 + 1e-38, "dtable")


@pytest.mark.parametrize("summed", [False, True], ids=["rank", "sum"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("case", TABLES, ids=str)
def test_small_tables(case, dtype, summed):
    N, T, V, D, kind = case
    say("embedding_grad", case, dtype, summed)
    ids = ints(N, T, 3)
    ids.copy_(draw_ids(N, T, V, kind, gen(T)))
    check(ids, V, D, dtype, summed, V)


@pytest.mark.parametrize("summed", [False, True], ids=["rank", "sum"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("width", [9, 260, 516, 1032])
def test_every_run_length(width, dtype, summed):
    """Words of 0 to 69 tokens: every rest of a batch, one wave's rows and four waves'."""
    say("embedding_grad runs", width, dtype, summed)
    check(runs_of(2, 70), 70, width, dtype, summed, width)
