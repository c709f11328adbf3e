"""The experts' feed-forward block on rows that are no whole 16-byte vectors and
are copied into padded ones: residues of both widths, experts without rows, a
workspace full of NaN, and rows that must not reach others."""
import math

import pytest
import torch

from gpu_util import DEV
from ring_allreduce_reduction_02_amd import ccgpu
from test_gpu_model import Ffn, say, spread

pytestmark = pytest.mark.gpu


def run(f, act):
    """Both passes, on workspaces that hold NaN in either type."""
    for grad in (False, True):
        ws = ccgpu.make_moe_ffn_workspace(f.counts, f.cap, f.W, f.F, f.dtype, grad=grad)
        ws.fill_(0xFF)
        if grad:
            ccgpu.moe_ffn_grad(f.x, f.w_in, f.w_out, f.pre, f.dy, f.dx, f.dw_in, f.dw_out, f.counts, f.cap, f.W, act=act,
                               workspace=ws)
        else:
            ccgpu.moe_ffn(f.x, f.w_in, f.w_out, f.y, f.counts, f.cap, f.W, pre=f.pre, act=act, workspace=ws)
    torch.cuda.synchronize()


def check(f, act):
    f.check_forward(act)
    f.check_backward(act)
    f.check_untouched()


# small: gradients only are copied; either width whole vectors, neither, 2 * hidden alone (132, 66)
SMALL = [(2, 4, 9, w, f, spread(2, 4, 9, 20 + w + f, 12)) for w in (1, 7, 64, 65, 127, 130) for f in (1, 9, 66, 132, 64)
         if w % 8 or f % 8]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("case", SMALL, ids=lambda c: f"{c[3]}x{c[4]}")
def test_residues(case, dtype):
    say("copies", case, dtype)
    f = Ffn(*case, dtype, 31, pad=5, offset=1)
    run(f, "silu")
    check(f, "silu")


# 1024 rows an expert or more, on average: the forward pass copies too
LARGE = [(2, 2, 1100, 515, 521, [[1024, 1024], [1023, 1025]]), (1, 3, 2000, 520, 513, [[1500, 0, 1700]]),
         (2, 2, 1030, 521, 512, [[1030, 1], [1027, 2000]]), (1, 1, 1024, 513, 514, [[1024]]), (1, 1, 1024, 513, 514, [[1023]])]


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("case", LARGE, ids=lambda c: f"{c[:5]}-{c[5][0][0]}")
def test_both_passes(case, dtype, act):
    say("copies", case, dtype, act)
    f = Ffn(*case, dtype, 32)
    run(f, act)
    check(f, act)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_nan_stays_in_its_rows(dtype):
    """NaN in one expert's weights and in single rows changes no row of another expert and no other row of y and dx."""
    f = Ffn(1, 3, 70, 61, 31, [[70, 0, 33]], dtype, 33)
    run(f, "silu")
    y, dx, dw = f.y.clone(), f.dx.clone(), f.dw_in.clone()
    f.w_in.view(3, -1)[1], f.w_out.view(3, -1)[1] = math.nan, math.nan          # the expert without rows
    f.x.view(210, 61)[3], f.dy.view(210, 61)[51, 60] = math.nan, math.inf
    run(f, "silu")
    for new, old, bad in ((f.y, y, (3,)), (f.dx, dx, (3, 51))):
        ok = torch.ones(210, dtype=torch.bool, device=DEV)
        ok[list(bad)] = False
        assert torch.equal(new.view(210, 61)[ok], old.view(210, 61)[ok])
    assert torch.equal(f.dw_in.view(3, -1)[1:], dw.view(3, -1)[1:])
    assert (f.dw_in.view(3, -1)[1] == 0).all() and torch.isnan(f.dw_in.view(3, -1)[0]).any()
