"""The expert feed-forward block in every tile size and form of its products
(a host test shows which of them each case takes), forward and gradients,
against plain 64-bit implementations, and once more on another workspace for
the same bits."""
import pytest
import torch

from model_tiles import CASES
from test_gpu_model import Ffn, say
from test_gpu_model_copies import run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("name", CASES)
def test_tiles(name, dtype):
    case, offset = CASES[name]
    act = "gelu" if name.startswith("c") else "silu"
    say("tiles", name, dtype)
    f = Ffn(*case, dtype, 41, offset=offset)
    run(f, act)
    f.check_forward(act)
    f.check_backward(act)
    f.check_untouched()
    outs = (f.y, f.pre, f.dx, f.dw_in, f.dw_out)
    first = [t.clone() for t in outs]
    for t in outs:
        t.fill_(7.0)
    f.forward(act)                      # workspaces with other contents
    f.backward(act)
    torch.cuda.synchronize()
    for t, was in zip(outs, first):
        assert torch.equal(t, was)
