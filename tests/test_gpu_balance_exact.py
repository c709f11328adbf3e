"""The balance loss on the GPU where its sums are exact, so that every token shows."""
import math

import numpy as np
import pytest
import torch

from gpu_util import DEV
from test_gpu_balance import forward
from test_gpu_model import TORCH_DT, gen, say

pytestmark = pytest.mark.gpu

# tokens around whole groups and workgroups of every number of lanes, long batches, many ranks
EXACT = [(1, 1, 1), (1, 511, 16), (1, 513, 16), (2, 1025, 5), (3, 257, 61), (1, 65 * 256 + 1, 33), (2, 40001, 16), (1, 300007, 3),
         (8, 4099, 64), (8, 32768, 256), (1, 70001, 200), (2, 9001, 300), (2, 5003, 700), (1, 4097, 1024), (64, 33, 9)]


@pytest.mark.parametrize("summed", [True, False], ids=["all", "own"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("case", EXACT, ids=str)
def test_every_token_counts_once(case, dtype, summed):
    """Logits that are equal at 1, 2 or 4 experts and -inf elsewhere: probabilities 1, 1/2 and 1/4, whose float32 sums
    are exact in any order below 2^22, so that P_e is their quotient rounded once.  A token that were left out, or
    counted twice, would show by a quarter."""
    N, T, E = case
    say("exact sums", case, dtype, summed)
    g = gen(T + E)
    many = torch.tensor([1, 2, 4], device=DEV)[torch.randint(0, 3, (N, T), generator=g, device=DEV)].clamp(max=E)
    many = torch.where(many == 3, 2, many)                               # (three experts of three are no power of two)
    first = torch.randint(0, E, (N, T), generator=g, device=DEV)
    z = torch.full((N, T, E), -math.inf, device=DEV)
    level = torch.randint(-3, 4, (N, T), generator=g, device=DEV).float()
    for k in range(4):
        on = many > k
        r, t = on.nonzero(as_tuple=True)
        z[r, t, (first[r, t] + k * max(1, E // 4)) % E if E >= 4 else (first[r, t] + k) % E] = level[r, t]
    pad = torch.rand((N, T), generator=g, device=DEV) < 0.05
    z[pad] = -math.inf
    logits = z.to(TORCH_DT[dtype]).reshape(N, T * E).contiguous()
    counts = torch.randint(0, 1000, (N, E), generator=g, device=DEV, dtype=torch.int32)
    total, prob, loss = forward(logits, counts, N, T, E, summed)
    torch.cuda.synchronize()
    live = z > -math.inf
    n = live.sum(-1, keepdim=True)
    p = torch.where(live, 1.0 / n.clamp(min=1).double(), 0.0).sum(1).cpu().numpy()            # multiples of a quarter
    tok, c = (n[..., 0] > 0).sum(1).cpu().numpy(), counts.cpu().numpy().astype(np.int64)
    if summed:
        p, tok, c = (np.broadcast_to(a.sum(0, keepdims=True), a.shape) for a in (p, tok, c))
    assert np.array_equal(total.cpu().numpy(), np.concatenate([c, tok[:, None]], 1))
    want = p.astype(np.float32) / np.maximum(tok, 1).astype(np.float32)[:, None]
    assert np.array_equal(prob.cpu().numpy(), want)
    f = c / np.maximum(c.sum(1, keepdims=True), 1)
    want = E * (f * want.astype(np.float64)).sum(1)
    # f rounded twice, its product once, at most E additions and the factor E
    assert (np.abs(loss.cpu().numpy()[:, 0] - want) <= (E + 5) * 2.0 ** -24 * want).all()
