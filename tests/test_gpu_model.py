"""Embedding, MoE routing and the experts' gated feed-forward block on the GPU
against plain 64-bit implementations, at the sizes and masks where they can go
wrong.  Integer results are compared exactly; each tolerance is an error bound
of the operation: half a step of the result's type for its one rounding, one
step of float32 for each float32 operation on the way."""
import math
import sys

import numpy as np
import pytest
import torch

from gpu_util import DEV, TORCH_DT, alloc_ranks
from ring_allreduce_reduction_02_amd import ccgpu

pytestmark = pytest.mark.gpu
U = 2.0 ** -24                                   # half a step of float32, relative
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}    # half a step of the result's type


def say(*a):
    print(*a, flush=True)
    sys.stdout.flush()


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def ranks(N, L, dtype, pad=0, offset=0, data=None, poison=float("nan")):
    """A rank-strided [N, L] buffer whose padding holds `poison`."""
    t = alloc_ranks(N, L, dtype, pad, offset, fill=None if dtype == "int32" else poison)
    if data is not None:
        t.copy_(data.reshape(N, L).to(TORCH_DT[dtype]))
    return t


def ints(N, L, pad=0, fill=-77):
    return alloc_ranks(N, L, "int32", pad, 0, fill=fill)


def near(got, want, bound, what):
    """|got - want| <= bound, element by element, in float64; NaN matches NaN."""
    got = got.double()
    nan = torch.isnan(want)
    assert torch.equal(torch.isnan(got), nan), f"{what}: NaN in other places"
    err = torch.where(nan, 0.0, (got - want).abs())
    over = err > torch.where(nan, 0.0, bound)
    assert not over.any(), (what, int(over.sum()), float((err / bound.clamp(min=1e-300))[over].max()))


# ------------------------------------------------------------------ embedding

# (ranks, tokens, vocab, width, pad, offset, shared table)
LOOKUPS = [(1, 1, 1, 1, 0, 0, False), (2, 5, 7, 8, 0, 0, False), (3, 33, 100, 515, 3, 1, False),
           (8, 4, 1000, 2048, 16, 0, True), (4, 257, 50, 264, 8, 8, False), (2, 3, 11, 4097, 0, 0, True),
           (64, 2, 9, 24, 0, 0, False), (2, 3, 11, 16384, 0, 0, False)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("case", LOOKUPS, ids=str)
def test_embedding(case, dtype):
    N, T, V, D, pad, off, shared = case
    say("embedding", case, dtype)
    g = gen(sum(case[:4]))
    table = ranks(1 if shared else N, V * D, dtype, pad, off, torch.randn((1 if shared else N, V, D), generator=g, device=DEV))
    if shared:
        table = table.expand(N, V * D)
    ids = ints(N, T, pad)
    ids.copy_(torch.randint(-2, V + 2, (N, T), generator=g, device=DEV, dtype=torch.int32))
    ids[0, 0] = V - 1
    if T > 2:
        ids[-1, 1:3] = torch.tensor([2 ** 31 - 1, -2 ** 31], device=DEV)
    out = ranks(N, T * D, dtype, pad, off)
    ccgpu.embedding(table, ids, out, D, scale=1.7)
    torch.cuda.synchronize()
    s = float(np.float32(1.7))
    at = ids.long()
    rows = torch.stack([table[r].reshape(V, D)[at[r].clamp(0, V - 1)] for r in range(N)]).float() * s
    want = torch.where(((at >= 0) & (at < V))[:, :, None], rows, 0.0).to(TORCH_DT[dtype])
    assert torch.equal(out.reshape(N, T, D), want)          # one product, one rounding: the same bits


def grad_reference(grad, ids, V, D, scale, summed):
    """The gradient and the sum of magnitudes, float64."""
    N, T = ids.shape
    d = torch.zeros((N, V, D), dtype=torch.float64, device=DEV)
    a = torch.zeros_like(d)
    n = torch.zeros((N, V, 1), dtype=torch.float64, device=DEV)
    for r in range(N):
        ok = (ids[r] >= 0) & (ids[r] < V)
        at, g = ids[r][ok].long(), grad[r].reshape(T, D)[ok].double()
        d[r].index_add_(0, at, g)
        a[r].index_add_(0, at, g.abs())
        n[r].index_add_(0, at, torch.ones((len(at), 1), dtype=torch.float64, device=DEV))
    if summed:
        d, a, n = (x.sum(0, keepdim=True).expand(N, -1, -1) for x in (d, a, n))
    return d * scale, a * abs(scale), n


# (ranks, tokens, vocab, width, ids): every word once, one word, long runs, nothing at all
GRADS = [(1, 1, 1, 1, "random"), (2, 7, 5, 8, "random"), (3, 1023, 307, 515, "zipf"), (4, 100, 9, 264, "none"),
         (2, 3000, 40, 72, "one"), (5, 129, 1000, 2056, "random"), (8, 257, 33, 24, "zipf"), (1, 5000, 70000, 16, "zipf"),
         (64, 33, 300, 8, "random"), (2, 64, 8, 40, "runs"), (3, 1025, 256, 8, "random"), (2, 4097, 255, 12, "zipf"),
         (1, 1500, 17000000, 1, "random"), (2, 70, 3, 20000, "random")]


def draw_ids(N, T, V, kind, g):
    if kind == "none":
        return torch.full((N, T), -1, dtype=torch.int32, device=DEV)
    if kind == "one":
        return torch.full((N, T), V - 1, dtype=torch.int32, device=DEV)
    if kind == "runs":                                  # runs that start and end inside and at piece borders
        return (torch.arange(T, device=DEV, dtype=torch.int32) // 32).clamp(max=V - 1).repeat(N, 1)
    u = torch.rand((N, T), generator=g, device=DEV, dtype=torch.float64)
    ids = torch.exp(u * math.log(V + 1.0)).long() - 1 if kind == "zipf" else (u * V).long()
    ids = ids.clamp(0, V - 1).int()
    ids[torch.rand((N, T), generator=g, device=DEV) < 0.05] = -1
    ids[torch.rand((N, T), generator=g, device=DEV) < 0.05] = V
    return ids


@pytest.mark.parametrize("summed", [False, True], ids=["rank", "sum"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("case", GRADS, ids=str)
def test_embedding_grad(case, dtype, summed):
    N, T, V, D, kind = case
    say("embedding_grad", case, dtype, summed)
    g = gen(N * 31 + T)
    ids = ints(N, T, 3)
    ids.copy_(draw_ids(N, T, V, kind, g))
    grad = ranks(N, T * D, dtype, 8, 0, torch.randn((N, T, D), generator=g, device=DEV))
    out = ranks(N, V * D, dtype, 16)
    ws = ccgpu.make_embedding_grad_workspace(N, V, T, D)
    f = ccgpu.all_reduce_embedding_grad if summed else ccgpu.embedding_grad
    f(grad, ids, out, D, scale=0.75, workspace=ws)
    torch.cuda.synchronize()
    d, a, n = grad_reference(grad, ids, V, D, 0.75, summed)
    # n - 1 additions and one product in float32 (each off by at most U of the magnitudes' sum), one rounding
    near(out.reshape(N, V, D), d, (n + 1) * U * 1.01 * a + HALF[dtype] * (d.abs() + (n + 1) * U * a) * 1.01 + 1e-38, "dtable")
    again = torch.full_like(out, 3.0)
    f(grad, ids, again, D, scale=0.75, workspace=ws)
    torch.cuda.synchronize()
    assert torch.equal(out, again)                      # no sum depends on timing


def test_embedding_grad_unaligned_rows_equal_aligned_ones():
    """An offset of one element takes the element-wise path: the same sums."""
    N, T, V, D = 2, 300, 20, 64
    g = gen(5)
    ids = torch.randint(0, V, (N, T), generator=g, device=DEV, dtype=torch.int32)
    data = torch.randn((N, T, D), generator=g, device=DEV)
    ws = ccgpu.make_embedding_grad_workspace(N, V, T, D)
    res = []
    for off in (0, 1):
        out = ranks(N, V * D, "f32", 0, off)
        ccgpu.embedding_grad(ranks(N, T * D, "f32", 0, off, data), ids, out, D, workspace=ws)
        res.append(out.clone())
    torch.cuda.synchronize()
    assert torch.equal(res[0], res[1])


# ------------------------------------------------------------------ routing

def softmax64(z):
    m = z.max(-1, keepdims=True)
    with np.errstate(invalid="ignore"):
        ex = np.exp(z - np.where(np.isneginf(m), 0.0, m))
    s = ex.sum(-1, keepdims=True)
    return np.divide(ex, s, out=np.zeros_like(ex), where=s > 0)


def route_reference(z, K, normalize):
    """experts, weights, order, counts of logits z [N, T, E] (float64, no NaN or +inf)."""
    N, T, E = z.shape
    pick = np.argsort(-z, axis=-1, kind="stable")[..., :K]
    top = np.take_along_axis(z, pick, -1)
    dead = np.isneginf(top)
    w = softmax64(top) if normalize else np.take_along_axis(softmax64(z), pick, -1)
    pick = np.where(dead, -1, pick).reshape(N, T * K)
    order = np.full((N, T * K), -1, np.int64)
    counts = np.zeros((N, E), np.int64)
    for r in range(N):
        at = np.flatnonzero(pick[r] >= 0)
        order[r, :len(at)] = at[np.argsort(pick[r, at], kind="stable")]
        counts[r] = np.bincount(pick[r, at], minlength=E)
    return pick, np.where(dead, 0.0, w).reshape(N, T * K), order, counts


def draw_logits(N, T, E, dtype, seed, mask):
    g = gen(seed)
    z = torch.randn((N, T, E), generator=g, device=DEV) * 2
    z = z.to(torch.bfloat16).float()                      # ties happen
    if mask:
        z[torch.rand((N, T, E), generator=g, device=DEV) < 0.3] = -math.inf
        z[:, ::5] = -math.inf                             # rows whose mask leaves nothing
        z[:, 1::7, 1:] = -math.inf                        # and one expert
        z[:, 2::11] = torch.finfo(torch.float32 if dtype == "f32" else torch.bfloat16).min
        z[:, 3::13] = 0.0
        z[:, 3::13, ::2] = -0.0                           # equal to +0: ties to the lowest index
    return z


# (ranks, tokens, experts, topk)
ROUTES = [(1, 1, 1, 1), (2, 3, 5, 5), (8, 4, 64, 8), (3, 257, 64, 2), (2, 130, 65, 7), (4, 33, 256, 8), (1, 19, 1000, 64),
          (2, 1100, 8, 1), (1, 70, 257, 4), (2, 0, 6, 2), (64, 5, 64, 1), (1, 3000, 128, 3), (1, 9, 600, 2)]


@pytest.mark.parametrize("mask", [False, True], ids=["full", "masked"])
@pytest.mark.parametrize("normalize", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("case", ROUTES, ids=str)
def test_moe_route(case, dtype, normalize, mask):
    N, T, E, K = case
    say("moe_route", case, dtype, normalize, mask)
    z = draw_logits(N, T, E, dtype, T + E, mask)
    logits = ranks(N, T * E, dtype, 3, 1, z)
    experts, order, counts = ints(N, T * K, 1), ints(N, T * K), ints(N, E, 5)
    weights = ranks(N, T * K, "f32", 2)
    ws = ccgpu.make_moe_route_workspace(N, T, E, K)
    ccgpu.moe_route(logits, experts, weights, order, counts, K, normalize=normalize, workspace=ws)
    torch.cuda.synchronize()
    zz = logits.reshape(N, T, E).double().cpu().numpy()
    e, w, o, c = route_reference(zz, K, normalize) if T else (np.zeros((N, 0)), np.zeros((N, 0)), np.zeros((N, 0)), np.zeros((N, E)))
    assert np.array_equal(experts.cpu().numpy(), e)
    assert np.array_equal(order.cpu().numpy(), o)
    assert np.array_equal(counts.cpu().numpy(), c)
    if T:
        # exp of a difference d rounded once (d U), exp itself and the division (4 U), E additions
        d = np.where(np.isneginf(zz), 0.0, zz - np.where(np.isneginf(zz.max(-1, keepdims=True)), 0.0, zz.max(-1, keepdims=True)))
        rel = (E + 8 + 2 * np.minimum(-d.min(-1), 110.0)) * U
        bound = torch.from_numpy(np.repeat(rel.reshape(N, T, 1), K, -1).reshape(N, T * K) * w + 1e-37).to(DEV)
        near(weights, torch.from_numpy(w).to(DEV), bound, "weights")


def test_moe_route_nan_and_infinity():
    """NaN is never chosen and makes the row's weights NaN, as +inf does; -inf and NaN alone choose nothing."""
    z = torch.tensor([[1.0, math.nan, 3.0, 2.0], [math.nan] * 4, [math.inf, 0.0, 1.0, -math.inf], [-math.inf, math.nan, -math.inf, 5.0]],
                     device=DEV)
    logits = z.reshape(1, 16).contiguous()
    experts, order, counts = ints(1, 8), ints(1, 8), ints(1, 4)
    weights = torch.zeros(1, 8, device=DEV)
    ccgpu.moe_route(logits, experts, weights, order, counts, 2, workspace=ccgpu.make_moe_route_workspace(1, 4, 4, 2))
    torch.cuda.synchronize()
    assert experts.tolist() == [[2, 3, -1, -1, 0, 2, 3, -1]]
    assert torch.isnan(weights).tolist() == [[True, True, False, False, True, True, True, False]]
    assert order.tolist() == [[4, 0, 5, 1, 6, -1, -1, -1]] and counts.tolist() == [[1, 0, 2, 2]]


def route_grad_reference(z, pick, dw, normalize):
    N, T, E = z.shape
    K = pick.shape[-1]
    chosen, up = np.zeros((N, T, E), bool), np.zeros((N, T, E))
    for k in range(K):
        n, t = np.nonzero((pick[..., k] >= 0) & (pick[..., k] < E))
        chosen[n, t, pick[n, t, k]] = True
        up[n, t, pick[n, t, k]] = dw[n, t, k]
    p = softmax64(np.where(chosen, z, -np.inf)) if normalize else softmax64(z)
    dot = (p * up).sum(-1, keepdims=True)
    return p * (up - dot), p * (np.abs(up) + (p * np.abs(up)).sum(-1, keepdims=True))


@pytest.mark.parametrize("mask", [False, True], ids=["full", "masked"])
@pytest.mark.parametrize("normalize", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("case", [c for c in ROUTES if c[1]], ids=str)
def test_moe_route_grad(case, dtype, normalize, mask):
    N, T, E, K = case
    say("moe_route_grad", case, dtype, normalize, mask)
    logits = ranks(N, T * E, dtype, 3, 1, draw_logits(N, T, E, dtype, T + E + 1, mask))
    zz = logits.reshape(N, T, E).double().cpu().numpy()
    pick = route_reference(zz, K, normalize)[0].reshape(N, T, K)
    pick[pick == -1] = np.random.default_rng(3).choice([-1, E, E + 70, 2 ** 31 - 1], size=int((pick == -1).sum()))
    experts = ints(N, T * K, 2)
    experts.copy_(torch.from_numpy(pick.astype(np.int32).reshape(N, T * K)))
    dw = ranks(N, T * K, "f32", 1, 0, torch.randn((N, T * K), generator=gen(9), device=DEV))
    out = ranks(N, T * E, dtype, 5)
    ccgpu.moe_route_grad(logits, experts, dw, out, K, normalize=normalize)
    torch.cuda.synchronize()
    d, a = route_grad_reference(zz, pick, dw.double().cpu().numpy().reshape(N, T, K), normalize)
    dist = np.where(np.isneginf(zz), 0.0, zz - np.where(np.isneginf(zz.max(-1, keepdims=True)), 0.0, zz.max(-1, keepdims=True)))
    # the probabilities' bound, and E more additions in their product's sum
    rel = (3 * E + 32 + 4 * np.minimum(-dist.min(-1, keepdims=True), 110.0)) * U
    bound = rel * a + HALF[dtype] * np.abs(d) * 1.01 + 1e-37
    near(out.reshape(N, T, E), torch.from_numpy(d).to(DEV), torch.from_numpy(bound).to(DEV), "dlogits")


@pytest.mark.parametrize("normalize", [False, True])
def test_moe_route_grad_against_differences(normalize):
    """The gradient of sum(c * weights) against central differences of the 64-bit weights."""
    N, T, E, K = 1, 6, 9, 3
    rng = np.random.default_rng(4)
    z, c = rng.permutation(T * E).reshape(N, T, E) * 0.11, rng.standard_normal((N, T * K))
    logits = torch.from_numpy(z.reshape(N, T * E)).float().to(DEV)
    z = logits.double().cpu().numpy().reshape(N, T, E)
    pick = route_reference(z, K, normalize)[0]
    out = torch.empty(N, T * E, device=DEV)
    ccgpu.moe_route_grad(logits, torch.from_numpy(pick).int().to(DEV), torch.from_numpy(c).float().to(DEV), out, K, normalize=normalize)
    got, h = out.double().cpu().numpy().reshape(N, T, E), 1e-4
    for t in range(T):
        for e in range(E):
            f = []
            for s in (h, -h):
                y = z.copy()
                y[0, t, e] += s
                f.append((route_reference(y, K, normalize)[1] * c).sum())
            assert abs((f[0] - f[1]) / (2 * h) - got[0, t, e]) < 2e-6      # h^2 of third derivatives below 1, and 100 U


# ------------------------------------------------------------------ expert feed-forward

def act64(g, act):
    if act == "silu":
        s = torch.sigmoid(g)
        return g * s, s + g * s * (1 - s)
    c = 0.5 * torch.special.erfc(-g / math.sqrt(2.0))
    return g * c, c + g * torch.exp(-g * g / 2) / math.sqrt(2 * math.pi)


class Ffn:
    """The buffers of one case; rows behind the kept ones hold NaN in every input and output."""

    def __init__(self, N, E, cap, W, F, counts, dtype, seed, pad=0, offset=0):
        self.N, self.E, self.cap, self.W, self.F, self.counts, self.dtype = N, E, cap, W, F, counts, dtype
        g, per = gen(seed), E // N
        self.per = per
        self.keep = torch.zeros((N, N, per, cap), dtype=torch.bool, device=DEV)
        for i in range(N):
            for e in range(E):
                self.keep[e // per, i, e % per, :min(counts[i][e], cap)] = True
        self.keep = self.keep.reshape(N, E * cap)

        def side(width, sigma):
            d = torch.randn((N, E * cap, width), generator=g, device=DEV) * sigma
            d[~self.keep] = math.nan
            return ranks(N, E * cap * width, dtype, pad, offset, d)
        self.x, self.dy = side(W, 1.0), side(W, 1.0)
        self.w_in = ranks(N, per * 2 * F * W, dtype, pad, offset, torch.randn((N, per * 2 * F * W), generator=g, device=DEV) / math.sqrt(W))
        self.w_out = ranks(N, per * W * F, dtype, pad, offset, torch.randn((N, per * W * F), generator=g, device=DEV) / math.sqrt(F))
        self.pre = ranks(N, E * cap * 2 * F, dtype, pad, offset, poison=7.0)
        self.y, self.dx = (ranks(N, E * cap * W, dtype, pad, offset, poison=7.0) for _ in range(2))
        self.pre.fill_(7.0), self.y.fill_(7.0), self.dx.fill_(7.0)
        self.dw_in = ranks(N, per * 2 * F * W, dtype, pad, offset)
        self.dw_out = ranks(N, per * W * F, dtype, pad, offset)

    def forward(self, act, keep_pre=True, stream=None):
        ws = ccgpu.make_moe_ffn_workspace(self.counts, self.cap, self.W, self.F, self.dtype)
        ws.fill_(0xA5)
        ccgpu.moe_ffn(self.x, self.w_in, self.w_out, self.y, self.counts, self.cap, self.W,
                      pre=self.pre if keep_pre else None, act=act, workspace=ws, stream=stream)

    def backward(self, act, stream=None):
        ws = ccgpu.make_moe_ffn_workspace(self.counts, self.cap, self.W, self.F, self.dtype, grad=True)
        ws.fill_(0xA5)
        ccgpu.moe_ffn_grad(self.x, self.w_in, self.w_out, self.pre, self.dy, self.dx, self.dw_in, self.dw_out, self.counts,
                           self.cap, self.W, act=act, workspace=ws, stream=stream)

    def expert(self, e):
        """Views of expert e: its kept rows' positions and its rank."""
        j, l = e // self.per, e % self.per
        block = torch.zeros((self.N, self.per, self.cap), dtype=torch.bool, device=DEV)
        block[:, l] = True
        return j, l, (block.reshape(-1) & self.keep[j]).nonzero().view(-1)

    def rows(self, t, j, at):
        return t[j].reshape(self.E * self.cap, 2 * self.F if t is self.pre else self.W)[at].double()

    def check_untouched(self):
        for t in (self.y, self.dx, self.pre):
            b = t.reshape(self.N, self.E * self.cap, -1) if t.numel() else None
            if b is not None:
                assert (b[~self.keep] == 7.0).all(), "a row behind the kept ones was written"

    def check_forward(self, act, keep_pre=True):
        W, F, r, per = self.W, self.F, HALF[self.dtype], self.per
        for e in range(self.E):
            j, l, at = self.expert(e)
            x = self.rows(self.x, j, at)
            wi, wo = self.w_in[j].reshape(per, 2 * F, W)[l].double(), self.w_out[j].reshape(per, W, F)[l].double()
            gu, s = x @ wi.t(), (W + 1) * U * (x.abs() @ wi.abs().t())       # W additions of exact products
            if keep_pre:
                near(self.rows(self.pre, j, at), gu, s + r * 1.01 * (gu.abs() + s), f"pre of expert {e}")
            g, u, sg, su = gu[:, :F], gu[:, F:], s[:, :F], s[:, F:]
            a, _ = act64(g, act)
            h = a * u
            # the activation's slope is below 1.13; its own error is below 16 U of |g| (and 4 U)
            dh = (1.13 * sg + (16 * g.abs() + 4) * U) * (u.abs() + su) + a.abs() * su
            dh = dh + (r + 2 * U) * 1.01 * (h.abs() + dh)
            y, m = h @ wo.t(), (h.abs() + dh) @ wo.abs().t()
            err = dh @ wo.abs().t() + (F + 1) * U * m
            near(self.rows(self.y, j, at), y, err + r * 1.01 * (y.abs() + err), f"y of expert {e}")

    def check_backward(self, act):
        W, F, r, per = self.W, self.F, HALF[self.dtype], self.per
        for e in range(self.E):
            j, l, at = self.expert(e)
            x, dy, gu = self.rows(self.x, j, at), self.rows(self.dy, j, at), self.rows(self.pre, j, at)
            wi, wo = self.w_in[j].reshape(per, 2 * F, W)[l].double(), self.w_out[j].reshape(per, W, F)[l].double()
            g, u = gu[:, :F], gu[:, F:]
            a, da = act64(g, act)
            h, sh = a * u, (16 * g.abs() + 4) * U * u.abs()
            sh = sh + (r + 2 * U) * 1.01 * (h.abs() + sh)
            dh, s = dy @ wo, (W + 1) * U * (dy.abs() @ wo.abs())
            ea = (16 * g.abs() + 8) * U                                         # of the activation and its derivative
            ga, gb = dh * u * da, dh * a
            eg = s * u.abs() * (da.abs() + ea) + (dh * u).abs() * ea
            eb = s * (a.abs() + ea) + dh.abs() * ea
            d = torch.cat([ga, gb], 1)
            ed = torch.cat([eg, eb], 1)
            ed = ed + (r + 3 * U) * 1.01 * (d.abs() + ed)
            dx = d @ wi
            err = ed @ wi.abs() + (2 * F + 1) * U * ((d.abs() + ed) @ wi.abs())
            near(self.rows(self.dx, j, at), dx, err + r * 1.01 * (dx.abs() + err), f"dx of expert {e}")
            n = len(at) + 1
            dwo = dy.t() @ h
            err = dy.abs().t() @ sh + n * U * (dy.abs().t() @ (h.abs() + sh))
            near(self.dw_out[j].reshape(per, W, F)[l], dwo, err + r * 1.01 * (dwo.abs() + err) + 1e-38, f"dw_out of expert {e}")
            dwi = d.t() @ x
            err = ed.t() @ x.abs() + n * U * ((d.abs() + ed).t() @ x.abs())
            near(self.dw_in[j].reshape(per, 2 * F, W)[l], dwi, err + r * 1.01 * (dwi.abs() + err) + 1e-38, f"dw_in of expert {e}")


def spread(N, E, cap, seed, most):
    rng = np.random.default_rng(seed)
    return [[int(v) for v in rng.integers(0, most + 1, size=E)] for _ in range(N)]


# (ranks, experts, capacity, width, hidden, counts): one row, one column, odd and ragged sizes, rows dropped at
# the capacity, experts and ranks without rows, row counts on both sides of every tile
FFNS = [(1, 1, 1, 1, 1, [[1]]), (1, 1, 3, 8, 8, [[2]]), (1, 2, 5, 16, 24, [[0, 4]]), (2, 4, 7, 33, 17, spread(2, 4, 7, 1, 9)),
        (1, 1, 128, 64, 64, [[128]]), (1, 1, 129, 72, 136, [[129]]), (2, 2, 300, 128, 64, [[300, 0], [1, 0]]),
        (3, 6, 40, 130, 66, spread(3, 6, 40, 2, 60)), (8, 8, 33, 264, 200, spread(8, 8, 33, 3, 33)),
        (2, 2, 16, 515, 331, spread(2, 2, 16, 4, 16)), (4, 8, 0, 16, 16, spread(4, 8, 1, 5, 3)), (2, 4, 6, 24, 40, [[0] * 4] * 2),
        (1, 1, 600, 136, 520, [[577]]), (1, 3, 260, 512, 256, [[256, 257, 255]]), (2, 2, 20, 1032, 1288, [[20, 1], [17, 0]]),
        (16, 64, 2, 64, 48, spread(16, 64, 2, 6, 3)), (1, 4, 64, 256, 192, [[64, 1, 33, 16]])]


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("case", FFNS, ids=[f"{c[:5]}-{i}" for i, c in enumerate(FFNS)])
def test_moe_ffn_and_grad(case, dtype, act):
    say("moe_ffn", case, dtype, act)
    f = Ffn(*case, dtype, 11)
    f.forward(act)
    torch.cuda.synchronize()
    f.check_forward(act)
    say("moe_ffn_grad", case, dtype, act)
    f.backward(act)
    torch.cuda.synchronize()
    f.check_backward(act)
    f.check_untouched()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("pad,offset", [(8, 0), (8, 8), (3, 0), (0, 1)], ids=str)
def test_moe_ffn_strides(dtype, pad, offset):
    """Padded ranks, and bases off 16 bytes (the element-wise path)."""
    say("moe_ffn strides", dtype, pad, offset)
    f = Ffn(2, 4, 37, 96, 80, spread(2, 4, 37, 8, 50), dtype, 12, pad, offset)
    f.forward("silu")
    f.backward("silu")
    torch.cuda.synchronize()
    f.check_forward("silu")
    f.check_backward("silu")
    f.check_untouched()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_moe_ffn_without_pre(dtype):
    """Inference keeps no pre-activations: the same y, pre untouched."""
    f = Ffn(2, 4, 9, 64, 48, spread(2, 4, 9, 9, 9), dtype, 13)
    f.forward("silu", keep_pre=False)
    torch.cuda.synchronize()
    assert (f.pre == 7.0).all()
    f.check_forward("silu", keep_pre=False)
    y = f.y.clone()
    f.forward("silu")
    torch.cuda.synchronize()
    assert torch.equal(torch.nan_to_num(y), torch.nan_to_num(f.y))


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_moe_ffn_grad_against_differences(act):
    """The gradients of sum(c * y) against central differences of the 64-bit forward pass."""
    f = Ffn(1, 2, 3, 5, 4, [[3, 2]], "f32", 14)
    f.forward(act)
    f.backward(act)
    torch.cuda.synchronize()
    F, W = f.F, f.W

    def loss(x, wi, wo):
        total = 0.0
        for e in range(2):
            j, l, at = f.expert(e)
            gu = x.reshape(-1, W)[at] @ wi.reshape(2, 2 * F, W)[l].t()
            total = total + ((act64(gu[:, :F], act)[0] * gu[:, F:]) @ wo.reshape(2, W, F)[l].t() * f.rows(f.dy, j, at)).sum()
        return float(total)
    args = [torch.nan_to_num(t[0].double()) for t in (f.x, f.w_in, f.w_out)]
    h = 1e-4
    for k, got in ((0, f.dx), (1, f.dw_in), (2, f.dw_out)):
        for i in range(args[k].numel()):
            if k == 0 and not f.keep[0, i // W]:
                continue
            v = []
            for s in (h, -h):
                y = [a.clone() for a in args]
                y[k][i] += s
                v.append(loss(*y))
            # h^2 / 6 of a third derivative below 100, and pre rounded to float32
            assert abs((v[0] - v[1]) / (2 * h) - float(got[0, i])) < 1e-5, (k, i)


def test_moe_ffn_many_ranks_and_experts():
    """More counts than one launch's arguments hold."""
    f = Ffn(32, 64, 2, 16, 8, spread(32, 64, 2, 10, 2), "f32", 15)
    f.forward("silu")
    f.backward("silu")
    torch.cuda.synchronize()
    f.check_forward("silu")
    f.check_backward("silu")
    f.check_untouched()


def test_moe_ffn_keeps_infinities_in_their_rows():
    """A NaN or infinite row changes no other row of y, pre or dx."""
    f = Ffn(1, 1, 70, 64, 32, [[70]], "bf16", 16)
    f.forward("silu")
    f.backward("silu")
    y, dx = f.y.clone(), f.dx.clone()
    x = f.x.view(1, 70, 64)
    x[0, 3], x[0, 40, 5], f.dy.view(1, 70, 64)[0, 51, 1] = math.nan, math.inf, math.nan
    f.forward("silu")
    f.backward("silu")
    torch.cuda.synchronize()
    for new, old, bad in ((f.y, y, (3, 40)), (f.dx, dx, (3, 40, 51))):
        ok = torch.ones(70, dtype=torch.bool, device=DEV)
        ok[list(bad)] = False
        assert torch.equal(new.view(70, 64)[ok], old.view(70, 64)[ok])
        assert torch.isnan(new.view(70, 64)[bad[0]]).all()
