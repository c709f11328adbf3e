"""The balance loss, the 8-bit products and the 8-bit checkpoints as a program uses
them: captured into a graph and replayed with new inputs, on other streams, two
calls at once, more counts than a launch's arguments hold, past 4 GiB, and
together -- a training step of an MoE layer and one that serves."""
import math

import numpy as np
import pytest
import torch

from gpu_util import DEV
from ring_allreduce_reduction_02_amd import ccgpu
from test_gpu_balance import reference as balance_reference
from test_gpu_ckpt import Ckpt
from test_gpu_int8 import Block, Product, bytes_of, quantized
from test_gpu_model import HALF, U, draw_logits, gen, near, ranks, route_grad_reference, route_reference, say, spread
from test_gpu_model_calls import replays

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("summed", [True, False], ids=["all", "own"])
@pytest.mark.parametrize("tokens,E", [(16, 64), (3000, 8), (5000, 600)])
def test_balance_in_a_graph(tokens, E, summed):
    N = 3
    logits = torch.empty(N, tokens * E, device=DEV)
    counts = torch.empty(N, E, dtype=torch.int32, device=DEV)
    total, prob, loss = torch.empty(N, E + 1, dtype=torch.int32, device=DEV), torch.empty(N, E, device=DEV), torch.empty(N, 1, device=DEV)
    dloss, d = torch.rand(N, 1, device=DEV), torch.empty_like(logits)
    ws = ccgpu.make_moe_balance_loss_workspace(N, tokens, E)

    def call():
        ccgpu.moe_balance_loss(logits, counts, total, prob, loss, summed=summed, workspace=ws)
        ccgpu.moe_balance_loss_grad(logits, total, dloss, d)

    def refresh(k):
        logits.copy_(draw_logits(N, tokens, E, "f32", k, True).reshape(N, -1))
        counts.copy_(torch.randint(0, 50, (N, E), generator=gen(k), device=DEV, dtype=torch.int32))
    say("balance in a graph", tokens, E, summed)
    replays(call, refresh, [total, prob, loss, d])


# fused with the plan, apart from it, and each with counts in memory
CASES = {"few rows": (2, 4, 40, 72, 136, spread(2, 4, 40, 1, 40)), "many rows": (2, 4, 2500, 64, 48, spread(2, 4, 2500, 2, 2500)),
         "counts in memory": (40, 40, 2, 16, 24, spread(40, 40, 2, 2, 2)),
         "many rows, counts in memory": (16, 64, 40, 64, 48, spread(16, 64, 40, 3, 40)), "odd": (1, 2, 300, 33, 65, [[257, 300]])}


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("name", CASES)
def test_checkpoint_in_a_graph(name, dtype):
    f = Ckpt(*CASES[name], dtype, 61)
    ws = [ccgpu.make_moe_ffn_checkpoint_workspace(f.counts, f.cap, f.W, f.F, dtype, grad=g) for g in (False, True)]

    def call():
        f.forward("silu", ws=ws[0])
        f.backward("silu", ws=ws[1])

    def refresh(k):
        for t in (f.x, f.dy):
            t.copy_(torch.where(torch.isnan(t), t.float(), torch.randn(t.shape, generator=gen(k), device=DEV)))
    say("ckpt in a graph", name, dtype)
    replays(call, refresh, [f.y, f.ckpt, f.dx, f.dw_in, f.dw_out])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("name", CASES)
def test_int8_in_a_graph(name, dtype):
    f = Block(*CASES[name], dtype, 62)
    p = Product(*CASES[name], dtype, 63)
    ws = ccgpu.make_moe_ffn_int8_workspace(f.counts, f.cap, f.W, f.F, dtype)
    wp = ccgpu.make_moe_matmul_int8_workspace(p.counts, p.cap, p.W, p.C)
    rows = torch.empty(p.N, 5 * p.W, device=DEV)
    q, s = torch.empty(p.N, 5 * p.W, dtype=torch.int8, device=DEV), torch.empty(p.N, 5, device=DEV)

    def call():
        f.forward8("gelu", ws=ws)
        ccgpu.moe_matmul_int8(p.x, p.sx, p.w, p.sw, p.y, p.counts, p.cap, p.W, workspace=wp)
        ccgpu.quantize_rows(rows, q, s, p.W)

    def refresh(k):
        f.x.copy_(torch.where(torch.isnan(f.x), f.x.float(), torch.randn(f.x.shape, generator=gen(k), device=DEV)))
        p.x.copy_(torch.randint(-127, 128, p.x.shape, generator=gen(k), device=DEV, dtype=torch.int8))
        rows.copy_(torch.randn(rows.shape, generator=gen(k), device=DEV))
    say("int8 in a graph", name, dtype)
    replays(call, refresh, [f.y, p.y, q, s])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("name", CASES)
def test_each_way_to_the_rows(name, dtype):
    say("rows", name, dtype)
    f = Ckpt(*CASES[name], dtype, 64)
    f.forward("gelu")
    f.backward("gelu")
    b = Block(*CASES[name], dtype, 65)
    b.forward8("silu")
    torch.cuda.synchronize()
    f.check("gelu")
    b.check8("silu")


def test_wide_rows_apart_from_the_plan():
    """More rows than the plan takes on the way, each longer than a wave keeps in registers."""
    f = Block(1, 1, 8300, 4104, 16, [[8290]], "bf16", 66)
    f.forward8("silu")
    torch.cuda.synchronize()
    f.check8("silu")


def test_two_streams_with_a_workspace_each():
    """Calls of every kind in flight at once, each on its stream and workspace, give what each gives alone."""
    fs = [(Ckpt(2, 4, 200, 128, 256, spread(2, 4, 200, 30 + k, 200), "bf16", 67 + k),
           Block(2, 4, 200, 128, 256, spread(2, 4, 200, 40 + k, 200), "bf16", 77 + k)) for k in range(2)]
    ws = [[ccgpu.make_moe_ffn_checkpoint_workspace(c.counts, c.cap, c.W, c.F, "bf16", grad=g) for g in (False, True)]
          + [ccgpu.make_moe_ffn_int8_workspace(b.counts, b.cap, b.W, b.F, "bf16")] for c, b in fs]
    bal = []
    for k in range(2):
        lg = draw_logits(2, 900, 32, "f32", k, True).reshape(2, -1).contiguous()
        bal.append([lg, torch.full((2, 32), 7 + k, dtype=torch.int32, device=DEV), torch.empty(2, 33, dtype=torch.int32, device=DEV),
                    torch.empty(2, 32, device=DEV), torch.empty(2, 1, device=DEV), ccgpu.make_moe_balance_loss_workspace(2, 900, 32),
                    torch.empty_like(lg)])

    def step(k, stream):
        (c, b), w, (lg, cnt, tot, pr, ls, wb, d) = fs[k], ws[k], bal[k]
        c.forward("silu", stream=stream, ws=w[0])
        b.forward8("silu", stream=stream, ws=w[2])
        ccgpu.moe_balance_loss(lg, cnt, tot, pr, ls, workspace=wb, stream=stream)
        ccgpu.moe_balance_loss_grad(lg, tot, ls, d, stream=stream)
        c.backward("silu", stream=stream, ws=w[1])

    def outs(k):
        (c, b), x = fs[k], bal[k]
        return [c.y, c.ckpt, c.dx, c.dw_in, c.dw_out, b.y, *x[2:5], x[6]]
    alone = []
    for k in range(2):
        step(k, None)
        torch.cuda.synchronize()
        alone.append([t.clone() for t in outs(k)])
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(3):
        for k, s in enumerate(streams):
            step(k, s)
    torch.cuda.synchronize()
    for k in range(2):
        for t, want in zip(outs(k), alone[k]):
            assert torch.equal(torch.nan_to_num(t.float()), torch.nan_to_num(want.float()))


@pytest.mark.parametrize("size", [0.95, 1.5])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_int8_past_4_gib(dtype, size):
    """8-bit rows of an expert behind byte 2^31 of its rank's buffer, where 32-bit offsets still reach them, and behind
    byte 2^32."""
    W, C = 256, 32
    p = object.__new__(Product)
    p.N, p.E, p.per, p.W, p.C, p.dtype = 1, 4, 4, W, C, dtype
    p.cap = int(size * (1 << 32)) // (4 * W)
    p.counts = [[3, 0, 0, 70]]
    f = object.__new__(Ckpt)
    f.N, f.E, f.cap, f.per, f.counts = 1, 4, p.cap, 4, p.counts
    f.keep = torch.zeros(1, 4 * p.cap, dtype=torch.bool, device=DEV)
    f.keep[0, :3] = f.keep[0, 3 * p.cap:3 * p.cap + 70] = True
    p.f = f
    at, g = f.keep[0].nonzero().view(-1), gen(70)
    p.x = torch.empty(1, 4 * p.cap * W, dtype=torch.int8, device=DEV)
    p.x.view(-1, W)[at] = torch.randint(-127, 128, (len(at), W), generator=g, device=DEV, dtype=torch.int8)
    p.w = torch.randint(-127, 128, (1, 4 * C * W), generator=g, device=DEV, dtype=torch.int8)
    p.sx, p.sw = torch.rand(1, 4 * p.cap, generator=g, device=DEV), torch.rand(1, 4 * C, generator=g, device=DEV)
    p.y = torch.full((1, 4 * p.cap * C), 7.0, dtype={"f32": torch.float32, "bf16": torch.bfloat16}[dtype], device=DEV)
    say("int8 past 4 GiB", dtype, size)
    p.run()
    torch.cuda.synchronize()
    p.check()


def test_quantize_rows_past_4_gib_and_a_launchs_workgroups():
    """A row behind byte 2^32 of a rank's rows and integers; and more rows than one launch has workgroups for."""
    W, R = 8192, (1 << 19) + 3                            # 17 GB of float32, 4.3 GB of integers
    x = torch.zeros(1, R * W, device=DEV)
    last = torch.randn(W, generator=gen(71), device=DEV)
    x[0, -W:] = last
    q, s = torch.full((1, R * W), 5, dtype=torch.int8, device=DEV), torch.empty(1, R, device=DEV)
    ccgpu.quantize_rows(x, q, s, W)
    torch.cuda.synchronize()
    wq, ws = quantized(last)
    assert torch.equal(q[0, -W:].double(), wq) and s[0, -1] == ws
    assert not s[0, :-1].any() and not q[0, :-W].any()
    del x, q, s
    R = (1 << 24) + 9
    x = torch.randn(1, R * 2, generator=gen(72), device=DEV)
    q, s = bytes_of(1, R * 2), torch.empty(1, R, device=DEV)
    ccgpu.quantize_rows(x, q, s, 2)
    torch.cuda.synchronize()
    wq, ws = quantized(x.view(R, 2))
    assert torch.equal(s[0], ws) and torch.equal(q.view(R, 2).double(), wq + 0.0)


def test_many_ranks_share_one_quantisation():
    """64 ranks, blocks of rows of every length."""
    for W in (1, 31, 130):
        x = torch.randn(64, 7 * W, generator=gen(W), device=DEV).bfloat16()
        q, s = bytes_of(64, 7 * W, 3, 1), ranks(64, 7, "f32", 1)
        ccgpu.quantize_rows(x, q, s, W)
        torch.cuda.synchronize()
        wq, ws = quantized(x.view(64, 7, W).float())
        assert torch.equal(s, ws) and torch.equal(q.reshape(64, 7, W).double(), wq + 0.0)


def layer(N, T, W, F, E, K, seed, dtype=torch.float32):
    """A layer's inputs up to the experts' rows: logits, routing and dispatched rows of `tokens` embeddings."""
    g, per = gen(seed), E // N
    x = torch.randn(N, T * W, generator=g, device=DEV).to(dtype)
    logits = (x.float().view(N, T, W) @ torch.randn(W, E, generator=g, device=DEV) / math.sqrt(W) * 2)
    logits[:, -3:] = -math.inf                                     # padding tokens
    logits = logits.reshape(N, T * E).contiguous()
    experts, order = (torch.empty(N, T * K, dtype=torch.int32, device=DEV) for _ in range(2))
    weights, counts = torch.empty(N, T * K, device=DEV), torch.empty(N, E, dtype=torch.int32, device=DEV)
    ccgpu.moe_route(logits, experts, weights, order, counts, K, normalize=True, workspace=ccgpu.make_moe_route_workspace(N, T, E, K))
    host = counts.tolist()
    cap = max(max(row) for row in host)
    token = torch.where(order >= 0, order // K, -1).int()
    rows = torch.empty(N, T * K * W, dtype=dtype, device=DEV)
    ccgpu.embedding(x, token, rows, W)
    xe = torch.zeros(N, E * cap * W, dtype=dtype, device=DEV)
    ccgpu.moe_dispatch_padded(rows, xe, host, cap, W)
    w_in = (torch.randn(N, per * 2 * F * W, generator=g, device=DEV) / math.sqrt(W)).to(dtype)
    w_out = (torch.randn(N, per * W * F, generator=g, device=DEV) / math.sqrt(F)).to(dtype)
    return x, logits, experts, weights, counts, host, cap, token, rows, xe, w_in, w_out


def holder(cls, N, E, cap, W, F, host, dtype, **bufs):
    f = object.__new__(cls)
    f.N, f.E, f.cap, f.W, f.F, f.counts, f.dtype, f.per = N, E, cap, W, F, host, dtype, E // N
    f.keep = torch.zeros((N, N, f.per, cap), dtype=torch.bool, device=DEV)
    for i in range(N):
        for e in range(E):
            f.keep[e // f.per, i, e % f.per, :host[i][e]] = True
    f.keep = f.keep.reshape(N, E * cap)
    for k, v in bufs.items():
        setattr(f, k, v)
    return f


def test_training_step_with_balance_and_checkpoint():
    """Routing, balance loss, dispatch, experts with a checkpoint, combine; back through the checkpoint, the combine's
    transpose and the routing, the balance loss's gradient added to the routing's in place: y as the block without a
    checkpoint gives it, the experts' gradients at the kept values, the logits' against 64 bits."""
    N, T, W, F, E, K, lam = 4, 96, 64, 80, 8, 2, 0.01
    x, logits, experts, weights, counts, host, cap, token, rows, xe, w_in, w_out = layer(N, T, W, F, E, K, 80)
    total, prob, loss = torch.empty(N, E + 1, dtype=torch.int32, device=DEV), torch.empty(N, E, device=DEV), torch.empty(N, 1, device=DEV)
    ccgpu.moe_balance_loss(logits, counts, total, prob, loss, workspace=ccgpu.make_moe_balance_loss_workspace(N, T, E))
    ckpt = ccgpu.make_moe_ffn_checkpoint(host, cap, W, F)
    ckpt.fill_(0x5A)
    ye, yn, dye, dxe = (torch.zeros(N, E * cap * W, device=DEV) for _ in range(4))
    ccgpu.moe_ffn_checkpoint(xe, w_in, w_out, ckpt, ye, host, cap, W, workspace=ccgpu.make_moe_ffn_checkpoint_workspace(host, cap, W, F, "f32"))
    ccgpu.moe_ffn(xe, w_in, w_out, yn, host, cap, W, workspace=ccgpu.make_moe_ffn_workspace(host, cap, W, F, "f32"))
    assert torch.equal(ye, yn)
    back = torch.zeros(N, T * K * W, device=DEV)
    ccgpu.moe_combine_padded(ye, back, host, cap, W)
    drow = torch.randn(N, T * K * W, generator=gen(81), device=DEV)
    ccgpu.moe_dispatch_padded(drow, dye, host, cap, W)
    dw_in, dw_out = torch.empty_like(w_in), torch.empty_like(w_out)
    ccgpu.moe_ffn_checkpoint_grad(ckpt, w_in, w_out, dye, dxe, dw_in, dw_out, host, cap, W,
                                  workspace=ccgpu.make_moe_ffn_checkpoint_workspace(host, cap, W, F, "f32", grad=True))
    dweights = torch.randn(N, T * K, generator=gen(82), device=DEV)
    dlogits = torch.empty_like(logits)
    ccgpu.moe_route_grad(logits, experts, dweights, dlogits, K, normalize=True)
    ccgpu.moe_balance_loss_grad(logits, total, torch.full((N, 1), lam, device=DEV), dlogits, base=dlogits)
    torch.cuda.synchronize()

    f = holder(Ckpt, N, E, cap, W, F, host, "f32", x=xe, w_in=w_in, w_out=w_out, ckpt=ckpt, dy=dye, y=ye, dx=dxe, dw_in=dw_in,
               dw_out=dw_out, pre=None)
    f.check_forward("silu", keep_pre=False)
    f.check_kept()
    f.at_kept()
    f.check_backward("silu")
    z, c = logits.double().cpu().numpy().reshape(N, T, E), counts.cpu().numpy().astype(np.int64)
    tot, pw, lw, p, fr = balance_reference(z, c, True)
    assert np.array_equal(total.cpu().numpy(), tot)
    near(loss, torch.from_numpy(lw).to(DEV), torch.full((N, 1), (N * T + E + 40) * U * float(lw.max()), device=DEV, dtype=torch.float64), "loss")
    pick = route_reference(z, K, True)[0].reshape(N, T, K)
    d, a = route_grad_reference(z, pick, dweights.double().cpu().numpy().reshape(N, T, K), True)
    fv = fr[:1, None, :]
    dot = (fv * p).sum(-1, keepdims=True)
    scale = float(np.float32(lam)) * E / tot[0, E]
    want = d + scale * p * (fv - dot)
    # the bounds of the two gradients' own tests, and the rounding of their sum
    bound = (3 * E + 32 + 4 * 30) * U * a + (4 * E + 40 + 4 * 30) * U * scale * p * (fv + dot) + 2 * U * np.abs(want) + 1e-37
    near(dlogits.view(N, T, E), torch.from_numpy(want).to(DEV), torch.from_numpy(bound).to(DEV), "dlogits")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_serving_step_in_8_bits(dtype):
    """The same layer served: routed rows through moe_ffn_int8, and the first product from rows that were quantised
    before the dispatch, which equals the one of rows quantised behind it."""
    N, T, W, F, E, K = 4, 9, 64, 80, 8, 2
    dt = {"f32": torch.float32, "bf16": torch.bfloat16}[dtype]
    x, logits, experts, weights, counts, host, cap, token, rows, xe, w_in, w_out = layer(N, T, W, F, E, K, 83, dt)
    per = E // N
    q_in, q_out = torch.empty(w_in.shape, dtype=torch.int8, device=DEV), torch.empty(w_out.shape, dtype=torch.int8, device=DEV)
    s_in, s_out = torch.empty(N, per * 2 * F, device=DEV), torch.empty(N, per * W, device=DEV)
    ccgpu.quantize_rows(w_in, q_in, s_in, W)
    ccgpu.quantize_rows(w_out, q_out, s_out, F)
    ye = torch.full_like(xe, 7.0)
    ccgpu.moe_ffn_int8(xe, q_in, s_in, q_out, s_out, ye, host, cap, W, workspace=ccgpu.make_moe_ffn_int8_workspace(host, cap, W, F, dtype))
    torch.cuda.synchronize()
    f = holder(Block, N, E, cap, W, F, host, dtype, x=xe, y=ye, q_in=q_in, q_out=q_out, s_in=s_in, s_out=s_out, pre=None)
    f.check8("silu")
    q, s = torch.empty(rows.shape, dtype=torch.int8, device=DEV), torch.empty(N, T * K, device=DEV)
    ccgpu.quantize_rows(rows, q, s, W)
    eq, es = torch.zeros(N, E * cap * W // 4, dtype=torch.int32, device=DEV), torch.zeros(N, E * cap, device=DEV)
    ccgpu.moe_dispatch_padded(q.view(torch.int32), eq, host, cap, W // 4)
    ccgpu.moe_dispatch_padded(s, es, host, cap, 1)
    kq, ks = torch.empty(xe.shape, dtype=torch.int8, device=DEV), torch.empty(N, E * cap, device=DEV)
    ccgpu.quantize_rows(xe, kq, ks, W)
    outs = []
    for a, b in ((eq.view(torch.int8), es), (kq, ks)):
        y = torch.zeros(N, E * cap * 2 * F, dtype=dt, device=DEV)
        ccgpu.moe_matmul_int8(a, b, q_in, s_in, y, host, cap, W, workspace=ccgpu.make_moe_matmul_int8_workspace(host, cap, W, 2 * F))
        outs.append(y)
    torch.cuda.synchronize()
    assert torch.equal(*outs) and outs[0].any() and HALF[dtype] > 0


def test_binding_refuses_other_devices_and_missing_workspaces():
    x = torch.zeros(1, 8, device=DEV)
    i = torch.zeros(1, 4, dtype=torch.int32, device=DEV)
    outs = torch.zeros(1, 5, dtype=torch.int32, device=DEV), torch.zeros(1, 4, device=DEV), torch.zeros(1, 1, device=DEV)
    with pytest.raises(ccgpu.CCError, match="workspace"):
        ccgpu.moe_balance_loss(x, i, *outs)
    with pytest.raises(ValueError, match="current device"):
        ccgpu.moe_balance_loss(x, i, *outs, workspace=torch.zeros(4096, dtype=torch.uint8))
    with pytest.raises(ValueError, match="device tensors"):
        ccgpu.quantize_rows(x.cpu(), torch.zeros(1, 8, dtype=torch.int8, device=DEV), x[:, :2], 4)
    with pytest.raises(ccgpu.CCError, match="overlap"):
        ccgpu.quantize_rows(x, x.view(torch.int8)[:, :8], torch.zeros(1, 2, device=DEV), 4)
    with pytest.raises(ValueError, match="q must be torch.int8"):
        ccgpu.quantize_rows(x, torch.zeros(1, 8, dtype=torch.uint8, device=DEV), torch.zeros(1, 2, device=DEV), 4)
