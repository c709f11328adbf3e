"""8-bit rows whose scale is the product of max|x| and float32(1/127), on the GPU:
scales and integers bit for bit, and the block on them within the bounds of its
own tests."""
import math

import pytest
import torch

import test_gpu_int8
from gpu_util import DEV
from model_tiles import CASES
from ring_allreduce_reduction_02_amd import ccgpu
from test_gpu_int8 import ROWS, Block, Product, bytes_of
from test_gpu_model import FFNS, TORCH_DT, gen, ranks, say, spread
from test_gpu_model_calls import replays

pytestmark = pytest.mark.gpu


def product(top):
    """max|x| times float32(1 / 127), rounded once."""
    return top * torch.full_like(top, 1.0).div(torch.full_like(top, 127.0))


def quantized(v):
    s = product(v.abs().amax(-1).float())
    q = torch.where(s[..., None] > 0, torch.round(v.double() / s.double()[..., None]), 0.0).clamp(-127, 127)
    return q, s


def test_the_scale_is_what_torch_makes_of_a_division_by_a_number():
    top = torch.rand(1 << 18, generator=gen(1), device=DEV) * torch.exp(20 * torch.randn(1 << 18, generator=gen(2), device=DEV))
    assert torch.equal(top / 127.0, product(top))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("case", ROWS, ids=str)
def test_rows(case, dtype):
    N, R, W, pad, off = case
    say("rows by a product", case, dtype)
    g = gen(R + W)
    v = torch.randn((N, R, W), generator=g, device=DEV) * torch.exp(3 * torch.randn((N, R, 1), generator=g, device=DEV))
    v[:, 1::5] = 0.0
    v[:, 2::7] = torch.round(v[:, 2::7] * 3) * 0.5            # halves of the maximum: at a border of 63.5
    if R > 6:
        v[:, 3] *= 1e-39                                      # subnormal rows
        v[:, 4] = v[:, 4] / v[:, 4].abs().amax(-1, keepdim=True) * 3e38
        v[:, 6, 0] = 127.0
        v[:, 6, 1:] = torch.randint(-200, 201, (N, W - 1), generator=g, device=DEV) * 0.5
    x = ranks(N, R * W, dtype, pad, off, v) if R else torch.empty(N, 0, dtype=TORCH_DT[dtype], device=DEV)
    q, s = bytes_of(N, R * W, pad, off), ranks(N, R, "f32", 2)
    ccgpu.quantize_rows(x, q, s, W, scale="product")
    torch.cuda.synchronize()
    wq, ws = quantized(x.reshape(N, R, W).float())
    assert torch.equal(s, ws.reshape(N, R))
    assert torch.equal(q.reshape(N, R, W).double(), wq + 0.0)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_values_next_to_the_borders(dtype):
    """Values one step of their type on either side of every half-integer of either scale, and on it where there is one."""
    R, W = 400, 1024
    g = gen(3)
    top = (torch.rand((R, 1), generator=g, device=DEV) + 0.5).to(TORCH_DT[dtype]).float()
    s = torch.where(torch.arange(R, device=DEV)[:, None] % 2 == 0, product(top), top / torch.full_like(top, 127.0))
    k = torch.randint(-127, 127, (R, W), generator=g, device=DEV) + 0.5
    v = (k.double() * s.double()).to(TORCH_DT[dtype])
    step = torch.randint(-1, 2, (R, W), generator=g, device=DEV)
    bits = v.view(torch.int16 if dtype == "bf16" else torch.int32)
    v = (bits + step.to(bits.dtype)).view(TORCH_DT[dtype])
    v[:, :1] = top.to(TORCH_DT[dtype])
    v = torch.where(v.float().abs() > top, top.to(TORCH_DT[dtype]), v)
    x = v.reshape(1, R * W).contiguous()
    q, sc = bytes_of(1, R * W), ranks(1, R, "f32")
    ccgpu.quantize_rows(x, q, sc, W, scale="product")
    torch.cuda.synchronize()
    wq, ws = quantized(x.reshape(1, R, W).float())
    assert torch.equal(sc, ws) and torch.equal(q.reshape(1, R, W).double(), wq)
    other = bytes_of(1, R * W)
    ccgpu.quantize_rows(x, other, sc, W)
    torch.cuda.synchronize()
    assert torch.equal(sc[0], (top / torch.full_like(top, 127.0))[:, 0]) and not torch.equal(q, other)


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf], ids=str)
@pytest.mark.parametrize("W", [7, 700, 9000])
def test_rows_that_are_not_finite(W, bad):
    x = torch.randn(1, 5 * W, generator=gen(4), device=DEV)
    x[0, 2 * W + W // 2] = bad
    q, s = bytes_of(1, 5 * W), ranks(1, 5, "f32")
    ccgpu.quantize_rows(x, q, s, W, scale="product")
    torch.cuda.synchronize()
    assert torch.isnan(s[0]).tolist() == [False, False, True, False, False]
    assert not q[0, 2 * W:3 * W].any() and q[0, 3 * W:].any()


def test_float32_rows_times_weights_as_torch_quantises_them():
    """cc_moe_matmul_int8 on rows kept by a product, 515 float32 columns: what torch code that divides by 127.0 gives,
    for inputs in which the quotient's integers are others."""
    N, E, cap, W, C = 2, 6, 139, 515, 331
    counts = [[139, 127, 108, 96, 88, 80]] * N
    moved = 0
    for seed in range(6):
        p = Product(N, E, cap, W, C, counts, "f32", 100 + seed)
        x = torch.randn(N, E * cap * W, generator=gen(seed), device=DEV)
        v = x.view(N, E * cap, W)
        v[:, ::3, 7] = v[:, ::3].abs().amax(-1) / 2              # a quotient of 63.5 but for the scale's last bit
        s = v.abs().amax(-1, keepdim=True) / 127.0
        want = torch.round(v.double() / s.double()).clamp(-127, 127)
        ccgpu.quantize_rows(x, p.x, p.sx, W)
        moved += int((p.x.view(N, E * cap, W) != want).sum())
        ccgpu.quantize_rows(x, p.x, p.sx, W, scale="product")
        assert torch.equal(p.x.view(N, E * cap, W).double(), want) and torch.equal(p.sx, s[..., 0])
        p.run()
        torch.cuda.synchronize()
        p.check()
    assert moved > 0


class Scaled(Block):
    """The block on rows kept by a product."""

    def forward8(self, act, stream=None, ws=None):
        if ws is None:
            ws = ccgpu.make_moe_ffn_int8_workspace(self.counts, self.cap, self.W, self.F, self.dtype)
            ws.fill_(0xA5)
        ccgpu.moe_ffn_int8(self.x, self.q_in, self.s_in, self.q_out, self.s_out, self.y, self.counts, self.cap, self.W,
                           act=act, workspace=ws, stream=stream, scale="product")


@pytest.fixture
def by_a_product(monkeypatch):
    monkeypatch.setattr(test_gpu_int8, "scale", product)      # the block's reference takes its scales from there


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("case", FFNS, ids=[f"{c[:5]}-{i}" for i, c in enumerate(FFNS)])
def test_block(case, dtype, act, by_a_product):
    say("block by a product", case, dtype, act)
    f = Scaled(*case, dtype, 26)
    f.forward8(act)
    torch.cuda.synchronize()
    f.check8(act)


@pytest.mark.parametrize("name", CASES)
def test_block_in_tiles_of_every_size(name, by_a_product):
    case, offset = CASES[name]
    say("block by a product, tiles", name)
    f = Scaled(*case, "bf16", 27, offset=offset)
    f.forward8("silu")
    torch.cuda.synchronize()
    f.check8("silu")


def test_both_in_a_graph():
    f = Scaled(2, 4, 40, 72, 136, spread(2, 4, 40, 1, 40), "bf16", 62)
    ws = ccgpu.make_moe_ffn_int8_workspace(f.counts, f.cap, f.W, f.F, f.dtype)
    rows = torch.empty(2, 5 * 700, device=DEV)
    q, s = torch.empty(2, 5 * 700, dtype=torch.int8, device=DEV), torch.empty(2, 5, device=DEV)

    def call():
        f.forward8("gelu", ws=ws)
        ccgpu.quantize_rows(rows, q, s, 700, scale="product")

    def refresh(k):
        f.x.copy_(torch.where(torch.isnan(f.x), f.x.float(), torch.randn(f.x.shape, generator=gen(k), device=DEV)))
        rows.copy_(torch.randn(rows.shape, generator=gen(k), device=DEV))
    say("rows by a product in a graph")
    replays(call, refresh, [f.y, q, s])
