"""Host side of the balance loss, the 8-bit integer products and the 8-bit
checkpoints: sizes, the checkpoint's layout, and the refusal of bad arguments
before any launch (no GPU needed)."""
import ctypes
import os
import re

import pytest

from ring_allreduce_reduction_02_amd import ccgpu
from test_abi_cpu import FAKE, no_gpu_only
from test_model_cpu import COUNTS, GB, INVALID, NO_DEVICE, NONE, OK, UNSUPPORTED, buf, cfg, sizes

TWO = [COUNTS[:4], COUNTS[4:]]


def error():
    return ccgpu.load().cc_last_error().decode()


def test_limits_match_the_header():
    hdr = open(os.path.join(os.path.dirname(os.path.dirname(__file__)), "include", "cc.h")).read()
    assert int(re.search(r"#define CC_CKPT_BLOCK (\d+)", hdr).group(1)) == 32
    assert ccgpu.moe_balance_loss_workspace_size(1, 10, 1024) > 0
    for bad in (0, 1025):
        with pytest.raises(ccgpu.CCError):
            ccgpu.moe_balance_loss_workspace_size(1, 10, bad)


# ------------------------------------------------------------------ balance loss

def balance(bufs=None, tokens=10, E=8, summed=1, dtype=1, N=4, c=None):
    return ccgpu.raw("cc_moe_balance_loss", *(bufs or [buf(i) for i in range(5)]), tokens, E, summed, dtype, N, c or cfg(), None)


def balance_grad(bufs=None, tokens=10, E=8, dtype=1, N=4, c=None):
    return ccgpu.raw("cc_moe_balance_loss_grad", *(bufs or [buf(i) for i in range(5)]), tokens, E, dtype, N, c or cfg(), None)


@no_gpu_only
@pytest.mark.parametrize("call", [balance, balance_grad])
def test_balance_refusals(call):
    assert call() == NO_DEVICE
    assert call(E=1024) == NO_DEVICE
    for kw in (dict(N=0), dict(N=65), dict(E=0), dict(E=1025), dict(dtype=9), dict(tokens=1 << 24), dict(c=cfg(blocks_per_cu=-1))):
        assert call(**kw) == INVALID, kw
        assert error()
    for kw in (dict(dtype=0), dict(c=cfg(algo=1)), dict(c=cfg(fuse_depth=1))):
        assert call(**kw) == UNSUPPORTED, kw
    outs = {2, 3, 4} if call is balance else {4}
    for i in range(5):
        b = [buf(k) for k in range(5)]
        b[i] = ccgpu.RankBuf(None, 1 << 20)
        assert call(b) == (NO_DEVICE if call is balance_grad and i == 3 else INVALID), i      # base is optional
        b[i] = buf(i, 2)
        assert call(b) == INVALID, i
        b[i] = buf(i, off=1)
        assert call(b) == INVALID, i
        for j in range(5):
            if j != i:
                b[i] = buf(j)
                same = call is balance_grad and {i, j} == {3, 4}                              # in place
                assert call(b) == (INVALID if outs & {i, j} and not same else NO_DEVICE), (i, j)
    if call is balance_grad:
        b = [buf(k) for k in range(5)]
        b[3] = buf(4, off=16)                              # base over dlogits, but not the same
        assert call(b) == INVALID and "overlap" in error()
        assert call([NONE] * 5, tokens=0) == OK
    else:
        assert balance(summed=2) == INVALID
        assert call([NONE] + [buf(k) for k in range(1, 5)], tokens=0) == NO_DEVICE             # the loss is still written


@no_gpu_only
def test_balance_workspace():
    need = ccgpu.moe_balance_loss_workspace_size(4, 10, 8)
    assert need >= 4 * 9 * 4 and ccgpu.moe_balance_loss_workspace_size(4, 0, 8) > 0
    assert balance(c=cfg(workspace_bytes=need)) == NO_DEVICE
    for c in (cfg(workspace_bytes=need - 1), cfg(workspace=None), cfg(workspace=FAKE + 100 * GB + 8)):
        assert balance(c=c) == INVALID
    for i in range(5):
        assert balance(c=cfg(workspace=FAKE + i * GB)) == INVALID and "overlap" in error()
    assert balance_grad(c=cfg(workspace=None, workspace_bytes=0)) == NO_DEVICE


# ------------------------------------------------------------------ 8-bit integers

def rows(bufs=None, n=10, width=8, dtype=1, N=4, c=None):
    return ccgpu.raw("cc_quantize_rows", *(bufs or [buf(i) for i in range(3)]), n, width, dtype, N, c or cfg(), None)


@no_gpu_only
def test_quantize_rows_refusals():
    assert rows() == NO_DEVICE
    for kw in (dict(N=0), dict(N=65), dict(width=0), dict(width=1 << 31), dict(n=1 << 31), dict(dtype=5)):
        assert rows(**kw) == INVALID, kw
    for kw in (dict(dtype=0), dict(c=cfg(algo=3)), dict(c=cfg(fuse_depth=1))):
        assert rows(**kw) == UNSUPPORTED, kw
    for i in range(3):
        b = [buf(k) for k in range(3)]
        b[i] = ccgpu.RankBuf(None, 1 << 20)
        assert rows(b) == INVALID
        b[i] = buf(i, 12)
        assert rows(b) == INVALID
        b[i] = buf(i, off=1)
        assert rows(b) == (NO_DEVICE if i == 1 else INVALID)         # bytes lie anywhere
        b[i] = buf((i + 1) % 3, off=4)
        assert rows(b) == INVALID
    assert rows([NONE] * 3, n=0) == OK


def matmul(bufs=None, counts=COUNTS, E=4, cap=5, W=8, cols=16, dtype=1, N=2, c=None):
    cnt = sizes(counts) if counts is not None else None
    return ccgpu.raw("cc_moe_matmul_int8", *(bufs or [buf(i) for i in range(5)]), cnt, E, cap, W, cols, dtype, N, c or cfg(), None)


def ffn8(bufs=None, counts=COUNTS, E=4, cap=5, W=8, cols=16, act=0, dtype=1, N=2, c=None):
    cnt = sizes(counts) if counts is not None else None
    return ccgpu.raw("cc_moe_ffn_int8", *(bufs or [buf(i) for i in range(6)]), cnt, E, cap, W, cols, act, dtype, N, c or cfg(), None)


@no_gpu_only
@pytest.mark.parametrize("call", [matmul, ffn8])
def test_int8_refusals(call):
    n, out = (5, 4) if call is matmul else (6, 5)
    assert call() == NO_DEVICE
    far = dict(bufs=[buf(i, 1 << 28) for i in range(n)])
    assert call(W=(1 << 17) - 1, **far) == NO_DEVICE
    for kw in (dict(N=0), dict(N=65), dict(N=3), dict(E=1), dict(E=3), dict(W=0), dict(cols=0), dict(W=1 << 17), dict(cols=1 << 24),
               dict(dtype=3), dict(counts=None), dict(cap=1 << 29), dict(E=(1 << 20) + 2)):
        assert call(**kw) == INVALID, kw
    for kw in (dict(dtype=0), dict(c=cfg(algo=1)), dict(c=cfg(fuse_depth=1))):
        assert call(**kw) == UNSUPPORTED, kw
    if call is ffn8:
        assert call(cols=1 << 17, **far) == INVALID and call(act=2) == INVALID and call(act=-1) == INVALID
    else:
        assert call(cols=1 << 17, **far) == NO_DEVICE
    bytes_ = {0, 2} if call is matmul else {1, 3}                     # int8 operands lie anywhere
    for i in range(n):
        b = [buf(k) for k in range(n)]
        b[i] = ccgpu.RankBuf(None, 1 << 20)
        assert call(b) == INVALID
        b[i] = buf(i, 12)
        assert call(b) == INVALID
        b[i] = buf(i, off=1)
        assert call(b) == (NO_DEVICE if i in bytes_ else INVALID), i
        b[i] = buf((i + 1) % n, off=64)
        assert call(b) == (INVALID if out in (i, (i + 1) % n) else NO_DEVICE)
    if call is matmul:
        need = ccgpu.moe_matmul_int8_workspace_size(TWO, 5, 8, 16)
    else:
        need = ccgpu.moe_ffn_int8_workspace_size(TWO, 5, 8, 16, "f32")
    assert call(c=cfg(workspace_bytes=need)) == NO_DEVICE
    for c in (cfg(workspace_bytes=need - 1), cfg(workspace=None), cfg(workspace=FAKE + 100 * GB + 8), cfg(workspace=FAKE + GB)):
        assert call(c=c) == INVALID
    # rows that do not exist need no buffers
    w = [NONE if k in ((0, 1, 4) if call is matmul else (0, 5)) else buf(k) for k in range(n)]
    assert call(w, cap=0) == OK and call(w, counts=[0] * 8, cap=0) == OK


def test_int8_ffn_workspace_grows_with_the_kept_rows():
    a = ccgpu.moe_ffn_int8_workspace_size([[100, 0], [0, 0]], 64, 100, 200, "bf16")
    b = ccgpu.moe_ffn_int8_workspace_size([[64, 64], [64, 64]], 64, 100, 200, "bf16")
    assert a >= 64 * (128 + 256 + 200 * 2) and b >= 256 * (128 + 256 + 200 * 2) > a


def test_odd_widths_are_copied_from_1024_rows_an_expert():
    """Weights (and a product's rows) whose rows are no whole 16-byte vectors: copies in the workspace where they pay."""
    def block(rows, W, F):
        return ccgpu.moe_ffn_int8_workspace_size([[rows, rows]], rows, W, F, "bf16")

    def product(rows, W, C):
        return ccgpu.moe_matmul_int8_workspace_size([[rows, rows]], rows, W, C)
    line = lambda v: -(-v // 128) * 128  # noqa: E731
    for W, F in ((2047, 1001), (201, 333)):
        rest = 2048 * (line(W) + line(F) + 2 * F + 12) + (64 << 10)
        weights = 2 * (2 * F * line(W) + W * line(F))
        assert block(1023, W, F) < rest and weights <= block(1024, W, F) < rest + weights
    assert block(1024, 2048, 1008) < 2048 * (2048 + 1024 + 2016 + 12) + (64 << 10)              # whole vectors
    assert product(1023, 2047, 515) < 64 << 10 and product(1024, 2048, 515) < 64 << 10
    assert 2048 * 2048 + 2 * 515 * 2048 <= product(1024, 2047, 515) < 2048 * 2048 + 2 * 515 * 2048 + (64 << 10)
    assert product(1024, 2047, 511) < 64 << 10                                                  # too few columns


# ------------------------------------------------------------------ checkpoints

def test_checkpoint_row():
    for W, F in ((1, 1), (32, 16), (33, 31), (515, 331), (2048, 2048)):
        up, blocks = lambda v: -(-v // 16) * 16, lambda v: -(-v // 32)  # noqa: E731
        assert ccgpu.moe_ffn_checkpoint_row(W, F) == up(up(W) + 2 * up(F) + blocks(W) + 2 * blocks(F))
    for bad in ((0, 1), (1, 0), (1 << 24, 1), (1, 1 << 24)):
        with pytest.raises(ccgpu.CCError):
            ccgpu.moe_ffn_checkpoint_row(*bad)


def ckpt(grad, bufs=None, counts=COUNTS, E=4, cap=5, W=8, F=16, act=0, dtype=1, N=2, c=None):
    n = 7 if grad else 5
    cnt = sizes(counts) if counts is not None else None
    return ccgpu.raw("cc_moe_ffn_checkpoint_grad" if grad else "cc_moe_ffn_checkpoint", *(bufs or [buf(i) for i in range(n)]),
                     cnt, E, cap, W, F, act, dtype, N, c or cfg(), None)


@no_gpu_only
@pytest.mark.parametrize("grad", [False, True])
def test_checkpoint_refusals(grad):
    names = ("ckpt w_in w_out dy dx dw_in dw_out" if grad else "x w_in w_out ckpt y").split()
    n = len(names)
    assert ckpt(grad) == NO_DEVICE
    for kw in (dict(N=0), dict(N=65), dict(N=3), dict(E=1), dict(E=3), dict(W=0), dict(F=0), dict(W=1 << 24), dict(F=1 << 24),
               dict(act=2), dict(act=-1), dict(dtype=3), dict(counts=None), dict(cap=1 << 29)):
        assert ckpt(grad, **kw) == INVALID, kw
    for kw in (dict(dtype=0), dict(c=cfg(algo=1)), dict(c=cfg(fuse_depth=1))):
        assert ckpt(grad, **kw) == UNSUPPORTED, kw
    outs = {"dx", "dw_in", "dw_out"} if grad else {"y", "ckpt"}
    for i in range(n):
        b = [buf(k) for k in range(n)]
        b[i] = ccgpu.RankBuf(None, 1 << 20)
        assert ckpt(grad, b) == INVALID
        b[i] = buf(i, 60)
        assert ckpt(grad, b) == INVALID
        b[i] = buf(i, off=1)
        assert ckpt(grad, b) == INVALID
        b[i] = buf(i, off=4)
        assert ckpt(grad, b) == (INVALID if names[i] == "ckpt" else NO_DEVICE)      # checkpoints on 16 bytes
        b[i] = buf(i, (1 << 20) + 4)
        assert ckpt(grad, b) == (INVALID if names[i] == "ckpt" else NO_DEVICE)
        b[i] = buf((i + 1) % n, off=64)
        assert ckpt(grad, b) == (INVALID if outs & {names[i], names[(i + 1) % n]} else NO_DEVICE)
    need = ccgpu.moe_ffn_checkpoint_workspace_size(TWO, 5, 8, 16, "f32", grad)
    assert ckpt(grad, c=cfg(workspace_bytes=need)) == NO_DEVICE
    for c in (cfg(workspace_bytes=need - 1), cfg(workspace=None), cfg(workspace=FAKE + 100 * GB + 8), cfg(workspace=FAKE + GB)):
        assert ckpt(grad, c=c) == INVALID
    none = [NONE if names[k] in ("x", "ckpt", "y", "dy", "dx") else buf(k) for k in range(n)]
    assert ckpt(grad, none, cap=0) == (NO_DEVICE if grad else OK)                   # the weights' zero gradients
    assert ckpt(grad, none, counts=[0] * 8, cap=0) == (NO_DEVICE if grad else OK)


def test_checkpoint_workspace_holds_the_rows_x():
    args = [[64, 64], [64, 64]], 64, 128, 256, "bf16"
    assert ccgpu.moe_ffn_checkpoint_workspace_size(*args) == ccgpu.moe_ffn_workspace_size(*args)
    assert ccgpu.moe_ffn_checkpoint_workspace_size(*args, True) >= ccgpu.moe_ffn_workspace_size(*args, True) + 256 * 128 * 2


def test_binding_checks_shapes_and_types():
    import torch
    z, i32, i8, u8 = torch.zeros, torch.int32, torch.int8, torch.uint8
    with pytest.raises(ValueError, match="total"):
        ccgpu.moe_balance_loss_grad(z(2, 8), z(2, 1, dtype=i32), z(2, 1), z(2, 8))
    with pytest.raises(ValueError, match="logits"):
        ccgpu.moe_balance_loss(z(2, 7), z(2, 3, dtype=i32), z(2, 4, dtype=i32), z(2, 3), z(2, 1))
    with pytest.raises(ValueError, match="device tensors"):
        ccgpu.moe_balance_loss(z(2, 6), z(2, 3, dtype=i32), z(2, 4, dtype=i32), z(2, 3), z(2, 1))
    with pytest.raises(ValueError, match="x must be"):
        ccgpu.quantize_rows(z(2, 7), z(2, 7, dtype=i8), z(2, 1), 4)
    with pytest.raises(ValueError, match="experts"):
        ccgpu.moe_matmul_int8(z(2, 8, dtype=i8), z(2, 2), z(2, 8, dtype=i8), z(2, 2), z(2, 4), [[1, 1, 1], [1, 1, 1]], 1, 4)
    with pytest.raises(ValueError, match="x must be torch.int8"):
        ccgpu.moe_matmul_int8(z(2, 8), z(2, 2), z(2, 8, dtype=i8), z(2, 2), z(2, 4), [[1, 1], [1, 1]], 1, 4)
    with pytest.raises(ValueError, match="counts"):
        ccgpu.moe_ffn_int8(z(2, 8), z(2, 16, dtype=i8), z(2, 4), z(2, 8, dtype=i8), z(2, 4), z(2, 8), [[1, 1], [1]], 1, 4)
    with pytest.raises(ValueError, match="x must be"):
        ccgpu.moe_ffn_checkpoint(z(2, 9), z(2, 32), z(2, 16), z(2, 96, dtype=u8), z(2, 8), [[1, 1], [1, 1]], 1, 4)
    with pytest.raises(ValueError, match="2 x 2"):
        ccgpu.make_moe_ffn_checkpoint([[1, 1], [1]], 1, 4, 4)
