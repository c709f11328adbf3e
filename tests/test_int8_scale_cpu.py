"""The scale's arithmetic as an argument of the 8-bit rows: what is refused before
any launch, and how often the two kinds differ (no GPU needed)."""
import numpy as np
import pytest

from ring_allreduce_reduction_02_amd import ccgpu
from test_abi_cpu import no_gpu_only
from test_model_cpu import COUNTS, INVALID, NO_DEVICE, NONE, OK, UNSUPPORTED, buf, cfg, sizes


def rows(scale, bufs=None, n=10, width=8, dtype=1, N=4, c=None):
    return ccgpu.raw("cc_quantize_rows_scaled", *(bufs or [buf(i) for i in range(3)]), n, width, scale, dtype, N, c or cfg(), None)


def ffn8(scale, bufs=None, counts=COUNTS, act=0, dtype=1, N=2, c=None):
    return ccgpu.raw("cc_moe_ffn_int8_scaled", *(bufs or [buf(i) for i in range(6)]), sizes(counts), 4, 5, 8, 16, act, scale, dtype, N,
                     c or cfg(), None)


@no_gpu_only
@pytest.mark.parametrize("scale", [0, 1])
@pytest.mark.parametrize("call", [rows, ffn8])
def test_either_scale_is_taken_and_checked_alike(call, scale):
    assert call(scale) == NO_DEVICE
    for kw in (dict(N=0), dict(N=65), dict(dtype=5)):
        assert call(scale, **kw) == INVALID, kw
    for kw in (dict(dtype=0), dict(c=cfg(algo=1))):
        assert call(scale, **kw) == UNSUPPORTED, kw
    if call is rows:
        assert call(scale, [NONE] * 3, n=0) == OK and call(scale, width=0) == INVALID
        assert call(scale, [buf(0), buf(0), buf(2)]) == INVALID
    else:
        assert call(scale, act=2) == INVALID and call(scale, c=cfg(workspace=None)) == INVALID


@pytest.mark.parametrize("scale", [-1, 2, 127, -(1 << 31), (1 << 31) - 1])
@pytest.mark.parametrize("call", [rows, ffn8])
def test_other_scales_are_refused(call, scale):
    assert call(scale) == INVALID and "scale" in ccgpu.load().cc_last_error().decode()


def test_the_binding_names_two():
    import torch
    x = torch.zeros(1, 8)
    assert ccgpu.SCALES == {"quotient": 0, "product": 1}
    with pytest.raises((KeyError, ValueError)):
        ccgpu.quantize_rows(x, x.to(torch.int8), torch.zeros(1, 2), 4, scale="other")


def test_the_two_scales_are_a_step_apart_in_a_twentieth_of_rows():
    top = np.random.default_rng(1).random(1 << 16, dtype=np.float32) + np.float32(0.5)
    quotient, product = top / np.float32(127), top * (np.float32(1) / np.float32(127))
    # 1 / 127 is off by at most U of its value before its product is rounded: two steps of 2 U between the results at most
    assert (np.abs(quotient.view(np.int32) - product.view(np.int32)) <= 2).all()
    assert 0.03 < (quotient != product).mean() < 0.07
