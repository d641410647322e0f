"""The block-scaled FP8 operators at the ends of their ranges, on the GPU against 64-bit
forms (tolerances as in test_gpu_fp8_block.py)."""

import numpy as np
import pytest
import torch

from .test_gpu_fp8_block import (DTYPES, NORM, SILU, check_product, check_quantized, gen,
                                 quantized_pair, randn, silu_mul64)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("lo,hi,up", [
    (-87.2, -80, 1e34),        # the float32 exponential next to its overflow
    (-88.6, -87.4, 1e35),      # its reciprocal subnormal
    (-103, -88.8, 1e38)])      # its overflow
def test_swiglu_gates_that_set_the_scale_from_far_below_zero(gpu_lib, dtype, lo, hi, up):
    """Every value of every block has such a gate and an up that brings it back."""
    g = gen(51)
    gate = lo + (hi - lo) * torch.rand((64, 256), generator=g)
    u = up * (0.5 + torch.rand((64, 256), generator=g)) * torch.sign(randn(g, 64, 256))
    gu = torch.cat([gate, u], 1).to(DTYPES[dtype]).cuda()
    c, s = gpu_lib.swiglu_fp8(gu)
    check_quantized(c, s, silu_mul64(gu), SILU, "low gates")


def test_swiglu_low_gates_do_not_depend_on_the_path(gpu_lib):
    """The same low-gate values beside partners that do and do not send their block to the
    64-bit form, and beside none: one scale, set by the low gate."""
    gate, up = -95.0, 3e38
    want = abs(gate / (1 + np.exp(-gate)) * up)
    gu = torch.zeros((400, 256), device="cuda")
    gu[:, 0], gu[:, 128] = gate, up
    gu[1:, 1], gu[1:, 129] = 40.0, float(want) / 40 * torch.linspace(0.01, 0.99, 399, device="cuda")
    c, s = gpu_lib.swiglu_fp8(gu)
    assert np.all(np.abs(s.double().cpu().numpy() * 448 / want - 1) <= SILU + 2.0 ** -23)
    check_quantized(c, s, silu_mul64(gu), SILU, "path")
