"""The block-scaled FP8 operators at the ends of their ranges, on the GPU against 64-bit
forms (tolerances as in test_gpu_fp8_block.py)."""

import numpy as np
import pytest
import torch

from .test_gpu_fp8_block import (DTYPES, NORM, SILU, check_product, check_quantized,
                                 check_rounded, gen, quantized_pair, randn, silu_mul64)

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


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("K", [256, 20480])
def test_norm_of_rows_with_a_subnormal_mean_square(gpu_lib, K, dtype):
    """Powers of two without eps: squares and their sums are exact, y = sign(x) * weight."""
    g = gen(52)
    size = 2.0 ** torch.tensor([[-60.0], [-66.0], [-69.0], [-72.0]])
    x = (torch.sign(randn(g, 4, K)) * size).to(DTYPES[dtype]).cuda()
    w = (1 + 0.3 * randn(g, K)).to(DTYPES[dtype]).cuda()
    y = torch.empty_like(x)
    c, s, _ = gpu_lib.rms_norm_fp8(x, w, eps=0.0, y=y)
    ref = torch.sign(x).double().cpu().numpy() * w.double().cpu().numpy()
    check_quantized(c, s, ref, NORM, "subnormal")
    check_rounded(y, ref, NORM * np.abs(ref), "y")


def test_norm_of_a_zero_row_without_eps(gpu_lib):
    """0 / 0: NaN throughout, as the formula gives; the row beside it is not touched by it."""
    x = torch.ones((2, 256), device="cuda")
    x[0] = 0
    c, s, _ = gpu_lib.rms_norm_fp8(x, torch.ones(256, device="cuda"), eps=0.0)
    q = c.view(torch.float8_e4m3fn).float()
    assert bool(s[0].isnan().all()) and bool(q[0].isnan().all())
    assert bool((q[1] == 448).all())


@pytest.mark.parametrize("N", [2 ** 24 + 40, 2 ** 31 - 8, 2 ** 31 - 1])
def test_linear_up_to_the_largest_row_count(gpu_lib, N):
    """More items than a grid holds, and N next to 2^31: sampled weight rows from the whole
    range, the first turn of the item loop and the last."""
    if torch.cuda.mem_get_info()[0] < N * 20:
        pytest.skip("not enough free memory")
    a, sa, w16, sw = quantized_pair(gen(7), 1, 64, 16, whole=True)
    w = torch.zeros((N, 16), dtype=torch.uint8, device="cuda")
    at = torch.tensor([0, 17, 2 ** 23 + 5, 2 ** 24 + 16, N - 30, N - 9, N - 8, N - 2, N - 1], device="cuda")
    w[at] = w16[:9]
    one = sw[:1].expand((N + 127) // 128, 1)
    out = torch.full((1, N), 7.0, dtype=torch.bfloat16, device="cuda")
    gpu_lib.fp8_block_linear(a, sa, w, one, out=out)
    check_product(out[:, at], a, sa, w16[:9], sw, "rows", True)
    for lo in range(0, N, 2 ** 28):
        assert not bool((out[0, lo:lo + 2 ** 28] == 7.0).any())
    del w, out
    torch.cuda.empty_cache()


def test_scales_on_top_of_each_other_are_refused(gpu_lib):
    x, w = torch.ones((4, 256), device="cuda"), torch.ones(128, device="cuda")
    with pytest.raises(gpu_lib.FP4MoEError):
        gpu_lib.rms_norm_fp8(x[:, :128], w, scales=torch.empty((1, 1), device="cuda").expand(4, 1))
    with pytest.raises(gpu_lib.FP4MoEError):
        gpu_lib.swiglu_fp8(x, scales=torch.empty((1, 1), device="cuda").expand(4, 1))


@pytest.mark.parametrize("K,M", [(640, 12), (7168, 300), (20480, 3)])
def test_norm_y_and_residual_in_place(gpu_lib, K, M):
    """y on x and residual_out on residual at once, in every kind of kernel; an output
    that is shifted against its input is refused."""
    g = gen(K)
    x, r = randn(g, M, K).bfloat16().cuda(), randn(g, M, K).bfloat16().cuda()
    w = (1 + 0.3 * randn(g, K)).bfloat16().cuda()
    y = torch.empty_like(x)
    c, s, ro = gpu_lib.rms_norm_fp8(x, w, residual=r, y=y)
    x2, r2 = x.clone(), r.clone()
    c2, s2, ro2 = gpu_lib.rms_norm_fp8(x2, w, residual=r2, residual_out=r2, y=x2)
    assert ro2 is r2 and torch.equal(r2, ro) and torch.equal(x2, y)
    assert torch.equal(c, c2) and torch.equal(s, s2)
    with pytest.raises(gpu_lib.FP4MoEError):
        gpu_lib.rms_norm_fp8(x[:-1], w, residual=r[:-1], residual_out=r[1:])


def test_a_single_row_may_have_any_stride(gpu_lib):
    """One row cut out of a buffer whose rows are not 16 bytes apart, on every side."""
    a, sa, w, sw = quantized_pair(gen(1), 2, 40, 256)

    def cut(t, pad):
        room = torch.zeros((t.shape[0], t.shape[1] + pad), dtype=t.dtype, device="cuda")
        room[:, :t.shape[1]] = t
        return room[:1, :t.shape[1]]

    want = gpu_lib.fp8_block_linear(a, sa, w, sw)
    out = torch.zeros((1, 43), dtype=torch.bfloat16, device="cuda")[:, :40]
    got = gpu_lib.fp8_block_linear(cut(a, 4), cut(sa, 1), w, cut(sw, 3), out=out)
    assert got is out and torch.equal(got, want[:1])
    assert torch.equal(gpu_lib.fp8_block_linear(a, sa, cut(w, 12), sw), want[:, :1])
    perm = dict(expert_offsets=torch.tensor([0, 1], dtype=torch.int32, device="cuda"),
                sorted_pairs=torch.zeros(1, dtype=torch.int32, device="cuda"),
                tiles=torch.zeros((1, 2), dtype=torch.int32, device="cuda"),
                n_tiles=torch.ones(1, dtype=torch.int32, device="cuda"), max_tiles=1)
    got = gpu_lib.fp8_block_grouped_gemm(cut(a, 4), cut(sa, 1), cut(w, 12)[None], sw[None], perm, 16)
    assert torch.equal(got, want[:1, :1])


def test_an_output_that_does_not_fit(gpu_lib):
    """torch's own out-of-memory error, as from any allocation; the next call works."""
    a = torch.zeros((1, 256), dtype=torch.uint8, device="cuda").expand(2 ** 31 - 1, 256)
    sa = torch.ones((1, 2), device="cuda").expand(2 ** 31 - 1, 2)
    w = torch.zeros((8192, 256), dtype=torch.uint8, device="cuda")
    sw = torch.ones((64, 2), device="cuda")
    with pytest.raises(torch.OutOfMemoryError):
        gpu_lib.fp8_block_linear(a, sa, w, sw)               # 32 TiB
    assert not bool(gpu_lib.fp8_block_linear(a[:3].contiguous(), sa[:3], w, sw).any())


@pytest.mark.parametrize("K", [640, 7168, 20480])
def test_norm_for_a_layer_that_takes_the_rows(gpu_lib, K):
    """quantize=False: y and the residual stream as with codes; nothing else is asked for."""
    g = gen(K + 1)
    x, r = randn(g, 9, K).bfloat16().cuda(), randn(g, 9, K).bfloat16().cuda()
    w = (1 + 0.3 * randn(g, K)).bfloat16().cuda()
    y, y2 = torch.empty_like(x), torch.empty_like(x)
    _, _, ro = gpu_lib.rms_norm_fp8(x, w, residual=r, y=y)
    c, s, ro2 = gpu_lib.rms_norm_fp8(x, w, residual=r, y=y2, quantize=False)
    assert c is None and s is None and torch.equal(ro, ro2) and torch.equal(y, y2)
    c, s, none = gpu_lib.rms_norm_fp8(x, w, y=x, quantize=False)
    assert c is None and none is None
    with pytest.raises(ValueError):
        gpu_lib.rms_norm_fp8(x, w, y=y, scales=torch.empty((9, K // 128), device="cuda"), quantize=False)
    with pytest.raises(gpu_lib.FP4MoEError):              # nothing to write
        gpu_lib.rms_norm_fp8(x, w, quantize=False)
