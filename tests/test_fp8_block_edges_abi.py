"""What the C ABI of the block-scaled FP8 operators refuses because of where the outputs
lie, on the host: no call here reaches a device (a valid one stops at the missing GPU)."""

import ctypes

import pytest
import torch

from .test_fp8_block_abi import NormArgs, _lib, _message

pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="its pointers are not memory")


def norm(**kw):
    a = NormArgs(dtype=0, M=2, K=64, eps=1e-6, x=4096, ldx=64, weight=65536, codes=131072, ldc=64,
                 scales=196608, scale_row=1, scale_blk=2)
    for k, v in kw.items():
        setattr(a, k, v)
    return _lib().rms_norm_fp8(ctypes.byref(a), None)


# M, K, row stride, block stride, whether every element has a place of its own
STRIDES = [
    (3, 384, 1, 3, True), (3, 384, 3, 1, True), (3, 384, 7, 2, True), (3, 384, 3, 2, True),
    (3, 384, 0, 1, False), (3, 384, 1, 0, False), (3, 384, 0, 0, False), (3, 384, 1, 1, False),
    (3, 384, 1, 2, False), (3, 384, 2, 1, False), (3, 384, 4, 2, False), (3, 384, 6, 4, True),
    (1, 384, 0, 1, True), (1, 384, 5, 0, False), (3, 128, 1, 0, True), (3, 128, 0, 9, False),
    (1, 128, 0, 0, True), (4, 300, 2, 3, False), (3, 300, 2, 3, True)]


@pytest.mark.parametrize("M,K,row,blk,apart", STRIDES)
def test_scales_of_an_output_lie_apart(M, K, row, blk, apart):
    places = [i * row + b * blk for i in range(M) for b in range(-(-K // 128))]
    assert (len(set(places)) == len(places)) == apart            # the table itself
    st = norm(M=M, K=K, ldx=K, ldc=K, scale_row=row, scale_blk=blk)
    assert (st == 1) == (not apart)
    if not apart:
        assert "rms_norm_fp8: scale strides" in _message()
    st = _lib().swiglu_fp8(0, 4096, M, K, 2 * K, None, 131072, K, 196608, row, blk, None)
    assert (st == 1) == (not apart)
    if not apart:
        assert "swiglu_fp8: scale strides" in _message()
