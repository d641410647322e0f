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


X, R, W, C, S, O = (i << 24 for i in range(1, 7))        # far apart


def packed(**kw):
    """Rows of 64 bfloat16 (128 bytes), four of them, everything apart."""
    a = dict(M=4, K=64, x=X, ldx=64, residual=R, ldr=64, weight=W, codes=C, ldc=64, scales=S,
             scale_row=1, scale_blk=4)
    a.update(kw)
    return norm(**a)


@pytest.mark.parametrize("fine", [
    dict(), dict(residual_out=X, ldro=64), dict(residual_out=R, ldro=64), dict(y_out=X, ldy=64),
    dict(residual_out=R, ldro=64, y_out=X, ldy=64), dict(residual_out=O, ldro=80),
    # column ranges of one buffer, in any order
    dict(ldx=200, residual_out=X + 128, ldro=200), dict(x=X + 272, ldx=200, residual_out=X, ldro=200),
    dict(ldx=200, codes=X + 128, ldc=400, scales=X + 192, scale_row=100),
    # behind the last row, before the first
    dict(residual_out=X + 512, ldro=64), dict(residual_out=X - 512, ldro=64),
    dict(ldx=100, residual_out=X + 728, ldro=64), dict(weight=X + 512), dict(weight=X - 128),
    # of a single row the stride says nothing
    dict(M=1, residual_out=X, ldro=99), dict(ldx=200, weight=X + 128),
    dict(codes=C, scales=C + 256), dict(codes=C, ldc=68, scales=C + 64, scale_row=17),
    dict(codes=None, scales=None, y_out=O, ldy=64)])
def test_norm_takes_outputs_that_lie_apart_or_on_an_input(fine):
    assert packed(**fine) != 1, _message()


@pytest.mark.parametrize("bad,which", [
    (dict(residual_out=X, ldro=72), "residual_out"), (dict(residual_out=R, ldro=128), "residual_out"),
    (dict(residual_out=X + 128, ldro=64), "residual_out"), (dict(residual_out=X - 384, ldro=64), "residual_out"),
    (dict(residual_out=X + 2, ldro=64), "residual_out"), (dict(ldx=200, residual_out=X + 126, ldro=200), "residual_out"),
    (dict(ldx=200, residual_out=X + 274, ldro=200), "residual_out"),
    (dict(y_out=X + 2, ldy=64), "y_out"), (dict(y_out=W - 510, ldy=64), "y_out"),
    (dict(residual_out=O, ldro=64, y_out=O, ldy=64), "y_out"),
    (dict(codes=X), "codes"), (dict(codes=W + 127), "codes"), (dict(codes=R + 511), "codes"),
    (dict(residual_out=O, ldro=64, codes=O + 511), "codes"),
    (dict(scales=X + 508), "scales"), (dict(scales=C), "scales"), (dict(scales=C + 252), "scales"),
    (dict(codes=C, ldc=68, scales=C + 60, scale_row=17), "scales"),
    (dict(y_out=O, ldy=64, scales=O - 12), "scales")])
def test_norm_refuses_other_overlaps(bad, which):
    assert packed(**bad) == 1 and f"rms_norm_fp8: {which} overlaps" in _message()
