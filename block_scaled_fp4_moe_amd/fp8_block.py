"""The block-scaled FP8 operators (C ABI in include/fp8block.h).

    rms_norm_fp8            RMS norm of x + residual, quantized 1x128
    swiglu_fp8              SiLU(gate) * up, quantized 1x128
    fp8_block_linear        E4M3 x E4M3 product with 1x128 / 128x128 scales
    fp8_block_grouped_gemm  the same per expert, over moe_permute's segments

Signatures only: the native module _fp8_block checks the arguments (ValueError),
allocates outputs that are not passed in and calls the library (FP4MoEError for
what that refuses).  Codes are uint8 or torch.float8_e4m3fn tensors; activation
scales are float32 [rows, ceil(K/128)] tensors of any strides (as outputs, of any that
keep the elements apart; allocated with the scales of one K block side by side, the
order the products read).  An output may not overlap an input.  Work and
allocations go to `stream`, the current one by default.
"""

import torch

from . import FP4MoEError, load

_OUT = {torch.bfloat16: 0, torch.float16: 1}
_raw_stream = torch._C._cuda_getCurrentRawStream if torch.cuda._is_compiled() else None


class _Native:
    """The native module, loaded with the library at the first call (there is no
    fallback: a missing build raises)."""

    def __getattr__(self, name):
        load()
        from . import _fp8_block
        _fp8_block.set_error_class(FP4MoEError)
        for f in ("rms_norm_fp8", "swiglu_fp8", "fp8_block_linear", "fp8_block_grouped_gemm"):
            setattr(self, f, getattr(_fp8_block, f))
        return getattr(_fp8_block, name)


_native = _Native()


def _on(stream, lead, function, *args):
    """function on the current stream of lead's device, or on `stream` with its
    allocations made there."""
    if stream is None:
        index = lead.device.index
        return function(*args, 0 if index is None else _raw_stream(index))
    with torch.cuda.stream(stream):
        return function(*args, stream.cuda_stream)


def rms_norm_fp8(x, weight, eps=1e-6, residual=None, residual_out=None, y=None, codes=None,
                 scales=None, stream=None, quantize=True):
    """v = x + residual; y = v * weight / sqrt(mean(v^2) + eps), quantized 1x128.

    x, residual [M, K] and weight [K] of one dtype (bfloat16, float16 or
    float32).  Returns (codes uint8 [M, K], scales float32 [M, ceil(K/128)],
    residual_out): residual_out is v rounded to the dtype (None without a
    residual; a new tensor unless one is passed).  y: a tensor that receives the
    normalised rows in the dtype.  residual_out and y may each be x or residual itself;
    any other overlap of an output is refused.  quantize=False: y and residual_out alone
    are written (for a layer that takes the rows themselves); codes and scales are None."""
    if not quantize:
        if codes is not None or scales is not None:
            raise ValueError("codes and scales are not written with quantize=False")
        codes = False
    return _on(stream, x, _native.rms_norm_fp8, x, weight, eps, residual, residual_out, y, codes,
               scales)


def swiglu_fp8(gate_up, row_count=None, codes=None, scales=None, stream=None):
    """SiLU(gate) * up of gate_up [M, 2I] (gate columns first), quantized 1x128.

    row_count: int32 [1] on the device; rows at or past it are not written.
    Returns (codes uint8 [M, I], scales float32 [M, ceil(I/128)])."""
    return _on(stream, gate_up, _native.swiglu_fp8, gate_up, row_count, codes, scales)


def _out_code(dtype):
    code = _OUT.get(dtype)
    if code is None:
        raise ValueError(f"out_dtype {dtype} is not bfloat16 or float16")
    return code


def fp8_block_linear(a, a_scale, w, w_scale, out=None, out_dtype=torch.bfloat16, stream=None):
    """out [M, N] = (a * a_scale) . (w * w_scale)^T.

    a codes [M, K], a_scale float32 [M, ceil(K/128)], w codes [N, K], w_scale
    float32 [ceil(N/128), ceil(K/128)]; K and the row strides multiples of 16.  out: a
    bfloat16 or float16 tensor, whose own type then counts."""
    return _on(stream, a, _native.fp8_block_linear, a, a_scale, w, w_scale, out,
               _out_code(out_dtype))


def fp8_block_grouped_gemm(a, a_scale, w, w_scale, perm, block_m, a_row_gather=None, gather_div=1,
                           out=None, out_dtype=torch.bfloat16, stream=None):
    """The product per expert over the segments of `perm` (moe_permute's dict for
    the same block_m: 16, 32, 64 or 128).

    w codes [E, N, K], w_scale float32 [E, ceil(N/128), ceil(K/128)].  Sorted row
    r reads row a_row_gather[r] // gather_div of a when a gather is given, else
    row r.  Returns out [rows, N], rows = the length of perm["sorted_pairs"];
    rows outside every segment are left as they are."""
    return _on(stream, a, _native.fp8_block_grouped_gemm, a, a_scale, w, w_scale, out,
               _out_code(out_dtype), perm["expert_offsets"], perm["sorted_pairs"], perm["tiles"],
               perm["n_tiles"], perm["max_tiles"], block_m, a_row_gather, gather_div)
