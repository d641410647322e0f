"""The FP8 feed-forward blocks: types that they do not take are refused before any work."""

import pytest
import torch

import block_scaled_fp4_moe_amd as fm


def blocks(device, dtype):
    codes = lambda *s: torch.zeros(s, dtype=torch.uint8, device=device)      # noqa: E731
    ones = lambda *s: torch.ones(s, device=device)                           # noqa: E731
    norm = torch.ones(128, dtype=dtype, device=device)
    mlp = fm.FP8BlockMLP(norm, codes(256, 128), ones(2, 1), codes(128, 128), ones(1, 1))
    cfg = fm.FP8BlockMoEConfig(4, 0, 1, 1, 2)
    return mlp, fm.FP8BlockMoE(cfg, norm, codes(4, 256, 128), ones(4, 2, 1), codes(4, 128, 128),
                               ones(4, 1, 1), router=ones(4, 128))


@pytest.mark.parametrize("device", ["cpu", pytest.param("cuda", marks=pytest.mark.gpu)])
def test_types_are_refused_first(device):
    if device == "cuda" and not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    x = torch.zeros((3, 128), device=device)
    with pytest.raises(ValueError, match="wanted bfloat16 or float16"):
        blocks(device, torch.float32)[0].forward(x)
    for dtype in (torch.float16, torch.float32):
        with pytest.raises(ValueError, match="wanted bfloat16"):
            blocks(device, dtype)[1].forward(x.to(dtype), x.to(dtype))


@pytest.mark.gpu
def test_an_empty_batch(gpu_lib):
    mlp, moe = blocks("cuda", torch.bfloat16)
    x = torch.zeros((0, 128), dtype=torch.bfloat16, device="cuda")
    for layer in (mlp, moe):
        out, residual = layer.forward(x, x)
        assert out.shape == (0, 128) and residual.shape == (0, 128)
        assert out.dtype == residual.dtype == torch.bfloat16
