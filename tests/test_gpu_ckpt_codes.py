"""Restoring checkpoints of any codes and bytes, those that the quantiser never writes among them: the
definition's value rounded once to bf16 (a step of 2^-133 at the smallest, 2^128 and more infinite); with byte
255, which stands for a block that was not finite, zeros come back as NaN and all other codes as infinities."""
import numpy as np
import pytest
import torch

from oracle import block as B

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


def definition(codes, scales, fmt):
    """bf16 values as fp64; every code times its power of two is an fp32 number or beyond the largest."""
    s = np.repeat(scales.astype(np.float64), 32, axis=1)
    c = codes.view(np.int8).astype(np.float64) if fmt == "int8" else B.E4M3[codes]
    with np.errstate(over="ignore", invalid="ignore"):
        v = c * 2.0 ** (s - (133 if fmt == "int8" else 127))
        v = np.where(s == 255, c * np.inf, v).astype(np.float32)
    return torch.from_numpy(v).to(BF16)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_every_code_under_every_byte(rlk, cuda_device, fmt):
    codes = np.tile(np.arange(256, dtype=np.uint8), (256, 1))            # a row a byte
    scales = np.repeat(np.arange(256, dtype=np.uint8)[:, None], 8, axis=1)
    saved = rlk.Saved(torch.from_numpy(codes).to(cuda_device).view(rlk.SAVED_DTYPES[fmt]), torch.from_numpy(scales).to(cuda_device))
    back = rlk.act_dequantize(saved).cpu()
    want = definition(codes, scales, fmt)
    both_nan = torch.isnan(back) & torch.isnan(want)
    assert torch.equal(torch.isnan(back), torch.isnan(want))
    assert torch.equal(back.masked_fill(both_nan, 0).view(torch.int16), want.masked_fill(both_nan, 0).view(torch.int16))
    # what rounds at all: the smallest e4m3 codes under the bytes 0, 1 and 2
    exact = codes.view(np.int8) * 2.0 ** (scales.repeat(32, 1) - 133.0) if fmt == "int8" else B.E4M3[codes] * 2.0 ** (scales.repeat(32, 1) - 127.0)
    rounds = (want.double().numpy() != exact) & (np.abs(exact) < 2.0 ** 128) & (scales.repeat(32, 1) != 255)
    assert int(rounds.sum()) == (0 if fmt == "int8" else 96)
    assert np.unique(np.nonzero(rounds)[0]).tolist() == ([] if fmt == "int8" else [0, 1, 2])


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_the_quantiser_writes_none_that_round(rlk, cuda_device, fmt):
    """Every bf16 number below 2^-117 as a block's largest, with smaller ones of the same block's grid beside
    it: what comes back is codes times scale exactly."""
    top = torch.arange(1, 10 * 128, dtype=torch.int32, device=cuda_device)[:, None]
    below = torch.arange(64, dtype=torch.int32, device=cuda_device)[None]
    x = torch.where(below % 32 == 0, top, top * below // 64).to(torch.int16).view(BF16)
    saved = rlk.act_quantize(x, fmt)
    exact = B.dequantize(saved.codes.view(torch.uint8).cpu().numpy(), saved.scales.cpu().numpy(), fmt)
    assert np.array_equal(rlk.act_dequantize(saved).double().cpu().numpy(), exact)
