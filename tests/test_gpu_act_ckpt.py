"""8-bit activation checkpoints on the GPU: every code and scale byte equals the definition's (the
scales are powers of two, so nothing but the code itself is rounded)."""
import numpy as np
import pytest
import torch

from oracle import block as B

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16
FORMATS = ["int8", "e4m3"]


def n64(t):
    return t.double().cpu().numpy()


def code_bytes(saved):
    return saved.codes.view(torch.uint8).cpu().numpy(), saved.scales.cpu().numpy()


def check(rlk, x, fmt):
    saved = rlk.act_quantize(x, fmt)
    codes, scales = code_bytes(saved)
    want_codes, want_scales = B.quantize(n64(x), fmt)
    assert np.array_equal(scales, want_scales)
    assert np.array_equal(codes, want_codes)
    back = rlk.act_dequantize(saved)
    want = B.dequantize(want_codes, want_scales, fmt)
    assert np.array_equal(n64(back), want, equal_nan=True)
    return saved, back


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("T,H", [(1, 64), (3, 192), (17, 1024), (5, 8192), (33, 4160), (2, 16448)])
def test_parity(rlk, cuda_device, T, H, fmt):
    g = torch.Generator(device=cuda_device)
    g.manual_seed(T * H)
    x = torch.randn(T, H, generator=g, device=cuda_device) * torch.exp(4 * torch.randn(T, 1, generator=g, device=cuda_device))
    x[:, :: 97] *= 80
    x[0, :32] = 0
    x = x.to(BF16)
    _, back = check(rlk, x, fmt)
    # a value that a checkpoint holds stays what it is
    again = rlk.act_dequantize(rlk.act_quantize(back, fmt))
    assert torch.equal(again, back)
    # half a step: 2^-7 of the block's largest power of two, or 2^-4 of the feature and 2^-10 of its scale
    top = np.repeat(np.abs(n64(x)).reshape(T, -1, 32).max(2), 32, 1)
    power = 2.0 ** np.floor(np.log2(np.where(top > 0, top, 1)))
    off = np.abs(n64(back) - n64(x))
    assert np.all(off <= (2.0 ** -7 * power if fmt == "int8" else np.maximum(2.0 ** -4 * np.abs(n64(x)), 2.0 ** -17 * power)))


@pytest.mark.parametrize("fmt", FORMATS)
def test_every_magnitude(rlk, cuda_device, fmt):
    """Each of the 32768 non-negative bf16 numbers and its negative, infinities and NaN among them,
    as a block's largest and below every larger power of two."""
    bits = torch.arange(32768, dtype=torch.int32, device=cuda_device)
    alone = torch.zeros((32768, 64), dtype=torch.int32, device=cuda_device)
    alone[:, 3] = bits
    alone[:, 40] = bits + 32768
    check(rlk, alone.to(torch.int16).view(BF16), fmt)
    # 31 smaller ones under a power of two
    powers = torch.arange(0, 255, 2, dtype=torch.int32, device=cuda_device) << 7
    g = torch.Generator(device=cuda_device)
    g.manual_seed(7)
    rows = torch.randint(0, 2 ** 30, (powers.numel(), 64), generator=g, device=cuda_device, dtype=torch.int32)
    low = (powers - 7 * 128).clamp(min=0)[:, None]
    rows = low + rows % (powers[:, None] - low + 1) + (rows % 7 // 4) * 32768
    rows[:, ::32] = powers[:, None]
    check(rlk, rows.to(torch.int16).view(BF16), fmt)


@pytest.mark.parametrize("fmt", FORMATS)
def test_not_a_number_stays_in_its_block(rlk, cuda_device, fmt):
    x = torch.ones((4, 128), dtype=BF16, device=cuda_device)
    x[1, 40], x[2, 5], x[3, 127] = float("nan"), float("inf"), -float("inf")
    saved, back = check(rlk, x, fmt)
    bad = torch.zeros((4, 4), dtype=torch.bool, device=cuda_device)
    bad[1, 1] = bad[2, 0] = bad[3, 3] = True
    assert torch.equal(saved.scales == 255, bad)
    assert torch.equal(torch.isnan(back), bad.repeat_interleave(32, 1))
    assert torch.all(back[~bad.repeat_interleave(32, 1)] == 1)


@pytest.mark.parametrize("fmt", FORMATS)
def test_canaries_streams_graph(rlk, cuda_device, fmt):
    T, H = 37, 320
    sets = [torch.randn(T, H, device=cuda_device).to(BF16) for _ in range(2)]
    want = [rlk.act_quantize(x, fmt) for x in sets]
    codes = torch.zeros((T + 2, H), dtype=torch.uint8, device=cuda_device) + 77
    scales = torch.zeros(T * H // 32 + 9, dtype=torch.uint8, device=cuda_device) + 77
    out = rlk.Saved(codes[1:T + 1].view(rlk.SAVED_DTYPES[fmt]), scales[5:5 + T * H // 32].view(T, H // 32))
    s = torch.cuda.Stream(cuda_device)
    s.wait_stream(torch.cuda.current_stream(cuda_device))
    got = rlk.act_quantize(sets[0], fmt, out=out, stream=s)
    back = rlk.act_dequantize(got, stream=s)
    s.synchronize()
    assert torch.equal(got.codes.view(torch.uint8), want[0].codes.view(torch.uint8)) and torch.equal(got.scales, want[0].scales)
    assert torch.all(codes[0] == 77) and torch.all(codes[T + 1] == 77)
    assert torch.all(scales[:5] == 77) and torch.all(scales[5 + T * H // 32:] == 77)
    assert torch.equal(back, rlk.act_dequantize(want[0]))
    held = sets[0].clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        again = rlk.act_dequantize(rlk.act_quantize(held, fmt))
    held.copy_(sets[1])
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(again, rlk.act_dequantize(want[1]))


def test_more_than_2_31_elements(rlk, cuda_device):
    T, H = 262147, 8192
    x = torch.zeros((T, H), dtype=BF16, device=cuda_device)
    x[-3:] = torch.randn(3, H, device=cuda_device).to(BF16)
    for fmt in FORMATS:
        saved = rlk.act_quantize(x, fmt)
        part = rlk.act_quantize(x[-3:], fmt)
        assert torch.equal(saved.codes[-3:].view(torch.uint8), part.codes.view(torch.uint8))
        assert torch.equal(saved.scales[-3:], part.scales) and not saved.scales[:-3].any()
        back = rlk.act_dequantize(saved)
        assert torch.equal(back[-3:], rlk.act_dequantize(part)) and not back[:-3].any()
        del saved, back


def test_binding_checks(rlk, cuda_device):
    x = torch.zeros((4, 128), dtype=BF16, device=cuda_device)
    saved = rlk.act_quantize(x)
    assert rlk.act_quantize(x[:0]).codes.shape == (0, 128)
    assert rlk.act_dequantize(rlk.act_quantize(x[:0])).shape == (0, 128)
    for bad in (lambda: rlk.act_quantize(x, out=rlk.act_quantize(x, "e4m3")), lambda: rlk.act_quantize(x.half()),
                lambda: rlk.act_dequantize((saved.codes, saved.scales)),
                lambda: rlk.act_dequantize(rlk.Saved(saved.codes.view(torch.uint8), saved.scales))):
        with pytest.raises(TypeError):
            bad()
    for bad in (lambda: rlk.act_quantize(x[:, :96]), lambda: rlk.act_dequantize(rlk.Saved(saved.codes, saved.scales[:2])),
                lambda: rlk.act_quantize(x[:2], out=saved), lambda: rlk.act_quantize(x.t())):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(rlk.RlkError):
        rlk.act_quantize(x[:, :96].contiguous())
