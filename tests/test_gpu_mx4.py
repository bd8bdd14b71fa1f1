"""Microscaled 4-bit matrices on the GPU: codes and scale tiles equal the plain
64-bit reference bit for bit, and reading them back is exact."""
import numpy as np
import pytest
import torch

import mx4_ref
import sparse_moe_layer_top_b200 as moe

pytestmark = pytest.mark.gpu


def _rand(shape, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(shape, generator=g)
    # blocks of very different size: exponents spread over 2^-20 .. 2^20
    e = torch.randint(-20, 21, tuple(shape[:-1]) + (shape[-1] // 32,), generator=g).float()
    return (x * torch.exp2(e).repeat_interleave(32, -1)).to(dtype)


SHAPES = [(1, 32), (16, 2048), (128, 128), (129, 160), (127, 96), (3, 5, 64), (2, 3, 130, 224), (300, 1376), (4, 256, 512)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("shape", SHAPES)
def test_quantize_equals_the_reference_bit_for_bit(shape, dtype):
    x = _rand(shape, dtype, sum(shape))
    codes, scales = moe.quantize_mx4(x.cuda())
    c, b = mx4_ref.quantize(x)
    assert np.array_equal(codes.cpu().numpy(), c)
    assert np.array_equal(scales.cpu().numpy(), mx4_ref.tiles(b))
    v = mx4_ref.values(c, b)
    for dt in (torch.bfloat16, torch.float32):
        out = moe.dequantize_mx4(codes, scales, dtype=dt)
        assert out.dtype == dt and np.array_equal(out.double().cpu().numpy(), v)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_special_blocks(dtype):
    x = torch.zeros(14, 64)
    x[0, 3] = -0.0
    x[1, 0] = float("inf")
    x[2, 40] = float("nan")
    x[3, :32] = torch.linspace(-6, 6, 32)
    x[4, 0] = torch.finfo(dtype).max
    x[5, 0] = torch.finfo(dtype).tiny
    x[6, 7] = 2.0 ** -133  # a bf16 subnormal
    x[7, :16] = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.0] * 2)  # the middles, below a largest of 7
    x[8, :16] = -x[7, :16]
    x[9] = 1.0
    x[10, 31] = 2.0 ** -126
    x[11, 32:] = 2.0 ** 100
    x[12, 0], x[12, 1] = 2.0 ** 127, 2.0 ** -126
    x = x.to(dtype)
    codes, scales = moe.quantize_mx4(x.cuda())
    c, b = mx4_ref.quantize(x)
    assert np.array_equal(codes.cpu().numpy(), c)
    assert np.array_equal(scales.cpu().numpy(), mx4_ref.tiles(b))
    v = mx4_ref.values(c, b)
    got = moe.dequantize_mx4(codes, scales, dtype=torch.float32).double().cpu().numpy()
    assert np.array_equal(got, v, equal_nan=True)
    assert np.isnan(v[1, :32]).all() and not np.isnan(v[1, 32:]).any()


def test_every_code_and_scale_byte_reads_back():
    """All 16 codes under all 256 scale bytes: exact in fp32 (past its largest
    value infinity, byte 255 NaN)."""
    byte = torch.arange(256, dtype=torch.uint8).reshape(128, 2).repeat(1, 2)  # [128, 4] blocks
    codes = torch.arange(256, dtype=torch.uint8).reshape(16, 16)[torch.arange(128) % 16].repeat(1, 4)  # [128, 64]
    v = mx4_ref.values(codes.numpy(), byte.numpy())
    ref = torch.from_numpy(v).float().double().numpy()
    s = moe.mx4_scale_tiles(byte).cuda()
    for dt in (torch.float32, torch.bfloat16):
        out = moe.dequantize_mx4(codes.cuda(), s, dtype=dt).double().cpu().numpy()
        want = ref if dt == torch.float32 else torch.from_numpy(v).to(torch.bfloat16).double().numpy()
        assert np.array_equal(out, want, equal_nan=True)


def test_given_buffers_streams_and_empty_inputs():
    x = _rand((130, 96), torch.bfloat16, 3).cuda()
    ref = moe.quantize_mx4(x)
    codes = torch.full((140, 48), 99, dtype=torch.uint8, device="cuda")
    scales = torch.full((3, 1, 512), 99, dtype=torch.uint8, device="cuda")
    out = torch.full((140, 96), 7.0, dtype=torch.bfloat16, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    moe.quantize_mx4(x, codes, scales, stream=s)
    moe.dequantize_mx4(codes[:130], scales, out=out, stream=s)
    s.synchronize()
    assert torch.equal(codes[:130], ref[0]) and torch.equal(scales[:2], ref[1])
    assert (codes[130:] == 99).all() and (scales[2] == 99).all()  # past the matrix: left alone
    assert torch.equal(out[:130], moe.dequantize_mx4(*ref)) and (out[130:] == 7).all()
    for shape in ((0, 64), (0, 3, 64), (2, 0, 64)):
        c, sc = moe.quantize_mx4(torch.zeros(shape, device="cuda"))
        assert c.shape == shape[:-1] + (32,) and moe.dequantize_mx4(c, sc).shape == shape


def test_a_matrix_past_32_bit_offsets():
    """4.3e9 values: the last rows are addressed past 2^32 elements."""
    rows, cols = 524416, 8192
    x = torch.zeros((rows, cols), dtype=torch.bfloat16, device="cuda")
    tail = _rand((200, cols), torch.bfloat16, 5)
    x[-200:] = tail.cuda()
    codes, scales = moe.quantize_mx4(x)
    c, b = mx4_ref.quantize(tail)
    assert np.array_equal(codes[-200:].cpu().numpy(), c)
    out = moe.dequantize_mx4(codes, scales, out=x)
    assert np.array_equal(out[-200:].double().cpu().numpy(), mx4_ref.values(c, b))
    assert (out[:128] == 0).all()
