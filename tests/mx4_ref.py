"""Plain 64-bit reference of the microscaled 4-bit format, in numpy."""
import numpy as np
import torch

VALUES = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6], np.float64)


def quantize(x):
    """x [..., rows, cols] (tensor) -> (packed codes [..., rows, cols / 2], scale bytes [..., rows, cols / 32]).

    Codes are the nearest of the eight magnitudes; at an exact middle the even
    code."""
    v = x.detach().cpu().double().numpy()
    b = v.reshape(v.shape[:-1] + (-1, 32))
    amax = np.abs(b).max(-1)
    finite = np.isfinite(b).all(-1)
    e = np.frexp(np.where(finite, amax, 1.0))[1] - 1 - 2
    byte = np.where(amax > 0, np.maximum(e, -127) + 127, 127)
    byte = np.where(finite, byte, 255).astype(np.uint8)
    s = np.ldexp(1.0, byte.astype(np.int64) - 127)
    a = np.where(finite[..., None], np.abs(b) / s[..., None], 0.0)
    mid = (VALUES[1:] + VALUES[:-1]) / 2
    code = np.zeros(a.shape, np.int64)
    for i, m in enumerate(mid):  # past the middle to code i + 1; at it only when i + 1 is even
        code = np.where((a > m) | ((a == m) & ((i + 1) % 2 == 0)), i + 1, code)
    code = code + 8 * (np.signbit(b) & finite[..., None])
    code = code.reshape(v.shape).astype(np.uint8)
    return code[..., 0::2] | (code[..., 1::2] << 4), byte


def tiles(byte):
    """Scale bytes [..., rows, cols / 32] -> [..., row tiles, column tiles, 512], 127 past the end; one byte at a time."""
    lead, (R, C) = byte.shape[:-2], byte.shape[-2:]
    rt, ct = -(-R // 128), -(-C // 4)
    flat = byte.reshape((-1, R, C))
    out = np.full((flat.shape[0], rt, ct, 512), 127, np.uint8)
    for r in range(R):
        for c in range(C):
            out[:, r // 128, c // 4, (r % 32) * 16 + (r % 128) // 32 * 4 + c % 4] = flat[:, r, c]
    return out.reshape(lead + (rt, ct, 512))


def values(codes, byte):
    """float64 values of packed codes and row-major scale bytes."""
    q = np.stack([codes & 15, codes >> 4], -1).reshape(codes.shape[:-1] + (-1,)).astype(np.int64)
    v = np.where(q >= 8, -1.0, 1.0) * VALUES[q & 7]
    with np.errstate(invalid="ignore", over="ignore"):
        s = np.where(byte == 255, np.nan, np.ldexp(1.0, byte.astype(np.int64) - 127))
        return (v.reshape(v.shape[:-1] + (-1, 32)) * s[..., None]).reshape(v.shape)


def weights(w):
    """A weight stack [E, N, K] or matrix [N, K] -> (codes tensor, flat scale tiles tensor, float64 values tensor)."""
    c, b = quantize(w)
    return (torch.from_numpy(c), torch.from_numpy(tiles(b).reshape(-1)), torch.from_numpy(values(c, b)))
