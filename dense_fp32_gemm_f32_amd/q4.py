"""Weights in 4 bits, as ``gemm_f32_q4`` takes them: made once from an fp32 matrix
when a model is loaded, with torch operations on whatever device it is on."""
from __future__ import annotations

import torch

from dense_fp32_gemm_f32_amd.binding import Q4_E2M1, Q4_INT

# What an e2m1 code stands for; bit 3 is the sign.
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)


def pack(codes):
    """Codes 0 .. 15 (..., K) as bytes (..., (K + 1) // 2), the even k in the low half."""
    codes = codes.to(torch.uint8)
    if codes.shape[-1] % 2:
        codes = torch.cat((codes, torch.zeros_like(codes[..., :1])), dim=-1)
    return (codes[..., 0::2] | (codes[..., 1::2] << 4)).contiguous()


def unpack(packed, K):
    """The K codes of each row of bytes."""
    return torch.stack((packed & 15, packed >> 4), dim=-1).flatten(-2)[..., :K]


def scale_values(scale):
    """Scales as fp32; bytes are e8m0, the power of two 2^(e - 127) with 255 NaN."""
    if scale.dtype in (torch.uint8, torch.float8_e8m0fnu):
        e = scale.view(torch.uint8).to(torch.float64)
        return torch.where(e == 255, torch.full_like(e, float("nan")),
                           torch.exp2(e - 127)).to(torch.float32)
    return scale.to(torch.float32)


def dequantize(codes, scale, K, *, zero=None, group=128, format=Q4_INT, dtype=torch.float32):
    """The weights (..., N, K) that codes, scales and zero points stand for."""
    c = unpack(codes, K)
    at = torch.arange(K, device=codes.device) // group
    if format == Q4_E2M1:
        w = torch.tensor(E2M1, dtype=dtype, device=codes.device)[c.long()]
    else:
        w = c.to(dtype) - (8 if zero is None else zero.to(dtype)[..., at])
    return w * scale_values(scale).to(dtype)[..., at]


def quantize(W, *, group=128, format=Q4_INT, symmetric=True, scale_dtype=torch.float32):
    """(codes, scale, zero) of weights (..., N, K): each group of ``group`` columns
    has the scale that its largest weight needs, and zero points too (Q4_INT with
    ``symmetric`` false; None otherwise).  ``scale_dtype`` float32, float16,
    bfloat16, or uint8 for e8m0 (then the next power of two above)."""
    K = W.shape[-1]
    along = (K + group - 1) // group
    w = torch.nn.functional.pad(W.float(), (0, along * group - K)).unflatten(-1, (along, group))
    # (padding is zeros: it is inside every range that holds zero)
    low, high = w.amin(-1), w.amax(-1)
    zero = None
    if format == Q4_E2M1:
        size = torch.maximum(-low, high) / 6
    elif symmetric:
        size = torch.maximum(-low / 8, high / 7)
    else:
        low, high = low.clamp_max(0), high.clamp_min(0)
        size = (high - low) / 15
    size = torch.where(size > 0, size, torch.ones_like(size))
    if scale_dtype == torch.uint8:
        scale = (torch.ceil(torch.log2(size)) + 127).clamp(0, 254).to(torch.uint8)
    else:
        scale = size.clamp_max(torch.finfo(scale_dtype).max).to(scale_dtype)
    by = scale_values(scale).unsqueeze(-1)
    by = torch.where(by > 0, by, torch.ones_like(by))   # too small for the type: zeros
    if format == Q4_E2M1:
        steps = torch.tensor(E2M1[:8], device=W.device)
        x = (w / by).abs()
        code = torch.bucketize(x, (steps[1:] + steps[:-1]) / 2)
        code = code + 8 * (w < 0)
    elif symmetric:
        code = torch.round(w / by).clamp(-8, 7) + 8
    else:
        zero = torch.round(-low.unsqueeze(-1) / by).clamp(0, 15)
        code = (torch.round(w / by) + zero).clamp(0, 15)
        zero = zero.squeeze(-1).to(torch.uint8)
    return pack(code.flatten(-2)[..., :K]), scale, zero
