"""Plain 64-bit forms of the e4m3 operators, shared by their tests.

e4m3 keeps 4 significant bits: rounding a value v is off by at most 2^-4 of
|v| (half a step of 2^-3 relative to the power of two below it), and by at most
2^-10 below the smallest normal value 2^-6.
"""
from __future__ import annotations

import torch

BLOCK = 128
E4M3 = torch.float8_e4m3fn


def blocks(n: int) -> int:
    return -(-n // BLOCK)


def spread(scale, rows, cols, block_rows):
    """Block scales [..., br, bc] as one value per element [..., rows, cols]."""
    s = scale.repeat_interleave(block_rows, -2)[..., :rows, :]
    return s.repeat_interleave(BLOCK, -1)[..., :cols]


def e4m3_round(v):
    """v (float64) to the nearest e4m3 value: ties to even, saturated at 448."""
    _, e = torch.frexp(v)
    step = torch.exp2((e - 1).clamp_min(-6).double() - 3.0)
    return (torch.round(v / step) * step).clamp(-448.0, 448.0)


def block_scales(x, block_rows):
    """max(amax / 448, 2^-126) of each block of x [..., rows, cols] (float64)."""
    rows, cols = x.shape[-2:]
    br, bc = -(-rows // block_rows), blocks(cols)
    pad = torch.zeros(*x.shape[:-2], br * block_rows, bc * BLOCK, dtype=torch.float64, device=x.device)
    pad[..., :rows, :cols] = x.abs()
    pad = pad.view(*x.shape[:-2], br, block_rows, bc, BLOCK)
    return (pad.amax(dim=(-3, -1)) / 448.0).clamp_min(2.0 ** -126)


def quantize(x, block_rows):
    """(codes as float8_e4m3fn, fp32 scales) of x [..., rows, cols]."""
    rows, cols = x.shape[-2:]
    s = block_scales(x.double(), block_rows).float()
    return e4m3_round(x.double() / spread(s.double(), rows, cols, block_rows)).float().to(E4M3), s


def values(q, scale, block_rows):
    """The float64 values that codes with block scales stand for."""
    return q.double() * spread(scale.double(), q.shape[-2], q.shape[-1], block_rows)


def check_quantized(q, scale, x, block_rows, rel=1e-6):
    """Codes and scales of x (float64): the scales within `rel` (fp32 roundings),
    and each code within half an e4m3 step of x / scale, widened by the same."""
    rows, cols = x.shape[-2:]
    want = block_scales(x, block_rows)
    assert torch.all((scale.double() - want).abs() <= rel * want)
    v = x / spread(scale.double(), rows, cols, block_rows)
    got = q.double()
    assert torch.all(torch.isfinite(got))
    half = torch.maximum(v.abs() * 2.0 ** -4, torch.full_like(v, 2.0 ** -10))
    assert torch.all((got - v).abs() <= half * (1 + 16 * rel))
    # and it is the nearest code, unless v lies within rel of the middle between two codes
    best = e4m3_round(v)
    off = got != best
    assert torch.all(((got - v).abs() - (best - v).abs())[off] <= 2 * rel * v.abs()[off])


def product(a, b, sizes):
    """Groups of `sizes` rows of a times b[g]^T; and the same of the absolute values
    (what a sum's rounding errors are measured against)."""
    out = torch.zeros(a.shape[0], b.shape[1], dtype=torch.float64, device=a.device)
    mag = torch.zeros_like(out)
    at = 0
    for g, m in enumerate(sizes):
        if m:
            out[at:at + m] = a[at:at + m] @ b[g].T
            mag[at:at + m] = a[at:at + m].abs() @ b[g].abs().T
        at += m
    return out, mag
