"""The norms and the 8-bit format in 64 bits, written out from their definitions, and how far a kernel that works in
fp32 may be from them.

Error model, with u = 2^-24 (half a step of fp32):
  - a sum over a row: a thread adds 64 terms or fewer in sequence, then 5 steps of a butterfly and 16 warps or fewer:
    at most K u sum|terms| with K = 90 roundings, one more for each rounding inside a term;
  - the mean: the first estimate m1 is within K u mean|h|, and the sum of the differences from it corrects it to
    (K + 3) u mean|d| and its own rounding u |mean|;
  - rstd: its square's relative error is that of the sum of squares, K + 4, halved by the root, and 4 more u;
  - results are rounded once to their type: half a step, finfo.eps / 2.
"""
from __future__ import annotations

import math

import torch

U = 2.0 ** -24
K = 90.0
F64 = torch.float64
QMAX = {"int8": 127.0, "e4m3": 448.0}


def half_step(dtype) -> float:
    return torch.finfo(dtype).eps / 2


def forward64(x, weight, bias, kind, eps, residual=None, mask=None):
    """(y, h, mean, rstd, bound of y before its rounding, bound of mean, bound of rstd) of CPU tensors; masked rows are 0."""
    h = x if residual is None else (x.float() + residual.float()).to(x.dtype)
    v = h.to(F64)
    if mask is not None:
        v = torch.where((mask != 0)[:, None], v, torch.zeros((), dtype=F64))
        h = torch.where((mask != 0)[:, None], h, torch.zeros((), dtype=h.dtype))
    C = v.shape[1]
    mean = v.sum(1) / C if kind == "layer" else torch.zeros(len(v), dtype=F64)
    d = v - mean[:, None]
    rstd = (d.square().sum(1) / C + eps) ** -0.5
    w = torch.ones(C, dtype=F64) if weight is None else weight.to(F64)
    b = torch.zeros(C, dtype=F64) if bias is None else bias.to(F64)
    xh = d * rstd[:, None]
    y = xh * w + b
    spread = d.abs().mean(1)
    e_mean = U * mean.abs() + (K + 3) * U * spread
    e_rstd = (K / 2 + 8) * U * rstd
    e_d = (4 * U * d.abs() + ((K + 3) * U * spread)[:, None]) if kind == "layer" else torch.zeros_like(d)
    e_y = e_d * rstd[:, None] * w.abs() + (K / 2 + 12) * U * (xh * w).abs() + 2 * U * b.abs()
    if mask is not None:
        on = (mask != 0).to(F64)
        y, mean, rstd, e_y = y * on[:, None], mean * on, rstd * on, e_y * on[:, None]
    return y, h, mean, rstd, e_y, e_mean, e_rstd


def backward64(h, dy, weight, mean, rstd, kind, dsummed=None, mask=None):
    """(dx, dweight, dbias, bounds of the three before dx is rounded) with the statistics as the kernel gets them. h: what
    the norm's input is taken to be, in 64 bits."""
    on = torch.ones(len(h), dtype=torch.bool) if mask is None else mask != 0
    zero = torch.zeros((), dtype=F64)
    h, g = torch.where(on[:, None], h.to(F64), zero), torch.where(on[:, None], dy.to(F64), zero)
    R, C = h.shape
    m = mean.to(F64)[:, None] if kind == "layer" else torch.zeros((R, 1), dtype=F64)
    m = torch.where(on[:, None], m, zero)
    s = torch.where(on, rstd.to(F64), zero)[:, None]
    w = torch.ones(C, dtype=F64) if weight is None else weight.to(F64)
    d = h - m
    r = g * s
    u = r * w
    c1 = u.mean(1, keepdim=True) if kind == "layer" else torch.zeros((R, 1), dtype=F64)
    c2 = (u * d).mean(1, keepdim=True) * s * s
    dx = u - c1 - d * c2
    if dsummed is not None:
        dx = dx + torch.where(on[:, None], dsummed.to(F64), zero)
    e = (7 * U * u.abs() + (K + 8) * U * u.abs().mean(1, keepdim=True) * (kind == "layer")
         + d.abs() * s * s * (K + 15) * U * (u * d).abs().mean(1, keepdim=True) + 4 * U * (c1.abs() + (d * c2).abs()) + 2 * U * dx.abs())
    # a thread's rows in sequence (152 blocks at least share them, or each row has its own), the block's, and an eighth
    # of 2432 blocks' or fewer
    k_rows = R / 152 + 400
    return (dx, (r * d).sum(0), g.sum(0), e, (k_rows + 4) * U * (r * d).abs().sum(0) + 1e-44, k_rows * U * g.abs().sum(0) + 1e-44)


def assert_within(name, got, want, bound, dtype=None):
    got = got.detach().cpu().to(F64)
    limit = bound if dtype is None else bound + half_step(dtype) * (want.abs() + bound) + torch.finfo(dtype).smallest_normal * 2.0 ** -7
    err = (got - want).abs()
    bad = ~(err <= limit)
    assert not bad.any(), f"{name}: {int(bad.sum())} of {bad.numel()} off, worst {float((err / limit).max()):.3g} times the bound"


# ---------------------------------------------------------------------------- the 8-bit format

def e4m3_values():
    """The value of each code 0 .. 126 (127 is NaN)."""
    out = []
    for c in range(127):
        e, m = c >> 3, c & 7
        out.append(math.ldexp(m, -9) if e == 0 else math.ldexp(8 + m, e - 10))
    return torch.tensor(out, dtype=F64)


def pack64(x, fmt):
    """(codes, scales) as torch.uint8, block by block from the definition."""
    R, C = x.shape
    v = x.to(F64)
    codes = torch.zeros((R, C), dtype=torch.uint8)
    scales = torch.zeros((R, (C + 31) // 32), dtype=torch.uint8)
    table = e4m3_values()
    for j in range(scales.shape[1]):
        b = v[:, 32 * j:32 * j + 32]
        for i in range(R):
            if not torch.isfinite(b[i]).all():
                scales[i, j] = 255
                continue
            top = float(b[i].abs().max())
            e = -126
            if top > 0:
                e = max(e, math.frexp(top / QMAX[fmt])[1] - 1)
                while QMAX[fmt] * 2.0 ** e < top:
                    e += 1
                while e > -126 and QMAX[fmt] * 2.0 ** (e - 1) >= top:
                    e -= 1
            scales[i, j] = e + 127
            q = b[i] * 2.0 ** -e
            if fmt == "int8":
                codes[i, 32 * j:32 * j + 32] = torch.round(q).to(torch.int64).to(torch.int8).view(torch.uint8)
            else:
                near = (q.abs()[:, None] - table[None, :]).abs()
                best = near.min(1, keepdim=True).values
                # the nearest code; of two as near, the even one
                order = torch.where(near == best, torch.arange(127)[None, :] % 2, torch.full((1, 127), 9))
                c = order.argmin(1)
                codes[i, 32 * j:32 * j + 32] = (c + 128 * torch.signbit(q).long()).to(torch.uint8)
    return codes, scales


def values64(codes, scales, fmt, dtype):
    """What codes and scales stand for when they are read as `dtype`, in 64 bits. (Exact in fp32; the smallest e4m3 codes
    of the smallest scale, 2^-9 2^-126, are below bf16's smallest number, 2^-133, and rounded to it.)"""
    C = codes.shape[1]
    if fmt == "int8":
        q = codes.view(torch.int8).to(F64)
    else:
        q = torch.cat([e4m3_values(), torch.tensor([math.nan], dtype=F64)])[(codes & 127).long()]
        q = torch.where(codes >= 128, -q, q)
    s = torch.where(scales == 255, torch.tensor(math.nan, dtype=F64), 2.0 ** (scales.to(F64) - 127))
    v = q * s.repeat_interleave(32, 1)[:, :C]
    most = torch.finfo(dtype).max
    return torch.where(v.isnan(), v, v.clamp(-most, most)).float().to(dtype).to(F64)


def same(a, b) -> bool:
    """Equal values, NaN where the other has it; a short answer for long tensors."""
    a, b = a.detach().cpu(), b.detach().cpu()
    if a.shape != b.shape:
        return False
    if a.is_floating_point():
        a, b = a.to(F64), b.to(F64)
        return bool(((a == b) | (a.isnan() & b.isnan())).all())
    return bool((a == b).all())


# ---------------------------------------------------------------------------- tensors

def matrix(g, rows, cols, dtype, layout, scale=1.0, shift=0.0):
    """A CPU tensor of normal values and a function that lays one like it out on the GPU: "tight" rows, "pad"ded ones on
    32-byte boundaries, on 16-byte ones ("pad16"), or rows that start at an odd "offset" of a wider matrix."""
    t = (torch.randn((rows, cols), generator=g) * scale + shift).to(dtype)
    return t, lambda v=t: on_gpu(v, layout)


def on_gpu(t, layout):
    rows, cols = t.shape
    es = t.element_size()
    if layout == "tight":
        return t.cuda()
    per = 32 // es
    if layout in ("pad", "pad16"):
        ld = (cols + per - 1) // per * per + (per // 2 if layout == "pad16" else 0)
        buf = torch.full((rows, ld), math.nan, dtype=t.dtype, device="cuda")
        buf[:, :cols] = t.cuda()
        return buf[:, :cols]
    buf = torch.full((rows, cols + 5), math.nan, dtype=t.dtype, device="cuda")
    buf[:, 3:3 + cols] = t.cuda()
    return buf[:, 3:3 + cols]
