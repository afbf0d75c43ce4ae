"""Float64 references of microscaled 4-bit floating point, straight from ``include/mx4.h``, on whatever device the
inputs are."""
import math

import torch

GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def encode(x):
    """Codes [..., K] (0 .. 15) and scale bytes [..., K / 32] of x [..., K], by distances to the grid."""
    b = x.double().reshape(*x.shape[:-1], -1, 32)
    top = b.abs().amax(dim=-1)
    bad = ~torch.isfinite(top)
    safe = torch.where(bad | (top == 0), 1.0, top)
    e = torch.frexp(safe)[1] - 1 - 2
    e = torch.where(top == 0, -127, e.clamp(min=-127))
    v = (torch.where(bad[..., None], 0.0, b) / torch.exp2(e.double())[..., None]).abs()
    grid = torch.tensor(GRID, dtype=torch.float64, device=x.device)
    far = (v[..., None] - grid).abs()
    # the nearest, of two equally near ones the even code
    rank = far * 16 + torch.tensor([0, 1] * 4, dtype=torch.float64, device=x.device) * 1e-9
    code = torch.where(v >= 6, 7, rank.argmin(dim=-1))
    sign = torch.signbit(b).long() * 8
    return (code + sign).reshape(x.shape), torch.where(bad, 255, e + 127)


def decode(code, scale):
    """Values in float64; a block of scale 255 is NaN."""
    grid = torch.tensor(GRID, dtype=torch.float64, device=code.device)
    v = grid[code & 7] * torch.where(code >= 8, -1.0, 1.0)
    s = torch.where(scale == 255, math.nan, torch.exp2(scale.double() - 127))
    return (v.reshape(*s.shape, 32) * s[..., None]).reshape(v.shape)


def pack(code, scale):
    """The codes' and scales' tensors of [..., rows, K], with a value that no product may look at behind the rows."""
    rows, K = code.shape[-2:]
    planes, deep = -(-K // 256), (rows // 4 + 1) * 4
    wide = torch.full((*code.shape[:-2], deep, planes * 8), 255, dtype=torch.uint8, device=code.device)
    wide[..., :rows, :] = 0
    wide[..., :rows, : K // 32] = scale.to(torch.uint8)
    scales = wide.reshape(*code.shape[:-2], deep, planes, 8).transpose(-3, -2).contiguous()
    code = code.to(torch.uint8)
    return (code[..., ::2] | code[..., 1::2] << 4).contiguous(), scales


def unpack(codes, scales):
    """Codes [..., rows, K] and every scale byte of those rows [..., rows, planes * 8]."""
    codes = codes.long()
    code = torch.stack([codes & 15, codes >> 4], dim=-1).flatten(-2)
    s = scales.transpose(-3, -2).flatten(-2)[..., : code.shape[-2], :]
    return code, s.long()


def transposed(x):
    """x^T with zeros behind its rows, up to whole blocks."""
    pad = -x.shape[-2] % 32
    return torch.nn.functional.pad(x, (0, 0, 0, pad)).transpose(-1, -2).contiguous()


def rounded(x):
    return decode(*encode(x))
