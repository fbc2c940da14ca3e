"""Rotary positions from their definition in 64 bits (torch float64, any device)."""
import math

import torch


def cos_sin(positions, turns, magnitude):
    """[..., rot/2] in float64; Python's whole numbers give each turn exactly."""
    flat, t = positions.flatten().tolist(), turns.tolist()
    frac = [[(p * x) % (1 << 64) for x in t] for p in flat]
    angle = torch.tensor([[f / 2.0 ** 64 for f in row] for row in frac], dtype=torch.float64).view(*positions.shape, len(t))
    angle = angle.to(turns.device) * (2 * math.pi)
    return torch.cos(angle) * magnitude, torch.sin(angle) * magnitude


def pairs(rot, interleaved):
    i = torch.arange(rot // 2)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)


def rotate(x, positions, rope, backward=False):
    """x [T, H, d] with positions [T]: the turned values in float64, and m (|a| + |b|) of each element's pair."""
    c, s = (t.unsqueeze(1) for t in cos_sin(positions, rope.turns, rope.magnitude))
    if backward:
        s = -s
    rot = 2 * rope.turns.numel()
    i, j = (t.to(x.device) for t in pairs(rot, rope.interleaved))
    y, size = x.double().clone(), torch.zeros(x.shape, dtype=torch.float64, device=x.device)
    a, b = x[..., i].double(), x[..., j].double()
    y[..., i], y[..., j] = a * c - b * s, a * s + b * c
    size[..., i] = size[..., j] = (a.abs() + b.abs()) * rope.magnitude
    return y, size


def bf16(x):
    """float64 rounded to the nearest bf16 (ties to even) at once."""
    f = x.float()
    rest = x - f.double()
    bits = f.view(torch.int32)
    tie = ((bits & 0xFFFF) == 0x8000) & (rest != 0)
    return torch.where(tie, torch.where((rest > 0) == (f > 0), bits + 1, bits - 1), bits).view(torch.float32).bfloat16()
