"""Plain 64-bit forms of the 8-bit cache's operators (test infrastructure only),
written token by token and row by row from the definitions in
include/dcp_mla_cache8.h, on whatever device the inputs are."""
from __future__ import annotations

import math

import torch

E4M3_MAX = 448.0


def place(pos: int, cp: int, interleave: int):
    """(shard, local index) of a position."""
    return (pos // interleave) % cp, pos // (interleave * cp) * interleave + pos % interleave


def rotate(x, positions, inv_freq, start, interleaved, mscale=1.0):
    """x [N, H, D] float64 with dims [start, start + 2 len(inv_freq)) rotated."""
    out = x.clone()
    half = inv_freq.shape[0]
    for i in range(half):
        ang = positions.double() * inv_freq[i].double()
        c, s = torch.cos(ang)[:, None] * mscale, torch.sin(ang)[:, None] * mscale
        a, b = (start + 2 * i, start + 2 * i + 1) if interleaved else (start + i, start + i + half)
        out[..., a] = x[..., a] * c - x[..., b] * s
        out[..., b] = x[..., b] * c + x[..., a] * s
    return out


def scale_for(peak: float) -> float:
    """The smallest power of two s with peak <= 448 s, at least 2^-60."""
    k = -60
    while peak > E4M3_MAX * 2.0 ** k:
        k += 1
    return 2.0 ** k


def to_e4m3(x):
    """float64 -> the nearest e4m3 value (ties to even), as float64; NaN for what is not finite. |x| <= 448 (1 + 2^-5)."""
    a = x.abs()
    _, e = torch.frexp(a)
    step = torch.exp2((e - 1).clamp(min=-6).double() - 3)  # 3 mantissa bits; subnormals below 2^-6
    y = torch.round(x / step) * step  # torch.round: ties to even
    return torch.where(torch.isfinite(x), y, torch.full_like(x, math.nan))


def append(x, counts, starts, values, scales, cp, interleave, block, held=None):
    """Append packed tokens x [N, Dk] (float64, keys rotated already). values: list
    of cp float64 [B, T, Dk] code values, scales: list of cp float64 [B, blocks];
    both changed in place. Shards not in ``held`` are skipped."""
    T = values[0].shape[1]
    n = 0
    for b, (count, start) in enumerate(zip(counts, starts)):
        by_block: dict = {}
        for i in range(count):
            j, t = place(start + i, cp, interleave)
            if t < T and (held is None or j in held):
                by_block.setdefault((j, t // block), []).append((t, n + i))
        for (j, blk), tokens in by_block.items():
            new = x[[k for _, k in tokens]]
            fin = new[torch.isfinite(new)]
            s = scale_for(float(fin.abs().max()) if fin.numel() else 0.0)
            first = min(t for t, _ in tokens)
            old = range(blk * block, first)
            if len(old):
                was = float(scales[j][b, blk])
                if was > s:
                    s = was
                elif s > was:
                    sl = slice(old[0], old[-1] + 1)
                    values[j][b, sl] = to_e4m3(values[j][b, sl] * (was / s))
            scales[j][b, blk] = s
            for t, k in tokens:
                values[j][b, t] = to_e4m3(x[k] / s)
        n += count


def gather(values, scales, b, positions, cp, interleave, block, held=None):
    """(float64 [n, Dk] cached values, mask of those that are held and exist)."""
    T = values[0].shape[1]
    rows, ok = [], []
    for pos in positions:
        j, t = place(pos, cp, interleave)
        here = t < T and (held is None or j in held)
        ok.append(here)
        rows.append(values[j][b, t] * scales[j][b, t // block] if here else torch.zeros_like(values[0][0, 0]))
    return torch.stack(rows), ok


def visible(length: int, window: int, sinks: int):
    return [p for p in range(length) if window == 0 or p >= length - window or p < sinks]


def attend(q, k, scale, dv=512):
    """q [H, Dk], k [n, Dk] float64 -> (out [H, dv], natural-log LSE [H])."""
    if k.shape[0] == 0:
        return torch.zeros((q.shape[0], dv), dtype=torch.float64, device=q.device), \
            torch.full((q.shape[0],), -math.inf, dtype=torch.float64, device=q.device)
    s = scale * (q @ k.T)
    m = s.max(1, keepdim=True).values
    p = torch.exp(s - m)
    total = p.sum(1, keepdim=True)
    return p @ k[:, :dv] / total, (m + torch.log(total))[:, 0]
