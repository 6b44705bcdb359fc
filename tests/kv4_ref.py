"""The 4-bit cache, its attention, collected weights and eviction in 64 bits
on the host, from their definitions (test infrastructure)."""
import math

import numpy as np
import torch


def bf16(x):
    return x.to(torch.bfloat16).to(torch.float64)


def quantise(x):
    """(codes, s, m) of bf16 rows [..., D] (float64 tensors holding bf16)."""
    lo, hi = x.amin(-1), x.amax(-1)
    s = bf16((hi - lo) / 15)
    m = bf16(lo + 8 * s)
    bad = ~torch.isfinite(x).all(-1)
    s, m = torch.where(bad, math.nan, s), torch.where(bad, math.nan, m)
    step = torch.where(s > 0, s, 1.0)
    code = torch.where((s > 0)[..., None], torch.round((x - m[..., None]) / step[..., None]) + 8, 8.0)
    return torch.nan_to_num(code, nan=8.0).clamp(0, 15), s, m


def values(x):
    c, s, m = quantise(x)
    return s[..., None] * (c - 8) + m[..., None]


def parse_record(block, D):
    """codes [32][D] and (s, m) [32][2] of K and V from a record's bytes."""
    out = []
    b = block.astype(np.uint8)
    for part in (b[:16 * D + 128], b[16 * D + 128:]):
        by = part[:16 * D].reshape(32, D // 2)
        if len(out) == 2 and D == 128:
            by = np.stack([np.roll(r, 32) if t & 2 else r for t, r in enumerate(by)])
        codes = np.stack([by & 15, by >> 4], -1).reshape(32, D)
        sm = part[16 * D:].view(np.uint16).astype(np.uint32) << 16
        out += [codes, sm.view(np.float32).reshape(32, 2)]
    return out


def scores(q, k, q_pos, k_pos, scale, cap=0.0, slope=0.0, window=0, start=None):
    """([rows][keys] scores, -inf where hidden; bound on the size of the dot
    product's terms) of one query head."""
    z = q @ k.T * scale
    size = (q.abs() @ k.abs().T * scale).max().item() if k.shape[0] and q.shape[0] else 0.0
    if cap:
        z = cap * torch.tanh(z / cap)
    far = (q_pos[:, None] - k_pos[None]).double()
    z = z - slope * far
    if window:
        z = z.masked_fill(far >= window, -math.inf)
    if start is not None:
        z = z.masked_fill((k_pos < start)[None].expand_as(z), -math.inf)
    return z, size


def softmax(z):
    top = z.amax(-1, keepdim=True) if z.shape[-1] else torch.full((z.shape[0], 1), -math.inf, dtype=z.dtype)
    top = torch.where(top == -math.inf, 0.0, top)
    p = torch.exp(z - top)
    l = p.sum(-1, keepdim=True)
    lse = torch.where(l > 0, top + torch.log(l), -math.inf)[:, 0]
    return torch.where(l > 0, p / l, 0.0), lse


def keep(weight, budget, recent, sinks):
    n = len(weight)
    if n <= budget:
        return list(range(n))
    w = [-math.inf if math.isnan(x) else x for x in weight]
    safe = set(range(sinks)) | set(range(n - recent, n))
    rest = sorted((i for i in range(n) if i not in safe), key=lambda i: (-w[i], i))
    return sorted(safe | set(rest[:budget - sinks - recent]))
