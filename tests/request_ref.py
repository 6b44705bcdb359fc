"""Rotary positions, attention over packed prompts and sampled tokens in 64
bits, from their definitions (test infrastructure)."""
import decimal
import math

import numpy as np
import torch

BF16 = 2.0 ** -8  # a rounding to bf16, relative to the value


def frequencies(rot, base, kind="plain", factor=1.0, original=1.0, low=1.0, high=2.0):
    """[rot / 2] angles a position, by plain loops."""
    out = []
    if kind == "ramp":
        lo, hi = (rot / 2 * math.log(original / (2 * math.pi * t), base) for t in (high, low))
        lo, hi = max(math.floor(lo), 0), min(math.ceil(hi), rot - 1)
    for i in range(rot // 2):
        f = base ** (-2 * i / rot)
        if kind == "linear":
            f = f / factor
        if kind == "bands":
            t = original * f / (2 * math.pi)
            if t < low:
                f = f / factor
            elif t <= high:
                s = (t - low) / (high - low)
                f = s * f + (1 - s) * f / factor
        if kind == "ramp":
            s = min(max((i - lo) / (hi - lo if hi > lo else 0.001), 0.0), 1.0)
            f = f * (1 - s) + f / factor * s
        out.append(f)
    return np.array(out)


def exact_turns(rot, base, kind="plain", factor=1, original=1, low=1, high=2):
    """[rot / 2] turns a position to 50 digits: the formulas of `frequencies` over 2 pi."""
    with decimal.localcontext(decimal.Context(prec=60)):
        D = decimal.Decimal
        pi = D("3.14159265358979323846264338327950288419716939937510582097494459")
        log, factor, original, low, high = D(base).ln(), D(factor), D(original), D(low), D(high)
        if kind == "ramp":
            lo, hi = (rot * (original / (2 * pi * t)).ln() / (2 * log) for t in (high, low))
            lo, hi = max(math.floor(lo), 0), min(math.ceil(hi), rot - 1)
        out = []
        for i in range(rot // 2):
            f, part = (log * -2 * i / rot).exp(), D(1)
            if kind == "linear":
                part = D(0)
            if kind == "bands":
                part = min(max((original * f / (2 * pi) - low) / (high - low), D(0)), D(1))
            if kind == "ramp":
                part = 1 - min(max(D(i - lo) / max(D(hi - lo), D("0.001")), D(0)), D(1))
            out.append((part * f + (1 - part) * f / factor) / (2 * pi))
        return out


def rotate(x, pos, freq, amplitude=1.0, interleaved=False):
    """x float64 [rows][heads][dim]; (turned rows, bound on the fp32 steps' error)."""
    rot = 2 * len(freq)
    angle = pos.double()[:, None] * torch.from_numpy(freq)
    c, s = (amplitude * torch.cos(angle))[:, None], (amplitude * torch.sin(angle))[:, None]
    a, b = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2), slice(rot // 2, rot))
    y, slack = x.clone(), torch.zeros_like(x)
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., a] * s + x[..., b] * c
    # sine and cosine: 2^-24 of half a turn (pi) and 2^-23 of themselves twice; products 2^-23
    size = (x[..., a].abs() + x[..., b].abs()) * amplitude * 2.0 ** -20
    slack[..., a], slack[..., b] = size, size
    return y, slack


def attend(q, k, v, cu_q, cu_k, scale=None, cap=0.0, slopes=None, window=0):
    """float64 q [rows][hq][d], k and v [keys][hkv][d] (bf16 values).  Returns
    out, lse and bounds on their errors: scores in fp32, weights and outputs in bf16."""
    n, hq, d = q.shape
    G = hq // k.shape[1]
    scale = scale or 1.0 / math.sqrt(d)
    out, lse = torch.zeros_like(q), torch.full((n, hq), -math.inf, dtype=torch.float64)
    tol, tol_lse = torch.zeros_like(q), torch.zeros(n, hq, dtype=torch.float64)
    for r in range(len(cu_q) - 1):
        a, b, x, y = int(cu_q[r]), int(cu_q[r + 1]), int(cu_k[r]), int(cu_k[r + 1])
        m, keys = b - a, y - x
        for i in range(m):
            p = keys - m + i
            first = max(0, p - window + 1) if window else 0
            if p < 0:
                continue
            K, V = k[x + first:x + p + 1], v[x + first:x + p + 1]
            K, V = K.repeat_interleave(G, 1), V.repeat_interleave(G, 1)
            z = torch.einsum("hd,khd->hk", q[a + i], K) * scale
            # fp32 sums of d products, the scale, the cap and the base of the exponential
            size = (torch.einsum("hd,khd->hk", q[a + i].abs(), K.abs()) * scale).amax(1)
            err = size * 2.0 ** -24 * (d / 4 + 8) + 2.0 ** -22
            if cap:
                z = cap * torch.tanh(z / cap)
                err = err + cap * 2.0 ** -21
            if slopes is not None:
                far = (torch.arange(first, p + 1) - p).double()
                z = z + slopes.double()[:, None] * far
                err = err + (slopes.double().abs() * far.abs().max()) * 2.0 ** -22
            err = err + z.abs().amax(1) * 2.0 ** -22
            w = torch.softmax(z, 1)
            out[a + i] = torch.einsum("hk,khd->hd", w, V)
            lse[a + i] = torch.logsumexp(z, 1)
            mass = torch.einsum("hk,khd->hd", w, V.abs())
            # a weight's rounding and its exponential's (2^-22), twice in a quotient
            tol[a + i] = mass * (BF16 + 4 * err[:, None] + 2.0 ** -18) + BF16 * out[a + i].abs() + 2.0 ** -130
            tol_lse[a + i] = 2 * err + 2.0 ** -20 * (1 + lse[a + i].abs())
    return out, lse, tol, tol_lse


def sample_row(logits, u, t, k=0, top_p=1.0, min_p=0.0):
    """(token, logprob, kept) of one row of float64 logits, token by token."""
    x = [(-l, i) for i, l in enumerate(logits.tolist()) if not math.isnan(l) and l != -math.inf]
    if not x:
        return -1, -math.inf, 0
    x.sort()
    most = -x[0][0]
    if t <= 0:
        return x[0][1], 0.0, 1
    if most == math.inf:
        w = np.array([1.0 if l == -math.inf else 0.0 for l, _ in x])
    else:
        w = np.exp((np.array([-l for l, _ in x]) - most) / t)
    n = len(x)
    if k > 0:
        n = min(n, k)
    n = min(n, int((w >= min_p).sum())) if min_p > 0 else n
    total = math.fsum(w[:n])
    if top_p < 1:
        run = np.cumsum(w[:n])
        n = min(n, int((run < top_p * total).sum()) + 1)
        total = math.fsum(w[:n])
    run = np.cumsum(w[:n])
    at = min(int((run <= u * total).sum()), n - 1)
    return x[at][1], math.log(w[at] / total), n
