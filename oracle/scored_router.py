"""Plain 64-bit reference of the scored router (moelb_route and
moelb_route_backward), one token after another for the picks, on any device."""
from __future__ import annotations

import math

import torch

EPS = 1e-20
F32_MAX = torch.finfo(torch.float32).max


def scores(z: torch.Tensor, score: str):
    """(s, on): scores in float64, 0 for masked experts; on: neither -inf nor NaN."""
    on = z > -math.inf
    x = torch.where(on, z.double().clamp(max=F32_MAX), torch.zeros((), dtype=torch.float64, device=z.device))
    if score == "sigmoid":
        return torch.where(on, torch.sigmoid(x), torch.zeros_like(x)), on
    m = torch.where(on, x, torch.full_like(x, -math.inf)).amax(1, keepdim=True)
    m = torch.where(m > -math.inf, m, torch.zeros_like(m))
    e = torch.where(on, torch.exp(x - m), torch.zeros_like(x))
    total = e.sum(1, keepdim=True)
    return torch.where(total > 0, e / total, torch.zeros_like(e)), on


def route(z, k, score="softmax", bias=None, groups=1, topk_groups=1, group_top=1, renorm=False, scale=1.0):
    """(idx [T, k], wts [T, k], gap [T]) of logits z [T, E]."""
    T, E = z.shape
    s, on = scores(z, score)
    c = s if bias is None else s + bias.double()
    c = torch.where(on & (c > -math.inf), c.clamp(max=F32_MAX), torch.full_like(s, -math.inf))
    key = c if bias is not None else torch.where(on, z.double().clamp(max=F32_MAX), torch.full_like(s, -math.inf))
    c, key, s = c.cpu().tolist(), key.cpu().tolist(), s.cpu().tolist()
    size = E // groups
    idx = torch.full((T, k), -1, dtype=torch.int32)
    wts = torch.zeros((T, k), dtype=torch.float64)
    gap = torch.full((T,), math.inf, dtype=torch.float64)
    for t in range(T):
        may = range(E)
        if groups > 1:
            mark = []
            for g in range(groups):
                top = sorted(c[t][g * size:(g + 1) * size], reverse=True)[:group_top]
                mark.append(-math.inf if -math.inf in top else sum(top))
            best = sorted(range(groups), key=lambda g: (-mark[g], g))[:topk_groups]
            may = [e for g in sorted(best) for e in range(g * size, (g + 1) * size)]
        order = [e for e in sorted(may, key=lambda e: (-key[t][e], e)) if key[t][e] > -math.inf]
        picks = order[:k]
        total = sum(s[t][e] for e in picks) + EPS
        for j, e in enumerate(picks):
            idx[t, j] = e
            wts[t, j] = scale * s[t][e] / (total if renorm else 1.0)
        if len(order) > k:
            gap[t] = c[t][order[k - 1]] - c[t][order[k]]
    return idx, wts, gap


def route_dz(z, idx, dwts, score="softmax", renorm=False, scale=1.0):
    """(dz, mag): the gradient of sum dwts * wts with respect to z in float64, and the sum of its terms' magnitudes."""
    s, on = scores(z, score)
    ok = (idx >= 0) & (idx < z.shape[1])
    e = idx.long().clamp(0, z.shape[1] - 1)
    sj = s.gather(1, e) * ok
    q = dwts.double() * ok
    S = sj.sum(1, keepdim=True) + EPS
    A, Aa = (q * sj).sum(1, keepdim=True), (q.abs() * sj).sum(1, keepdim=True)
    ds, dm = (scale * (q - A / S) / S, abs(scale) * (q.abs() + Aa / S) / S) if renorm else (scale * q, abs(scale * q))
    ds, dm = ds * ok, dm * ok
    full = torch.zeros_like(s).scatter_add_(1, e, ds)
    mag = torch.zeros_like(s).scatter_add_(1, e, dm)
    if score == "sigmoid":
        x = torch.where(on, z.double(), torch.zeros_like(s))
        slope = torch.sigmoid(x) * torch.sigmoid(-x) * on
        return full * slope, mag * slope
    C = scale * (A / S) * (EPS / S) if renorm else (s * full).sum(1, keepdim=True)
    Cm = C.abs() if renorm else (s * mag).sum(1, keepdim=True)
    return s * (full - C), s * (mag + Cm)
