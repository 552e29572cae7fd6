"""Plain 64-bit reference of MX 4-bit floating point (moelb_mx_quantize,
moelb_mx_dequantize, moelb_mx_grouped_ffn), on any device."""
from __future__ import annotations

import math

import torch

GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def scale_bytes(K: int) -> int:
    return (K // 32 + 15) // 16 * 16


def quantize(x: torch.Tensor):
    """(q, scales) of x [..., K], as moelb_mx_quantize lays them out."""
    K = x.shape[-1]
    b = x.double().reshape(*x.shape[:-1], K // 32, 32)
    bad = ~torch.isfinite(b).all(-1)
    a = torch.where(bad[..., None], torch.zeros_like(b), b)
    amax = a.abs().amax(-1)
    exp = torch.frexp(amax).exponent - 1 - 2  # float64: fp32's subnormals are normal here
    exp = torch.where(amax > 0, exp, torch.full_like(exp, -127)).clamp(-127, 127)
    v = a * torch.exp2(-exp.double())[..., None]
    grid = torch.tensor(GRID, dtype=torch.float64, device=x.device)
    dist = (v.abs()[..., None] - grid).abs()
    # nearest; of two equally near codes the even one (a penalty below every difference of two distances)
    dist = dist + 1e-12 * (torch.arange(8, device=x.device) % 2)
    code = dist.argmin(-1) + 8 * torch.signbit(b)
    code = torch.where(bad[..., None], torch.zeros_like(code), code).reshape(x.shape).to(torch.uint8)
    q = code[..., 0::2] | (code[..., 1::2] << 4)
    scales = torch.zeros((*x.shape[:-1], scale_bytes(K)), dtype=torch.uint8, device=x.device)
    scales[..., :K // 32] = torch.where(bad, torch.full_like(exp, 255), exp + 127).to(torch.uint8)
    return q.contiguous(), scales


def dequantize(q: torch.Tensor, scales: torch.Tensor) -> torch.Tensor:
    """float64 values of codes and scales."""
    K = q.shape[-1] * 2
    code = torch.stack([q & 15, q >> 4], -1).reshape(*q.shape[:-1], K).long()
    grid = torch.tensor(GRID + tuple(-g for g in GRID), dtype=torch.float64, device=q.device)
    s = scales[..., :K // 32].double()
    f = torch.where(s == 255, torch.full_like(s, math.nan), torch.exp2(s - 127))
    return (grid[code].reshape(*q.shape[:-1], K // 32, 32) * f[..., None]).reshape(*q.shape[:-1], K)


def rounded(x: torch.Tensor) -> torch.Tensor:
    return dequantize(*quantize(x))


def flip_step(a: torch.Tensor, err: torch.Tensor) -> torch.Tensor:
    """How far rounded(a') can lie from rounded(a) for |a' - a| <= err: 0 where no border lies within err of a, else
    the distance of the numbers on both sides.  A block whose largest magnitude may cross a power of two may change its
    scale: then each element may move by the coarser scale's step at its place."""
    b = a.reshape(*a.shape[:-1], -1, 32)
    e = err.reshape(b.shape)
    lo, hi = b - e, b + e
    amax_lo = torch.where(lo.sign() == hi.sign(), torch.minimum(lo.abs(), hi.abs()), torch.zeros_like(lo)).amax(-1)
    amax_hi = torch.maximum(lo.abs(), hi.abs()).amax(-1)

    def at(x, amax):
        exp = (torch.frexp(amax).exponent - 3).clamp(-127, 127)
        exp = torch.where(amax > 0, exp, torch.full_like(exp, -127))
        f = torch.exp2(exp.double())[..., None]
        v = (x / f).abs().clamp(max=6.0)
        grid = torch.tensor(GRID, dtype=torch.float64, device=x.device)
        near = grid[(v[..., None] - grid).abs().argmin(-1)]
        return near * torch.sign(x) * f
    vals = torch.stack([at(x, m) for x in (lo, hi, b) for m in (amax_lo, amax_hi)])
    return (vals.amax(0) - vals.amin(0)).reshape(a.shape)


def ffn_rows(x, w13, w2):
    """One expert's rows: (y, bound) in float64 for x, w13 [2I, d], w2 [d, I] given as the values they stand for.
    bound: how far fp32 sums and activations, rounded to the format where they cross a border, can move y."""
    i = w2.shape[1]
    z, zm = x @ w13.t(), x.abs() @ w13.abs().t()
    g, u = z[:, :i], z[:, i:]
    f = 2.0 ** -24
    ez = (x.shape[1] + 8) * f * zm
    act = g * torch.sigmoid(g) * u
    # silu in fp32: its slope is at most 1.1; the exponential's exponent is rounded (|g| 2^-24 and a few ulp)
    ea = 1.1 * ez[:, :i] * u.abs() + (g * torch.sigmoid(g)).abs() * ez[:, i:] + (2 * g.abs() + 16) * f * act.abs()
    ea = ea + ez[:, :i] * ez[:, i:]
    a = rounded(act)
    move = flip_step(act, ea)
    y = a @ w2.t()
    return y, move @ w2.abs().t() + (i + 8) * f * ((a.abs() + move) @ w2.abs().t())
