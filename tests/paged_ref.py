"""Plain 64-bit references of the rotary, paged-cache and prompt-attention calls (CPU, loops, no blocking).
Shared by their GPU tests and nothing else."""
import math

import torch

BF16 = 2.0 ** -8      # half a step, relative
F16 = 2.0 ** -11
F32 = 2.0 ** -24
E4M3 = torch.float8_e4m3fn


def rope(x, pos, freq, interleaved, amp):
    """x [T][H][d] -> (y fp64, bound on |u| + |v| of each value's pair)."""
    x = x.double().cpu()
    y, mag = x.clone(), torch.zeros_like(x)
    n = freq.numel()
    for t, p in enumerate(pos.tolist()):
        for i, f in enumerate(freq.tolist()):
            turn = ((p * (f % 2 ** 64)) % 2 ** 64) / 2 ** 64        # exact in integers
            c, s = amp * math.cos(2 * math.pi * turn), amp * math.sin(2 * math.pi * turn)
            a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + n)
            u, v = x[t, :, a], x[t, :, b]
            y[t, :, a], y[t, :, b] = u * c - v * s, u * s + v * c
            mag[t, :, a] = mag[t, :, b] = abs(amp) * (u.abs() + v.abs())
    return y, mag


def rope_bound(y, mag):
    """bf16's half step; sin, cos and the angle are within 2^-22, products and sum in fp32 within 2^-23."""
    return BF16 * y.abs() + 2.0 ** -21 * mag + 1e-38


def attention(q, k, v, weight_step):
    """One row: q [d], k, v [n][d] fp64 -> (o, lse, bound on o, bound on lse).

    The bounds count roundings: fp32 dot products (d + 2 steps of 2^-24 of the sum of magnitudes), the score's scaling
    and exponential (2^-22 of its size), weights to `weight_step`, fp32 sums (n / 16 tiles), the output to bf16.
    """
    d, n = q.numel(), k.shape[0]
    if n == 0:
        return torch.zeros(d, dtype=torch.float64), -math.inf, torch.zeros(d), 0.0
    s = k @ q / math.sqrt(d)
    lse = torch.logsumexp(s, 0)
    w = torch.exp(s - lse)
    o = w @ v
    ds = float((((k.abs() @ q.abs()) / math.sqrt(d)).max() * (d + 2) * F32 + s.abs().max() * 2.0 ** -22 + 2.0 ** -21))
    size = w @ v.abs()
    tol = (weight_step + 2 * ds + (n / 16 + 32) * F32) * size + BF16 * o.abs() + 1e-30
    return o, float(lse), tol, ds + (n / 16 + 32) * F32 + abs(float(lse)) * 2.0 ** -22


def check(got, want, tol, what):
    got, want, tol = got.double().cpu(), want.double(), tol.double()
    bad = ~((got - want).abs() <= tol) & ~(got == want)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} outside; worst error "
                           f"{float((got - want).abs()[bad].max()):.3e} against {float(tol[bad].max()):.3e}")
