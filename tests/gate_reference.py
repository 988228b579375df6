"""The gate's gradients in 64 bits, term by term, and how far a kernel's may be from them.

u = 2^-24 is an fp32 rounding.  A kernel sums four products over the d columns of a token and
branch; each passes through at most `m` roundings on its way, so a sum is off by at most m u times
the sum of its terms' magnitudes.  With S = sum h w k, D = sum dout v, and kS, kD the ratios of
those magnitudes' sums to |S| and |D|:
  x = rh rk S / sqrt(d)       m u (kS + 1) relative (the norms' sums enter through a root each)
  root = sqrt|x|              half of that
  dx = D g (1 - g) / (2 root) m u kD + (root + 1) / 2 times x's: the logarithm of g (1 - g) / root
                              falls by at most 1 + 1 / root per unit of root
so that dS = dx rh rk / sqrt(d) and dx x rh^2 / d are within rho = m u (kD + (root + 3) (kS + 2)) + 64 u,
64 u being the handful of roundings after the sums.  The outputs are
  dh = dout + dS w k - (dx x rh^2 / d) h      dk = dS w h - (dx x rk^2 / d) k
and are rounded to BF16 once (2^-8 of their size, with room for the step to the next binade), so
each is within 2^-8 |ref| + rho (|first term| + |second term|) + 4 u |dout|.
dv = sum_b g_b dout_b: g is off by its slope's share of x's error.
"""
from __future__ import annotations

import math

import torch

F = torch.float64
U = 2.0 ** -24


def roundings(hc, d):
    """m for any of the kernels: a thread's own columns (8 at a time, four running pairs, or 8 a
    step over 320 threads where a token does not fit a cluster), then a warp's five exchanges, ten
    warps, eight CTAs, and the products' own."""
    return 32 if d <= 20_480 and hc * d < 40_000 else 8 * -(-d // (8 * 320)) + 24


class GateGradients:
    """h [T, hc, d], kv [T, (hc + 1) d], dy [T, hc, d], weights [hc, d], on [T, 1, 1]: 1 for text."""

    def __init__(self, h, kv, on, wq, wk, dy, eps=1e-6):
        h, kv, wq, wk, dy, on = (t.to(F) for t in (h, kv, wq, wk, dy, on))
        T, hc, d = h.shape
        k, v, w = kv[:, :hc * d].reshape(T, hc, d), kv[:, hc * d:].reshape(T, 1, d), wq * wk
        rh = (h.square().mean(2, keepdim=True) + eps).rsqrt()
        rk = (k.square().mean(2, keepdim=True) + eps).rsqrt()
        S, D = (h * w * k).sum(2, keepdim=True), (dy * v).sum(2, keepdim=True)
        x = rh * rk * S / math.sqrt(d)
        root = x.abs().clamp_min(1e-6).sqrt()
        g = torch.sigmoid(torch.copysign(root, x))
        dx = on * (x.abs() > 1e-6) * D * g * (1 - g) / (2 * root)
        dS = dx * rh * rk / math.sqrt(d)
        self.first = dict(dh=dS * w * k, dk=dS * w * h)
        self.second = dict(dh=-dx * x * rh.square() / d * h, dk=-dx * x * rk.square() / d * k)
        self.dh = dy + self.first["dh"] + self.second["dh"]
        self.dk = self.first["dk"] + self.second["dk"]
        self.dv = (on * g * dy).sum(1)
        dwqk = (dS * h * k).sum(0)
        self.dwq, self.dwk = dwqk * wk, dwqk * wq
        self.hc, self.d, self.dy = hc, d, dy
        mu = roundings(hc, d) * U
        kS = (h * w * k).abs().sum(2, keepdim=True) / S.abs().clamp_min(1e-300)
        kD = (dy * v).abs().sum(2, keepdim=True) / D.abs().clamp_min(1e-300)
        self.rho = mu * (kD + (root + 3) * (kS + 2)) + 64 * U
        self.dg = g * (1 - g) * root / 2 * mu * (kS + 2) + 16 * U

    def misses(self, dh, dkv):
        """The outputs that are further off than they may be."""
        T, hc, d = self.dy.shape
        dkv = dkv.to(F)
        got = dict(dh=dh.to(F), dk=dkv[:, :hc * d].reshape(T, hc, d), dv=dkv[:, hc * d:])
        bad = []
        for name in ("dh", "dk"):
            ref = getattr(self, name)
            tol = (2.0 ** -8 * ref.abs() + self.rho * (self.first[name].abs() + self.second[name].abs()) +
                   4 * U * (self.dy.abs() if name == "dh" else 0))
            if not ((got[name] - ref).abs() <= tol).all():
                bad.append(name)
        tol = 2.0 ** -8 * self.dv.abs() + (self.dg * self.dy.abs()).sum(1)
        if not ((got["dv"] - self.dv).abs() <= tol).all():
            bad.append("dv")
        return bad


def gate_inputs(T, hc, d, seed, image=(1,)):
    """Dots from 2e-3 to 30 of either sign, a value so large that what the gate adds to dout is not
    lost in dh's rounding, and a small dout."""
    g = torch.Generator().manual_seed(seed)
    h = torch.randn(T, hc, d, generator=g).bfloat16()
    kv = torch.randn(T, (hc + 1) * d, generator=g)
    wq, wk = (1 + 0.1 * torch.randn(hc, d, generator=g) for _ in range(2))
    k, hw = kv[:, :hc * d].reshape(T, hc, d), h.float() * (wq * wk)
    k -= h.float() * ((hw * k).sum(2, keepdim=True) / (hw * h.float()).sum(2, keepdim=True))
    size = torch.tensor([2e-3, 0.05, 0.4, 2.0, 8.0, 30.0])[torch.arange(T * hc) % 6].reshape(T, hc, 1)
    size = size * torch.sign(torch.rand(T, hc, 1, generator=g) - 0.5)
    # x = lean sqrt(d) / sqrt(1 + lean^2) where k is lean times h and as much else as its norm
    lean = size / (d - size.square()).clamp_min(1.0).sqrt()
    kv[:, :hc * d] = (k + lean * h.float()).reshape(T, hc * d)
    kv[:, hc * d:] *= 64
    dy = (torch.randn(T, hc, d, generator=g) * 2.0 ** -6).bfloat16()
    win = torch.randint(0, 50, (T, 4), generator=g).int()
    for t in image:
        if t < T:
            win[t, 0] = -1
    on = (win[:, 0] != -1).to(F).reshape(T, 1, 1)
    return h, kv, win, wq, wk, dy, on
