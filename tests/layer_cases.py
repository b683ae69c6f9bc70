"""Plain forms of attention, layer norm and balance loss in 64 bits, and the
error bounds their tests use (no library code).

Bounds, to first order, u = 2^-24 (half a step of fp32) and h = eps/2 of the
inputs' type; sums of n fp32 products in any order are off by (n + 1) u times
the sum of the absolute products, taken twice here for the higher orders.

  scores        x = scale q k: e_x = 2 (d + 2) u sum |scale q k|; the exponent
                has two more roundings and a hardware power of two (one step)
  weights       P off by r = e_x + e_lse' + 8 u of its size (|x| u in it), and
                rounded to the type before the products: h more, for fp16 also
                half its smallest subnormal relative to a largest weight of 2^8;
                and 2^-126 of itself, as the instruction for powers of two gives
                0 below that: 2^-126 |dout| in dv, 2^-126 (|dP| + |delta|) in dS
  o             (2 r + h) sum P |v|, twice r for the softmax's sum, + n u of it
  lse           the largest e_x + (n + 8 + |lse|) u
  dP            2 (d + 2) u sum |dout v|
  delta         <dout, o> of the rounded o, or sum P dP: the larger, |dout| e_o
                + 2 (d + 2) u sum |dout o| + r sum P |dP|
  dS            P (e_dP + e_delta) + r |dS|, and h |dS| for the rounding
  gradients     sums of these times |k|, |q|, + n u of their terms
and one rounding of the result at the end.
"""
import math

import numpy as np
import torch

GONE = 2.0 ** -126
FLOATS = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
U = 2.0 ** -24


def half_step(dtype):
    """Half a step relative to the value, and half the smallest subnormal."""
    fi = torch.finfo(dtype)
    return fi.eps / 2, fi.smallest_normal * fi.eps / 2


def check(got, want, err, what):
    """got (any type) against want and its error before the last rounding, in fp64."""
    h, tiny = half_step(got.dtype)
    got = got.double().cpu().reshape(want.shape)
    bad = torch.isfinite(want) & ~(torch.abs(got - want) <= err + h * (want.abs() + err) + tiny)
    bad |= torch.isnan(want) & ~torch.isnan(got)
    bad |= torch.isinf(want) & (got != want)
    if bool(bad.any()):
        i = int(torch.nonzero(bad.reshape(-1))[0, 0])
        raise AssertionError("%s: %d of %d over the bound, first at %d: %r for %r (allowed %g)" % (
            what, int(bad.sum()), bad.numel(), i, float(got.reshape(-1)[i]), float(want.reshape(-1)[i]),
            float((err + h * (want.abs() + err) + tiny).reshape(-1)[i])))


class Attention:
    """Sizes and the exact results of one call.  q, k, v, do: fp64 of values of
    the type, [shards][heads][tokens][d]."""

    def __init__(self, N=1, B=1, G=1, S=1, Hq=1, Hkv=1, d=64, queries=None, window=1 << 30, sinks=0, order="head", dtype="bf16"):
        self.N, self.B, self.G, self.S, self.Hq, self.Hkv, self.d = N, B, G, S, Hq, Hkv, d
        self.queries, self.window, self.sinks = S if queries is None else queries, window, sinks
        self.order, self.dtype = order, FLOATS[dtype]
        P, Bl = N // G, B // G
        self.shards, self.hq, self.hkv = N * Bl, Hq // P, Hkv // P
        # rank r of group r // P holds the group's sequences
        self.sequence = [r // P * Bl + i for r in range(N) for i in range(Bl)]

    def inputs(self, seed, sharp=1.0):
        g = torch.Generator()
        g.manual_seed(seed)

        def make(heads, tokens, size=1.0):
            return (torch.randn(self.shards, heads, tokens, self.d, generator=g) * size).to(self.dtype).double()
        return (make(self.hq, self.queries, sharp), make(self.hkv, self.S), make(self.hkv, self.S), make(self.hq, self.queries))

    def buffer(self, x):
        """[shards][heads][tokens][d] as the library's buffer (any type)."""
        return (x if self.order == "head" else x.transpose(1, 2)).contiguous().reshape(-1)

    def shaped(self, flat, heads, tokens):
        if self.order == "head":
            return flat.reshape(self.shards, heads, tokens, self.d)
        return flat.reshape(self.shards, tokens, heads, self.d).transpose(1, 2)

    def sees(self, start, length):
        p = start + torch.arange(self.queries)[:, None]
        j = torch.arange(self.S)[None]
        return (j <= p) & ((p - j < self.window) | (j < self.sinks)) & (p >= 0) & (p < length) & (j < length)

    def exact(self, q, k, v, do, starts, lengths, scale):
        """(value, error before the last rounding) of o, lse, dq, dk, dv.  Hidden
        places take no part, whatever they hold."""
        h, tiny = half_step(self.dtype)
        d, ratio = self.d, self.hq // self.hkv
        names = ("o", "dq", "dk", "dv")
        out = {n: torch.zeros(self.shards, self.hq if n in ("o", "dq") else self.hkv, self.queries if n in ("o", "dq") else self.S, d,
                              dtype=torch.float64) for n in names}
        err = {n: torch.zeros_like(x) for n, x in out.items()}
        lse = torch.full((self.shards, self.hq, self.queries), -math.inf, dtype=torch.float64)
        lse_err = torch.zeros_like(lse)
        for n in range(self.shards):
            b = self.sequence[n]
            vis = self.sees(starts[b], max(0, min(lengths[b], self.S)))
            rows, keys = torch.nonzero(vis.any(1))[:, 0], torch.nonzero(vis.any(0))[:, 0]
            if not len(rows):
                continue
            m = vis[rows][:, keys]
            hide = lambda x: torch.where(m, x, torch.zeros((), dtype=torch.float64))
            # products that skip hidden pairs, so that what stands there reaches nothing
            sums = lambda w, x: torch.where(m[:, :, None], w[:, :, None] * x[None], torch.zeros((), dtype=torch.float64)).sum(1) \
                if not bool(torch.isfinite(x).all()) else torch.where(m, w, torch.zeros((), dtype=torch.float64)) @ x
            cols = lambda w, x: torch.where(m.T[:, :, None], w.T[:, :, None] * x[None], torch.zeros((), dtype=torch.float64)).sum(1) \
                if not bool(torch.isfinite(x).all()) else torch.where(m, w, torch.zeros((), dtype=torch.float64)).T @ x
            count = m.sum(1, keepdim=True).double()
            for hq in range(self.hq):
                hk = hq // ratio
                qi, kj, vj, gi = q[n, hq, rows], k[n, hk, keys], v[n, hk, keys], do[n, hq, rows]
                x = hide(qi @ kj.T * scale)
                ex = hide(2 * (d + 2) * U * (qi.abs() @ kj.abs().T * scale) + 4 * U * x.abs())
                most = torch.where(m, x, torch.full_like(x, -math.inf)).amax(1, keepdim=True)
                e = hide(torch.exp(x - most))
                total = e.sum(1, keepdim=True)
                P = e / total
                le = (ex.amax(1, keepdim=True) + (count + 8) * U + (most + total.log()).abs() * 2 * U)
                r = 2 * (ex + le + 16 * U)
                lost = tiny * 2.0 ** 1 / total if self.dtype is torch.float16 else torch.zeros_like(total)
                o = sums(P, vj)
                eo = sums(P * (2 * r + h + 2 * count * U) + lost, vj.abs())
                out["o"][n, hq, rows], err["o"][n, hq, rows] = o, eo
                lse[n, hq, rows], lse_err[n, hq, rows] = (most + total.log())[:, 0], le[:, 0]
                dP = hide(gi @ vj.T)
                edP = hide(2 * (d + 2) * U * (gi.abs() @ vj.abs().T))
                delta = (P * dP).sum(1, keepdim=True)
                edelta = (gi.abs() * (eo + h * o.abs() + tiny)).sum(1, keepdim=True) + \
                    2 * (d + 2) * U * (gi * o).abs().sum(1, keepdim=True) + (P * (r * dP.abs() + edP)).sum(1, keepdim=True)
                dS = P * (dP - delta)
                edS = P * (edP + edelta + 4 * U * (dP.abs() + delta.abs())) + (r + h) * dS.abs() + hide(tiny + GONE * (dP.abs() + delta.abs()))
                out["dq"][n, hq, rows] = sums(dS, kj) * scale
                err["dq"][n, hq, rows] = sums(edS + 2 * count * U * dS.abs(), kj.abs()) * scale
                many = 2 * (ratio * len(rows) + 4) * U
                out["dk"][n, hk, keys] += cols(dS, qi) * scale
                err["dk"][n, hk, keys] += cols(edS + many * dS.abs(), qi.abs()) * scale
                out["dv"][n, hk, keys] += cols(P, gi)
                err["dv"][n, hk, keys] += cols(P * (r + h + many) + hide(torch.full_like(P, tiny + GONE)), gi.abs())
        return {n: (out[n], err[n]) for n in names} | {"lse": (lse, lse_err)}


# ------------------------------------------------------ norm, balance loss --

def norm_exact(x, w, bias, eps):
    mean = x.mean(1, keepdim=True)
    var = (x - mean).square().mean(1, keepdim=True)
    rstd = (var + eps) ** -0.5
    return (x - mean) * rstd * w + (0 if bias is None else bias), mean[:, 0], rstd[:, 0]


def norm_errors(x, w, bias, eps):
    """Of y, mean and rstd before their last rounding: the mean is a sum of D
    numbers; x - mean carries its error, the squares twice that."""
    D = x.shape[1]
    y, mean, rstd = norm_exact(x, w, bias, eps)
    emean = 2 * (D + 2) * U * x.abs().mean(1)
    dev = (x - mean[:, None]).abs()
    evar = 2 * (D + 4) * U / rstd ** 2 + 2 * emean ** 2 + 4 * U * (x.abs().amax(1) * dev.amax(1))
    erstd = rstd * (evar * rstd ** 2 / 2 + 4 * U)
    ey = ((emean[:, None] + 2 * U * (x.abs() + mean.abs()[:, None])) * rstd[:, None] + dev * (erstd + 4 * U * rstd)[:, None]) * w.abs() \
        + 4 * U * y.abs() + (0 if bias is None else 2 * U * bias.abs())
    return ey, emean, erstd


def norm_grad_exact(dy, x, w, mean, rstd):
    """With the statistics as given."""
    xhat = (x - mean[:, None]) * rstd[:, None]
    g = dy * w
    D = x.shape[1]
    dx = rstd[:, None] * (g - g.mean(1, keepdim=True) - xhat * (g * xhat).mean(1, keepdim=True))
    exh = 4 * U * (x.abs() + mean.abs()[:, None]) * rstd[:, None]
    c = 2 * (D + 4) * U
    edx = rstd[:, None] * (8 * U * g.abs() + c * g.abs().mean(1, keepdim=True) + (exh + 8 * U * xhat.abs()) * (g * xhat).mean(1, keepdim=True).abs()
                           + xhat.abs() * ((c * (g * xhat).abs()).mean(1, keepdim=True) + (g.abs() * exh).mean(1, keepdim=True)))
    T = 2 * (x.shape[0] + 4) * U
    return (dx, edx), ((dy * xhat).sum(0), (dy.abs() * (exh + T * xhat.abs())).sum(0)), (dy.sum(0), T * dy.abs().sum(0))


def balance_exact(logits, ids, live, coef, E):
    """loss, counts, slope, p of rows of fp64 scores; live [T] truth values."""
    T, K = ids.shape
    rows = np.nonzero(live)[0]
    L = len(rows)
    chosen = ids[rows].reshape(-1)
    counts = np.bincount(chosen[(chosen >= 0) & (chosen < E)], minlength=E)
    x = logits[rows]
    p = torch.zeros(T, E, dtype=torch.float64)
    if L:
        p[rows] = torch.softmax(x, 1)
    slope = torch.from_numpy(coef * E * counts / (K * L) / L if L else np.zeros(E))
    return (slope * p.sum(0)).sum(), counts, slope, p
