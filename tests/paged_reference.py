"""Plain 64-bit implementations of the operators on a paged cache, on the CPU.

Written from the formulas in include/kvxfer.h: loops over sequences, indexing, products.
The attention reference also returns a bound on the kernel's error, element by element.
"""
from __future__ import annotations

import math

import torch

TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}


def paged(region: torch.Tensor, head_major: bool) -> torch.Tensor:
    """A region as [block][token][head][dim]."""
    return region.transpose(1, 2) if head_major else region


def cache_of(region, head_major, table, n):
    """The first n cached tokens of a sequence, [n][heads][dim] in 64 bits."""
    bits = region.view(torch.uint8 if region.element_size() == 1 else torch.int16)
    view = paged(bits, head_major)
    bs = view.shape[1]
    j = torch.arange(n)
    return view[table.long()[j // bs], j % bs].contiguous().view(region.dtype).to(torch.float32).double()


def visible(q_len, kv_len, window=0, prefix=0, full=False):
    """[q_len][kv_len] truth values."""
    p = kv_len - q_len + torch.arange(q_len)[:, None]
    j = torch.arange(kv_len)[None, :]
    if full:
        return torch.ones(q_len, kv_len, dtype=torch.bool)
    near = (j <= p) if window == 0 else (j <= p) & (j > p - window)
    return near | (j < prefix)


def attend(q, k, v, *, scale, softcap=0.0, slopes=None, window=0, prefix=0, full=False, k_scale=1.0,
           v_scale=1.0, kind="bf16", q_len=None):
    """One sequence: q [q_len][Hq][D], k and v [kv_len][H][D], all in 64 bits.  Returns out, lse
    and the bounds of their errors.

    The bounds.  u is half a step of the 16-bit type, f = 2^-24 of the 32-bit one.
      scores   |ds| <= f ((D + 8) scale sum|q k| + 8 |s|) + 2^-21 softcap + 4 f slope |p - j|: products are exact,
               the D sums, the scale and the base change round in 32 bits; tanh is
               1 - 2 / (e + 1) with a few roundings of values near 1
      weights  relative 2 |ds| + 8 f, plus u for their rounding (numerator only); half
               weights below 2^-14 lose up to 2^-25 absolute, the largest weight being >= 1
      sums     n additions in 32 bits, 4 n f at most with the join's
      out      half a step of the result at the end (and the smallest subnormals')
    with a = sum_j w_j |v_j| for what the errors of the weights are worth in the result."""
    n_q, hq, dim = q.shape
    n, h, _ = k.shape
    g = hq // h
    f = 2.0 ** -24
    u = torch.finfo(TYPES[kind]).eps / 2
    out = torch.zeros(n_q, hq, dim, dtype=torch.float64)
    lse = torch.full((n_q, hq), -math.inf, dtype=torch.float64)
    d_out, d_lse = torch.zeros_like(out), torch.zeros_like(lse)
    if n == 0 or n_q == 0:
        return out, lse, d_out, d_lse
    seen = visible(n_q, n, window, prefix, full)
    far = (n - n_q + torch.arange(n_q)[:, None] - torch.arange(n)[None, :]).abs().double()
    some = seen.any(-1)
    for x in range(hq):
        kk, vv = k[:, x // g] * k_scale, v[:, x // g] * v_scale
        s = q[:, x] @ kk.t() * scale
        ds = f * ((dim + 8) * abs(scale) * (q[:, x].abs() @ kk.abs().t()) + 8 * s.abs())
        if softcap:
            s = softcap * torch.tanh(s / softcap)
            ds = ds + 2.0 ** -21 * softcap
        if slopes is not None:
            s = s - float(slopes[x]) * far
            ds = ds + 4 * f * abs(float(slopes[x])) * far
        s = torch.where(seen, s, -math.inf)
        e = torch.where(seen, ds, 0.0).amax(-1)
        z = torch.logsumexp(s, -1)
        w = torch.where(seen, torch.exp(s - z[:, None]), 0.0)
        lse[:, x] = z
        o = torch.where(seen[:, :, None], w[:, :, None] * vv[None], 0.0).sum(1) if not torch.isfinite(vv).all() \
            else w @ vv
        va = torch.nan_to_num(vv.abs(), nan=0.0, posinf=0.0)
        a = w @ va
        out[:, x] = torch.where(some[:, None], o, 0.0)
        small = 2.0 ** -25 * (seen.double() @ va) if kind == "f16" else 0.0
        rel = (2 * e + (4 * n + 64) * f)[:, None]
        d_out[:, x] = a * (u + rel) + small + o.abs() * (u + rel) + torch.finfo(TYPES[kind]).smallest_normal * u * 2
        d_lse[:, x] = e + (4 * n + 64) * f + 8 * f * z.abs()
    return out, lse, d_out, torch.where(some[:, None], d_lse, 0.0)


def appended(x, scale, cache):
    """New tokens as the pool holds them."""
    if cache != "e4m3":
        return x.to(TYPES[cache])
    y = (x.float() / torch.tensor(scale, dtype=torch.float32)).clamp(-448, 448)
    return y.to(torch.float8_e4m3fn)
