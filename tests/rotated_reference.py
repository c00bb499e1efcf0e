"""Plain 64-bit implementations of the rotation and of 4-bit rows, on the CPU, written from the formulas in
include/kvxfer.h: whole-number angles, loops over groups, nearest values by distance."""
from __future__ import annotations

import math

import numpy as np
import torch

GRID = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def _pi_bits(n):
    """2^n pi, by whole numbers (Machin)."""
    one = 1 << (n + 64)

    def arctan_of_inverse(x):
        t = one // x
        total, k, sign = t, 3, -1
        while t:
            t //= x * x
            total += sign * (t // k)
            k, sign = k + 2, -sign
        return total

    return (4 * (4 * arctan_of_inverse(5) - arctan_of_inverse(239))) >> 64


_N = 320
_TWO_PI = 2 * _pi_bits(_N)


def turned_by(pos, inv_freq):
    """(cos, sin) [len(pos)][len(inv_freq)] of pos * inv_freq, reduced exactly: the frequency is the fraction that its
    64-bit float is."""
    c = np.empty((len(pos), len(inv_freq)))
    s = np.empty_like(c)
    for j, f in enumerate(inv_freq):
        num, den = float(f).as_integer_ratio()
        for i, p in enumerate(pos):
            scaled = (int(p) * num << _N) // den            # the angle in 2^-N radians
            rest = scaled % _TWO_PI
            rest = rest - _TWO_PI if rest > _TWO_PI // 2 else rest
            a = float(rest / (1 << _N)) if abs(rest) < 1 << 1000 else 0.0
            c[i, j], s[i, j] = math.cos(a), math.sin(a)
    return torch.from_numpy(c), torch.from_numpy(s)


def rotate(x, c, s, adjacent, amplitude=1.0):
    """[rows][heads][dim] in 64 bits, and the size of the pair each element comes from."""
    n = c.shape[-1]
    out, size = x.clone(), torch.zeros_like(x)
    for i in range(n):
        a, b = (2 * i, 2 * i + 1) if adjacent else (i, i + n)
        ci, si = c[:, i, None] * amplitude, s[:, i, None] * amplitude
        out[..., a] = x[..., a] * ci - x[..., b] * si
        out[..., b] = x[..., a] * si + x[..., b] * ci
        size[..., a] = size[..., b] = amplitude * (x[..., a].abs() + x[..., b].abs())
    return out, size


def mx4_of(x):
    """[..., dim] in 64 bits to (values' indexes into GRID with the sign in bit 3, scale bytes)."""
    flat = x.double().reshape(-1, 32).numpy()
    codes, scales = np.zeros(flat.shape, np.uint8), np.zeros(len(flat), np.uint8)
    grid = np.array(GRID)
    for i, g in enumerate(flat):
        if not np.isfinite(g).all():
            scales[i] = 255
            continue
        most = float(np.abs(g).max())
        e = 1
        if most > 0:
            e = max(1, math.frexp(most)[1] - 4 + 127)
            while most > 7 * 2.0 ** (e - 127):
                e += 1
        scales[i] = e
        y = np.abs(g) / 2.0 ** (e - 127)
        d = np.abs(y[:, None] - grid)
        near = d.min(1, keepdims=True)
        # of two equally near, the even index
        best = np.where(d == near, np.arange(8) % 2 + np.arange(8) / 100, 9).argmin(1)
        codes[i] = best | (np.signbit(g) << 3)
    return torch.from_numpy(codes).reshape(x.shape), torch.from_numpy(scales).reshape(x.shape[:-1] + (x.shape[-1] // 32,))


def pack(codes, scales, row):
    """Row bytes, 0xA5 behind the scales."""
    out = torch.full(codes.shape[:-1] + (row,), 0xA5, dtype=torch.uint8)
    half = codes.shape[-1] // 2
    out[..., :half] = codes[..., 0::2] | (codes[..., 1::2] << 4)
    out[..., half:half + scales.shape[-1]] = scales
    return out


def unpack(rows, dim):
    """Row bytes to their values in 64 bits."""
    half = dim // 2
    codes = torch.stack([rows[..., :half] & 15, rows[..., :half] >> 4], -1).flatten(-2).long()
    grid = torch.tensor(GRID + [-g for g in GRID], dtype=torch.float64)
    e = rows[..., half:half + dim // 32].double()
    scale = torch.where(e == 255, math.nan, torch.exp2(e - 127))
    return (grid[codes].unflatten(-1, (-1, 32)) * scale[..., None]).flatten(-2)


def row_bytes(dim, heads):
    row = -(-dim * 17 // 32 // 4) * 4
    while row * heads % 16:
        row += 4
    return row


def random_rows(shape, dim, row, gen, gain=1.0):
    """Random rows of a 4-bit pool: codes as rounding leaves them, scales around gain."""
    codes = torch.randint(0, 16, shape + (dim,), generator=gen, dtype=torch.uint8)
    e = torch.randint(-3, 1, shape + (dim // 32,), generator=gen) + 127 + round(math.log2(gain))
    return pack(codes, e.to(torch.uint8), row)
