"""A pool of random pages on the GPU with its host copy, and the calls of the rotated operators on it, for the GPU
tests of rotations and 4-bit pools."""
from __future__ import annotations

import math

import numpy as np
import torch

import paged_reference as ref
import rotated_reference as rot
from paged_layout_transfer_amd import kvxfer as K

KIND = {"f16": K.KV_TYPE_F16, "bf16": K.KV_TYPE_BF16, "e4m3": K.KV_TYPE_E4M3, "mx4": K.KV_TYPE_MX4}
TYPES = ref.TYPES


def say(*what):
    print("[gpu]", *what, flush=True)


def frequencies(pairs, base=10000.0):
    return base ** (-np.arange(pairs) / pairs)


class Cache:
    """Regions of raw bytes; `pad` bytes between blocks and the spare bytes of 4-bit rows hold 0xA5."""

    def __init__(self, *, layers=1, heads=2, dim=64, page=16, blocks=64, head_major=False, kind="bf16", cache="mx4",
                 seed=0, pad=0, row=0, gain=1.0):
        self.layers, self.heads, self.dim, self.page, self.blocks = layers, heads, dim, page, blocks
        self.head_major, self.kind, self.cache = head_major, kind, cache
        self.k_scale, self.v_scale = (0.037, 0.021) if cache == "e4m3" else (1.0, 1.0)
        self.wide = 1 if cache in ("e4m3", "mx4") else 2
        self.row = row or (rot.row_bytes(dim, heads) if cache == "mx4" else dim * self.wide)     # bytes of one head
        gen = torch.Generator().manual_seed(seed)
        shape = (2 * layers, blocks) + ((heads, page) if head_major else (page, heads))
        if cache == "mx4":
            rows = rot.random_rows(shape, dim, self.row, gen, gain)
        else:
            x = torch.randn(shape + (dim,), generator=gen) * gain
            x = (x * 25).clamp(-448, 448) if cache == "e4m3" else x
            rows = x.to(TYPES[cache]).view(torch.uint8)
        self.stride = page * heads * self.row + pad
        self.flat = torch.full((2 * layers, blocks, self.stride), 0xA5, dtype=torch.uint8)
        self.bytes = self.flat[:, :, :self.stride - pad].view(shape + (self.row,))      # a view: the host copy
        self.bytes.copy_(rows)
        self.dev = self.flat.cuda()
        self.handle = K.kv_pool_create(K.make_pool_desc(
            layers, 2, heads, self.row // self.wide, self.wide, page, blocks, self.stride,
            [self.dev.data_ptr() + i * self.dev.stride(0) for i in range(2 * layers)],
            K.KV_PAGE_HEAD_MAJOR if head_major else K.KV_PAGE_TOKEN_MAJOR))
        self.plans, self.rotations = [], []

    def plan(self, heads_q, max_seqs, max_tokens, window=0, full=False):
        h = K.kv_attn_plan_create(self.handle, K.make_attn_desc(
            heads_q, KIND[self.kind], KIND[self.cache], max_seqs, max_tokens, window, K.KV_ATTN_FULL if full else 0))
        self.plans.append(h)
        return h

    def rotation(self, freq, adjacent=False, amplitude=1.0):
        h = K.kv_rotation_create(K.make_rotation_desc(freq, K.KV_ROT_ADJACENT if adjacent else K.KV_ROT_HALVES, amplitude))
        self.rotations.append(h)
        return h

    def view(self, region):
        """[block][token][head][row bytes] of the host copy."""
        x = self.bytes[region]
        return x.transpose(1, 2) if self.head_major else x

    def rows(self, region, table, places):
        """The rows of a sequence's cached tokens, [n][heads][row bytes]; writable through put()."""
        places = torch.as_tensor(places).long()
        return self.view(region)[table.long()[places // self.page], places % self.page]

    def put(self, region, table, places, rows):
        places = torch.as_tensor(places).long()
        self.view(region)[table.long()[places // self.page], places % self.page] = rows

    def values(self, rows):
        """Row bytes as 64-bit values, e4m3 without its scale."""
        if self.cache == "mx4":
            return rot.unpack(rows, self.dim)
        return rows.contiguous().view(TYPES[self.cache]).to(torch.float32).double()

    def upload(self):
        self.dev.copy_(self.flat)

    def now(self):
        """The device's bytes in the host copy's shape, and the whole of them."""
        torch.cuda.synchronize()
        flat = self.dev.cpu()
        return flat[:, :, :self.bytes[0, 0].numel()].view(self.bytes.shape), flat

    def close(self):
        torch.cuda.synchronize()
        for h in self.plans:
            K.kv_attn_plan_destroy(h)
        for h in self.rotations:
            K.kv_rotation_destroy(h)
        K.kv_pool_destroy(self.handle)

    def __enter__(self):
        return self

    def __exit__(self, *_):
        self.close()


def deal(cache, lens, seed=1):
    """One table per sequence, its pages distinct; the tail of each table holds ids no one may follow."""
    ids = np.random.default_rng(seed).permutation(cache.blocks).astype(np.int32)
    tables, at = [], 0
    for _, n, *_ in lens:
        k = -(-n // cache.page)
        assert at + k <= cache.blocks, "pool too small"
        tables.append(torch.from_numpy(np.concatenate([ids[at:at + k], np.array([-7, 1 << 30], np.int32)])))
        at += k
    return tables


def seqs_of(tables_d, lens, first=0):
    out, at = [], first
    for t, (q, n, *prefix) in zip(tables_d, lens):
        out.append((t, t.numel(), n, at, q, prefix[0] if prefix else 0))
        at += q
    return out, at


def rounded(cache, y, size, scale):
    """What a row of the pool may hold of values y [.., dim] in 64 bits whose pairs have `size`: (lowest, highest)
    values for 16- and 8-bit pools.

    The error before the rounding: cosine and sine from a fraction of a turn cut to 2^-32 turns (1.5e-9 =
    2^-29), its conversion and the product with 2 pi / 2^32 (two roundings, so 2^-23 of an angle up to 0.79), the series'
    ends (2^-29, 2^-25 of roundings in its last two steps), the amplitude (2^-24): under 2^-22 of the pair's
    size; two products and a sum: 3 * 2^-24 of it.  2^-21 covers them.  e4m3 divides by the scale: 2^-24 more."""
    slack = size * 2.0 ** -21
    lo, hi = (y - slack) / scale, (y + slack) / scale
    if cache == "e4m3":
        lo, hi = lo - (y / scale).abs() * 2.0 ** -23, hi + (y / scale).abs() * 2.0 ** -23
        lo, hi = lo.clamp(-448, 448), hi.clamp(-448, 448)
    # rounding is monotonous: the value lies between the roundings of the bounds
    t = TYPES[cache]
    return round_to(lo, t), round_to(hi, t)


def round_to(x, t):
    """64-bit values to the nearest of a type, once (a cast through 32 bits could round twice: it is compared)."""
    y = x.to(torch.float32)
    # towards the odd neighbour where 32 bits are not exact, so that the second rounding sees which side is larger
    bits = y.view(torch.int32)
    wrong = y.double() != x
    toward = torch.where(y.double().abs() > x.abs(), bits - 1, bits)     # truncated
    bits = torch.where(wrong, toward | 1, bits)
    return bits.view(torch.float32).to(t).to(torch.float32).double()


def check_between(got, lo, hi, what):
    bad = (got < lo) | (got > hi) | torch.isnan(got) & ~torch.isnan(lo)
    assert not bad.any(), "%s: %d of %d off, the first at %s: %r outside %r .. %r" % (
        what, int(bad.sum()), bad.numel(), bad.nonzero()[0].tolist(), float(got[bad][0]), float(lo[bad][0]), float(hi[bad][0]))


def scale_of(dim):
    return 1 / math.sqrt(dim)
