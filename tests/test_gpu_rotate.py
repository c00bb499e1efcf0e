"""Rotated appends, shifts of cached keys, reads and 4-bit pools on the GPU, against plain 64-bit implementations
(tests/rotated_reference.py, tests/paged_reference.py).  Every case is printed before its first launch."""
from __future__ import annotations

import math

import numpy as np
import pytest
import torch

import paged_reference as ref
import rotated_reference as rot
from paged_layout_transfer_amd import kvxfer as K
from rotated_harness import (KIND, TYPES, Cache, check_between, deal, frequencies, round_to, rounded, say, scale_of,
                             seqs_of)

pytestmark = pytest.mark.gpu

LENS = [(5, 21), (0, 9), (1, 1), (33, 33), (1, 40), (0, 0), (8, 24), (16, 31), (2, 17)]


def new_tokens(rows, heads_q, heads, dim, kind, seed):
    """A fused projection's rows (q, k, v of a token side by side), three rows to spare."""
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn((rows + 3, heads_q + 2 * heads, dim), generator=gen) * 1.3
    return x.to(TYPES[kind])


def append_case(cache, lens, heads_q, freq, *, adjacent=False, amplitude=1.0, positions=None, seed=3, in_place=False,
                with_q=True, x=None):
    """kv_append_rotated, checked bit by bit (4-bit pools) or against bounds, and for what it must not touch."""
    H, D, n = cache.heads, cache.dim, len(freq)
    tables = deal(cache, lens)
    tables_d = [t.cuda() for t in tables]
    seqs, rows = seqs_of(tables_d, lens)
    x = new_tokens(rows, heads_q, H, D, cache.kind, seed) if x is None else x
    x_d = x.cuda()
    q_d, k_d, v_d = x_d.split([heads_q, H, H], dim=1)
    out = q_d if in_place else torch.full((rows + 3, heads_q + 1, D), 7.0, dtype=TYPES[cache.kind], device="cuda")[:, :heads_q]
    plan = cache.plan(heads_q, len(lens), max(1, rows))
    stream = torch.cuda.current_stream()
    K.kv_attn_plan_set(plan, K.make_seqs(seqs), stream)
    pos_d = None if positions is None else torch.tensor(positions + [11, 12, 13], dtype=torch.int32).cuda()
    r = cache.rotation(freq, adjacent, amplitude)
    torch.cuda.synchronize()
    say("append", cache.kind, cache.cache, "heads", heads_q, H, "dim", D, "pairs", n, "adjacent", adjacent, "page", cache.page,
        "head_major", cache.head_major, "row", cache.row, "positions", positions is not None, "in_place", in_place)
    K.kv_append_rotated(plan, 0, r, K.make_rotate_args(q_d if with_q else None, out if with_q else None, pos_d),
                        K.make_append_args(k_d, v_d, n_tokens=rows + 3, k_scale=cache.k_scale, v_scale=cache.v_scale), stream)
    assert K.kv_pool_get_error(cache.handle, stream) == 0
    place = np.concatenate([np.arange(c - q, c) for q, c, *_ in lens] + [np.zeros(0)]).astype(np.int64)
    c, s = rot.turned_by(place.tolist() if positions is None else positions, freq)
    q, k, v = (t[:rows].double() for t in x.split([heads_q, H, H], dim=1))
    got = out.cpu()
    if with_q:
        want, size = rot.rotate(q, c, s, adjacent, amplitude)
        check_between(got[:rows].double(), *rounded(cache.kind, want, size, 1.0), "q")
    untouched = x[rows:, :heads_q] if in_place else torch.full_like(got[rows:], 7.0)
    assert torch.equal(got[rows:], untouched) and (with_q or (got == 7).all())
    want, size = rot.rotate(k, c, s, adjacent, amplitude)
    now, flat = cache.now()
    live, at = cache.bytes, 0
    for t, (n_q, n_c, *_) in zip(tables, lens):
        places = np.arange(n_c - n_q, n_c)
        mine = slice(at, at + n_q)
        at += n_q
        if cache.cache == "mx4":
            for region, y in ((0, want), (1, v)):
                old = cache.rows(region, t, places)
                packed = rot.pack(*rot.mx4_of(y[mine]), cache.row)
                packed[..., D * 17 // 32:] = old[..., D * 17 // 32:]
                cache.put(region, t, places, packed)
            continue
        for region, y, z, scale in ((0, want, size, cache.k_scale), (1, v, torch.zeros_like(v), cache.v_scale)):
            f = float(np.float32(scale)) if cache.cache == "e4m3" else 1.0
            keep, cache.bytes = cache.bytes, now
            rows_now = cache.rows(region, t, places)
            cache.bytes = keep
            check_between(cache.values(rows_now), *rounded(cache.cache, y[mine], z[mine], f), "kv"[region])
            cache.put(region, t, places, rows_now)     # the rest of the pool is compared whole below
    assert torch.equal(now, live), "wrote outside its rows, or other 4-bit values"
    assert torch.equal(flat[:, :, live[0, 0].numel():], cache.flat[:, :, live[0, 0].numel():])


SHAPES = [      # heads_q, heads, dim, pairs, page, head_major
    (8, 2, 128, 64, 16, False),
    (8, 2, 64, 32, 16, True),
    (4, 4, 128, 16, 24, True),      # a quarter of the head turns
    (5, 1, 256, 128, 32, False),
    (3, 3, 96, 20, 7, False),       # a run of four past whole vectors
    (40, 8, 128, 64, 16, False),    # more units than threads
    (6, 6, 32, 4, 1, True),
]


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("adjacent", [False, True], ids=["halves", "adjacent"])
@pytest.mark.parametrize("kind,store", [("bf16", "bf16"), ("f16", "f16"), ("bf16", "e4m3"), ("f16", "mx4"), ("bf16", "mx4")])
def test_rotated_append(shape, adjacent, kind, store):
    heads_q, heads, dim, pairs, page, head_major = shape
    with Cache(heads=heads, dim=dim, page=page, blocks=200 if page < 16 else 40, head_major=head_major, kind=kind, cache=store, pad=32) as c:
        append_case(c, LENS, heads_q, frequencies(pairs), adjacent=adjacent)


@pytest.mark.parametrize("dim,pairs", [(72, 36), (80, 40), (8, 4), (104, 12)])
@pytest.mark.parametrize("store", ["f16", "e4m3"])
def test_rotated_append_of_odd_widths(dim, pairs, store):
    dim, pairs = (dim, pairs) if store == "f16" or dim % 16 == 0 else (112, 52)
    for adjacent in (False, True):
        with Cache(heads=2, dim=dim, page=16, blocks=40, kind="f16", cache=store) as c:
            append_case(c, LENS, 4, frequencies(pairs, 500000.0), adjacent=adjacent, amplitude=1.25)


@pytest.mark.parametrize("store", ["bf16", "mx4"])
@pytest.mark.parametrize("adjacent", [False, True])
def test_queries_turn_in_place_or_not_at_all(store, adjacent):
    with Cache(heads=2, dim=128, blocks=40, cache=store) as c:
        append_case(c, LENS, 8, frequencies(64), adjacent=adjacent, in_place=True)
    with Cache(heads=2, dim=128, blocks=40, cache=store) as c:
        append_case(c, LENS, 8, frequencies(64), adjacent=adjacent, with_q=False)


@pytest.mark.parametrize("store", ["bf16", "mx4"])
def test_positions_of_either_sign_and_any_size(store):
    rows = sum(q for q, *_ in LENS)
    far = np.random.default_rng(5).integers(-2 ** 31, 2 ** 31, rows).tolist()
    far[:8] = [0, -1, 1, 2 ** 31 - 1, -2 ** 31, 2 ** 30, 131072, -131071]
    # the slowest turns, none at all, more than one turn a position, and quarters of a turn
    freq = np.concatenate([frequencies(24), [0.0, 2.0 ** -30, 2.0 ** -60, math.pi / 2, math.pi, 100.0, 2.0 ** 20, 6.5]])
    with Cache(heads=2, dim=64, blocks=40, cache=store) as c:
        append_case(c, LENS, 4, freq, positions=far)


def test_rows_wider_than_their_values_keep_the_rest():
    for head_major in (False, True):
        with Cache(heads=1, dim=128, blocks=40, row=80, head_major=head_major) as c:
            append_case(c, LENS, 4, frequencies(64))
        with Cache(heads=4, dim=64, blocks=40, row=48, head_major=head_major) as c:
            append_case(c, LENS, 4, frequencies(32))


SPECIAL = [
    [0.0] * 32,
    [-0.0] * 32,
    [math.inf] + [1.0] * 31,
    [1.0] * 31 + [-math.inf],
    [1.0] * 9 + [math.nan] + [2.0] * 22,
    [7.0, -7.0, 6.9375, 5.0, 3.5, 2.5, 1.75, 1.25, 0.75, 0.25] + [0.125] * 22,      # ties, at the top of the scale
    [7.0625] + [0.5] * 31,                                                           # just above it
    [2.0 ** -20 * i for i in range(32)],
    [2.0 ** -24 * i for i in range(32)],                                             # half's smallest
    [60000.0, -65504.0] + [1000.0 * i for i in range(30)],
    [1e-3] * 31 + [1e3],
    [math.inf, -math.inf] + [math.nan] * 30,
]


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("rotated", [False, True])
def test_special_values_of_a_group(kind, rotated):
    """Plain and rotated appends (of a rotation that turns nothing) of groups at the edges of the format."""
    extra = [[2.0 ** -126 * i for i in range(32)], [3e38, -3e38] + [1e37] * 30, [2.0 ** 100] * 32] if kind == "bf16" else []
    groups = torch.tensor(SPECIAL + extra)
    rows = len(groups)
    x = torch.zeros(rows + 3, 6, 64)
    x[:rows, 2, :32], x[:rows, 2, 32:] = groups, groups.flip(0)
    x[:rows, 3, :32], x[:rows, 3, 32:] = groups.flip(0), groups * 0.5
    x[:rows, 4] = x[:rows, 2].flip(1)
    x[:rows, 5] = x[:rows, 3].flip(1)
    x = x.to(TYPES[kind])
    lens = [(rows, rows + 3)]
    with Cache(heads=2, dim=64, blocks=8, kind=kind) as c:
        if rotated:
            append_case(c, lens, 2, np.zeros(4), x=x, with_q=False)
            return
        tables = deal(c, lens)
        seqs, _ = seqs_of([t.cuda() for t in tables], lens)
        plan = c.plan(2, 1, rows)
        K.kv_attn_plan_set(plan, K.make_seqs(seqs), None)
        torch.cuda.synchronize()
        x_d = x.cuda()
        say("append of special groups", kind)
        K.kv_append_tokens(plan, 0, K.make_append_args(x_d[:, 2:4], x_d[:, 4:6], n_tokens=rows + 3), None)
        now, _ = c.now()
        for region in (0, 1):
            packed = rot.pack(*rot.mx4_of(x[:rows, 2 + 2 * region:4 + 2 * region].double()), c.row)
            packed[..., 34:] = c.rows(region, tables[0], np.arange(3, rows + 3))[..., 34:]
            c.put(region, tables[0], np.arange(3, rows + 3), packed)
        assert torch.equal(now, c.bytes)


def test_a_bad_block_id_skips_keys_and_values_only():
    for store in ("bf16", "e4m3", "mx4"):
        with Cache(heads=2, dim=64, blocks=8, cache=store) as c:
            table = torch.tensor([3, -1, 8, 5], dtype=torch.int32)
            t_d = table.cuda()
            plan, r = c.plan(4, 1, 64), c.rotation(frequencies(32))
            K.kv_attn_plan_set(plan, K.make_seqs([(t_d, 4, 64, 0, 64)]), None)
            x = new_tokens(64, 4, 2, 64, "bf16", 9)
            x_d = x.cuda()
            q, k, v = x_d.split([4, 2, 2], dim=1)
            out, read = torch.zeros_like(q), torch.full((1, 67, 2, 64), 7.0, dtype=torch.bfloat16, device="cuda")
            torch.cuda.synchronize()
            say("bad block ids", store)
            append = K.make_append_args(k, v, n_tokens=67, k_scale=c.k_scale, v_scale=c.v_scale)
            K.kv_append_rotated(plan, 0, r, K.make_rotate_args(q, out), append, None)
            assert K.kv_pool_get_error(c.handle) == K.KV_DEVERR_BLOCK_RANGE and K.kv_pool_get_error(c.handle) == 0
            now, _ = c.now()
            gone = [b for b in range(8) if b not in (3, 5)]
            assert torch.equal(now[:, gone], c.bytes[:, gone]) and not torch.equal(now[:, [3, 5]], c.bytes[:, [3, 5]])
            cs, sn = rot.turned_by(range(64), frequencies(32))
            want, size = rot.rotate(x[:64, :4].double(), cs, sn, False)
            check_between(out.cpu()[:64].double(), *rounded("bf16", want, size, 1.0), "q")
            if store == "mx4":
                K.kv_append_tokens(plan, 0, append, None)
                assert K.kv_pool_get_error(c.handle) == K.KV_DEVERR_BLOCK_RANGE
                now2, _ = c.now()
                assert torch.equal(now2[:, gone], c.bytes[:, gone])
            K.kv_read_tokens(plan, 0, 1, K.make_read_args(read, None, n_tokens=67), None)
            assert K.kv_pool_get_error(c.handle) == K.KV_DEVERR_BLOCK_RANGE
            assert (read[:, 16:48] == 7).all() and (read[:, 64:] == 7).all() and not (read[:, :16] == 7).all()
            before, _ = c.now()
            K.kv_rotate_cached(c.handle, r, KIND[store], K.make_shifts([(t_d, 4, 3, 60, 9)]), 0, 1, None)
            assert K.kv_pool_get_error(c.handle) == K.KV_DEVERR_BLOCK_RANGE
            now, _ = c.now()
            assert torch.equal(now[:, gone], before[:, gone]) and not torch.equal(now[0, [3, 5]], before[0, [3, 5]])


# ---- reads ------------------------------------------------------------------------------------

@pytest.mark.parametrize("kind,store", [("bf16", "bf16"), ("f16", "e4m3"), ("bf16", "e4m3"), ("f16", "mx4"), ("bf16", "mx4")])
@pytest.mark.parametrize("head_major", [False, True])
@pytest.mark.parametrize("heads,dim", [(2, 128), (3, 96), (1, 64)])
def test_reads_give_the_cached_values(kind, store, head_major, heads, dim):
    lens = [(21, 21), (0, 5), (1, 30), (17, 50), (1, 1)]
    with Cache(layers=3, heads=heads, dim=dim, page=16, blocks=12, head_major=head_major, kind=kind, cache=store, pad=16) as c:
        if store == "mx4":      # groups that are NaN, and the smallest and largest scales
            c.view(0)[:, ::3, 0, dim // 2] = 255
            c.view(1)[:, 1::3, 0, dim // 2] = 0
            c.view(2)[:, 2::5, 0, dim // 2] = 254
            c.upload()
        tables = deal(c, lens)
        seqs, rows = seqs_of([t.cuda() for t in tables], lens)
        plan = c.plan(heads, len(lens), rows)
        K.kv_attn_plan_set(plan, K.make_seqs(seqs), None)
        t = TYPES[kind]
        k = torch.full((2, rows + 2, heads + 1, dim), 7.0, dtype=t, device="cuda")
        v = torch.full((2, rows + 2, heads, dim), 7.0, dtype=t, device="cuda")
        torch.cuda.synchronize()
        say("read", kind, store, "head_major", head_major, "heads", heads, "dim", dim)
        K.kv_read_tokens(plan, 1, 3, K.make_read_args(k[:, :, :heads], v, n_tokens=rows + 2, k_scale=c.k_scale,
                                                      v_scale=c.v_scale), None)
        one = torch.full((rows, heads, dim), 7.0, dtype=t, device="cuda")
        K.kv_read_tokens(plan, 0, 1, K.make_read_args(one, None, n_tokens=rows, k_scale=c.k_scale), None)
        assert K.kv_pool_get_error(c.handle) == 0
        assert (k[:, rows:] == 7).all() and (v[:, rows:] == 7).all() and (k[:, :, heads:] == 7).all()
        for layer, kv, got, scale in ((1, 0, k[0], c.k_scale), (2, 0, k[1], c.k_scale), (1, 1, v[0], c.v_scale),
                                      (2, 1, v[1], c.v_scale), (0, 0, one, c.k_scale)):
            at = 0
            for table, (n_q, n_c) in zip(tables, lens):
                y = c.values(c.rows(2 * layer + kv, table, np.arange(n_c - n_q, n_c)))
                if store == "e4m3":     # one product in 32 bits (its rounding, then the type's)
                    y = y * float(np.float32(scale))
                    lo, hi = round_to(y - y.abs() * 2.0 ** -24, t), round_to(y + y.abs() * 2.0 ** -24, t)
                    check_between(got[at:at + n_q, :heads].cpu().double(), lo, hi, "read")
                else:
                    want = y.float().to(t)      # exact in 32 bits
                    g = got[at:at + n_q, :heads].cpu()
                    assert torch.equal(torch.isnan(g), torch.isnan(want))
                    assert torch.equal(torch.nan_to_num(g, nan=0.0), torch.nan_to_num(want, nan=0.0))
                at += n_q
        now, flat = c.now()
        assert torch.equal(flat, c.flat)


# ---- shifts -----------------------------------------------------------------------------------

def shift_case(c, spans, freq, adjacent=False, layers=(0, 1), seed=1):
    """spans: (t_begin, t_end, delta) of sequences of their own pages."""
    D = c.dim
    tables = deal(c, [(0, e) for _, e, _ in spans], seed)
    tables_d = [t.cuda() for t in tables]
    r = c.rotation(freq, adjacent, 3.0)     # an amplitude, which shifts leave out
    say("shift", c.cache, "dim", D, "pairs", len(freq), "adjacent", adjacent, "head_major", c.head_major, "page", c.page,
        "spans", spans[:6], len(spans))
    torch.cuda.synchronize()
    K.kv_rotate_cached(c.handle, r, KIND[c.cache], K.make_shifts(
        [(t, t.numel() - 2, b, e, d) for t, (b, e, d) in zip(tables_d, spans)]), *layers, None)
    assert K.kv_pool_get_error(c.handle) == 0
    now, flat = c.now()
    before = c.bytes.clone()
    for layer in range(*layers):
        for t, (b, e, d) in zip(tables, spans):
            places = np.arange(b, e)
            cs, sn = rot.turned_by([d], freq)
            old = c.rows(2 * layer, t, places)
            want, size = rot.rotate(c.values(old), cs.expand(len(places), -1), sn.expand(len(places), -1), adjacent)
            if c.cache == "mx4":
                packed = rot.pack(*rot.mx4_of(want), c.row)
                packed[..., D * 17 // 32:] = old[..., D * 17 // 32:]
                c.put(2 * layer, t, places, packed)
                continue
            keep, c.bytes = c.bytes, now
            rows = c.rows(2 * layer, t, places)
            c.bytes = keep
            check_between(c.values(rows), *rounded(c.cache, want, size, 1.0), "k")
            still = 2 * len(freq) * c.wide
            assert torch.equal(rows[..., still:], old[..., still:])
            c.put(2 * layer, t, places, rows)
    assert torch.equal(now, c.bytes), "wrote outside its rows, or other 4-bit values"
    assert torch.equal(flat[:, :, now[0, 0].numel():], c.flat[:, :, now[0, 0].numel():])
    return before


SPANS = [(0, 40, 5), (3, 4, -77777), (16, 32, 2 ** 31 - 1), (7, 7, 3), (31, 70, -2 ** 31), (0, 0, 1), (1, 18, 0)]


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("adjacent", [False, True], ids=["halves", "adjacent"])
@pytest.mark.parametrize("store", ["bf16", "f16", "e4m3", "mx4"])
def test_shift(shape, adjacent, store):
    _, heads, dim, pairs, page, head_major = shape
    with Cache(layers=3, heads=heads, dim=dim, page=page, blocks=200 if page < 16 else 40, head_major=head_major, kind="bf16", cache=store,
               pad=16) as c:
        shift_case(c, SPANS, frequencies(pairs), adjacent, (1, 3))


@pytest.mark.parametrize("store", ["bf16", "mx4"])
def test_shift_of_many_sequences(store):
    """More records than ride in the kernel arguments."""
    rng = np.random.default_rng(2)
    spans = [(int(b), int(b + n), int(d)) for b, n, d in zip(rng.integers(0, 5, 150), rng.integers(0, 12, 150),
                                                             rng.integers(-1000, 1000, 150))]
    with Cache(heads=2, dim=32, page=4, blocks=800, cache=store) as c:
        shift_case(c, spans, frequencies(16))


@pytest.mark.parametrize("store", ["bf16", "f16", "e4m3", "mx4"])
def test_a_shift_by_nothing_changes_nothing(store):
    with Cache(heads=2, dim=64, blocks=20, cache="mx4" if store == "mx4" else store, kind="bf16") as c:
        if store == "mx4":      # rows as an append leaves them
            x = torch.randn((2, 20, 16, 2, 64), generator=torch.Generator().manual_seed(4))
            c.bytes.copy_(rot.pack(*rot.mx4_of(x.double()), c.row))
            c.upload()
        before = shift_case(c, [(0, 100, 0), (3, 77, 0)], frequencies(32))
        now, _ = c.now()
        assert torch.equal(c.values(now), c.values(before))


def test_a_shifted_key_is_the_key_appended_there():
    """16-bit pools: turning by p and then by d is turning by p + d, to two roundings and their turn."""
    d = 4321
    with Cache(heads=2, dim=128, blocks=20, cache="f16", kind="f16") as c:
        freq = frequencies(64)
        table = torch.arange(8, dtype=torch.int32).cuda()
        plan, r = c.plan(2, 1, 100), c.rotation(freq)
        x = new_tokens(100, 2, 2, 128, "f16", 1).cuda()
        q, k, v = x.split([2, 2, 2], dim=1)
        append = K.make_append_args(k, v, n_tokens=103)
        K.kv_attn_plan_set(plan, K.make_seqs([(table, 8, 100, 0, 100)]), None)
        pos = (torch.arange(103, dtype=torch.int32) + d).cuda()
        got = [torch.zeros(100, 2, 128, dtype=torch.float16, device="cuda") for _ in range(2)]
        torch.cuda.synchronize()
        say("shift against append")
        K.kv_append_rotated(plan, 0, r, K.make_rotate_args(), append, None)
        K.kv_rotate_cached(c.handle, r, K.KV_TYPE_F16, K.make_shifts([(table, 8, 0, 100, d)]), 0, 1, None)
        K.kv_read_tokens(plan, 0, 1, K.make_read_args(got[0], None, n_tokens=100), None)
        K.kv_append_rotated(plan, 0, r, K.make_rotate_args(None, None, pos), append, None)
        K.kv_read_tokens(plan, 0, 1, K.make_read_args(got[1], None, n_tokens=100), None)
        torch.cuda.synchronize()
        a, b = (g.double().cpu() for g in got)
        _, size = rot.rotate(k[:100].double().cpu(), *rot.turned_by(range(100), freq), False)
        # half steps of the first key's two elements (each at most the pair's size), turned, and of either result
        assert ((a - b).abs() <= size * (4 * 2.0 ** -11 + 2.0 ** -19)).all()


# ---- refusals that need a plan ------------------------------------------------------------------

def test_refusals():
    with Cache(layers=2, heads=2, dim=64, blocks=8) as c, Cache(heads=2, dim=128, blocks=4, cache="bf16") as wide:
        plan, wide_plan = c.plan(4, 2, 32), wide.plan(4, 2, 32)
        r, too_wide = c.rotation(frequencies(32)), c.rotation(frequencies(64))
        table = torch.zeros(4, dtype=torch.int32, device="cuda")
        for p in (plan, wide_plan):
            K.kv_attn_plan_set(p, K.make_seqs([(table, 4, 8, 0, 8)]), None)
        x = torch.zeros(8, 8, 64, dtype=torch.bfloat16, device="cuda")
        q, k, v = x.split([4, 2, 2], dim=1)
        out = torch.zeros(8, 4, 64, dtype=torch.bfloat16, device="cuda")
        good_q, good = K.make_rotate_args(q, out), K.make_append_args(k, v, n_tokens=8)

        def refused(code, fn, *args):
            with pytest.raises(K.KvError) as e:
                fn(*args)
            assert e.value.code == code, e.value
        say("refusals")
        refused(K.KV_ERR_ARG, K.kv_append_rotated, plan, 2, r, good_q, good)
        refused(K.KV_ERR_ARG, K.kv_append_rotated, plan, -1, r, good_q, good)
        refused(K.KV_ERR_ARG, K.kv_append_rotated, plan, 0, too_wide, good_q, good)
        refused(K.KV_ERR_ARG, K.kv_append_rotated, plan, 0, None, good_q, good)
        refused(K.KV_ERR_ARG, K.kv_append_rotated, plan, 0, r, K.make_rotate_args(q, None), good)
        refused(K.KV_ERR_ARG, K.kv_append_rotated, plan, 0, r,
                K.make_rotate_args(q, out, out_strides=(256, 32)), good)                       # heads overlap
        refused(K.KV_ERR_ALIGN, K.kv_append_rotated, plan, 0, r, K.make_rotate_args(q, out, q_strides=(512, 60)), good)
        refused(K.KV_ERR_ALIGN, K.kv_append_rotated, plan, 0, r,
                K.make_rotate_args(q.data_ptr() + 8, out, q_strides=(512, 64)), good)
        refused(K.KV_ERR_ALIGN, K.kv_append_rotated, plan, 0, r, K.make_rotate_args(q, out, table.data_ptr() + 2), good)
        refused(K.KV_ERR_RANGE, K.kv_append_rotated, plan, 0, r, good_q, K.make_append_args(k, v, n_tokens=7))
        refused(K.KV_ERR_RANGE, K.kv_append_rotated, plan, 0, r,
                K.make_rotate_args(q, out, out_strides=(1 << 40, 64)), good)                   # past its allocation
        refused(K.KV_ERR_ARG, K.kv_append_rotated, plan, 0, r, good_q, K.make_append_args(k, v, n_tokens=-1))
        kk = torch.zeros(2, 8, 2, 64, dtype=torch.bfloat16, device="cuda")
        read = K.make_read_args(kk, kk, n_tokens=8)
        for a, b in ((0, 0), (1, 1), (-1, 1), (0, 3), (1, 0)):
            refused(K.KV_ERR_ARG, K.kv_read_tokens, plan, a, b, read)
        refused(K.KV_ERR_ARG, K.kv_read_tokens, plan, 0, 2, K.make_read_args(n_tokens=8))
        refused(K.KV_ERR_ARG, K.kv_read_tokens, plan, 0, 2, K.make_read_args(kk, None, n_tokens=8, k_strides=(512, 128, 64)))
        refused(K.KV_ERR_ARG, K.kv_read_tokens, plan, 0, 2, K.make_read_args(kk, None, n_tokens=8, k_strides=(1024, 64, 64)))
        refused(K.KV_ERR_ALIGN, K.kv_read_tokens, plan, 0, 2, K.make_read_args(kk, None, n_tokens=8, k_strides=(1028, 128, 64)))
        refused(K.KV_ERR_RANGE, K.kv_read_tokens, plan, 0, 2, K.make_read_args(kk, None, n_tokens=8, k_strides=(1 << 40, 128, 64)))
        refused(K.KV_ERR_RANGE, K.kv_read_tokens, plan, 0, 2, K.make_read_args(kk, None, n_tokens=7))
        ok = (table, 4, 0, 8, 1)
        for code, kind, spans, layers in (
                (K.KV_ERR_ARG, K.KV_TYPE_BF16, [ok], (0, 1)), (K.KV_ERR_ARG, 4, [ok], (0, 1)),
                (K.KV_ERR_ARG, K.KV_TYPE_MX4, [ok], (0, 3)), (K.KV_ERR_ARG, K.KV_TYPE_MX4, [ok], (1, 1)),
                (K.KV_ERR_ARG, K.KV_TYPE_MX4, [(table, 4, -1, 8, 1)], (0, 1)),
                (K.KV_ERR_ARG, K.KV_TYPE_MX4, [(table, 4, 9, 8, 1)], (0, 1)),
                (K.KV_ERR_ARG, K.KV_TYPE_MX4, [ok, (None, 4, 0, 8, 1)], (0, 1)),
                (K.KV_ERR_ALIGN, K.KV_TYPE_MX4, [(table.data_ptr() + 2, 4, 0, 8, 1)], (0, 1)),
                (K.KV_ERR_RANGE, K.KV_TYPE_MX4, [(table, 4, 0, 65, 1)], (0, 1)),
                (K.KV_ERR_RANGE, K.KV_TYPE_MX4, [(table, 1 << 30, 0, 64, 1)], (0, 1)),
                (K.KV_ERR_RANGE, K.KV_TYPE_MX4, [(table, 1 << 30, 0, 1 << 31, 1)], (0, 1)),
                (K.KV_ERR_ARG, K.KV_TYPE_MX4, [ok] * (K.KV_MAX_SHIFTS + 1), (0, 1))):
            refused(code, K.kv_rotate_cached, c.handle, r, kind, K.make_shifts(spans), *layers)
        refused(K.KV_ERR_ARG, K.kv_rotate_cached, c.handle, too_wide, K.KV_TYPE_MX4, K.make_shifts([ok]), 0, 1)
        K.kv_attn_plan_set(plan, K.make_seqs([(table, 4, 3, 0, 8)]), None)      # more new tokens than cached ones
        refused(K.KV_ERR_ARG, K.kv_append_rotated, plan, 0, r, good_q, good)
        refused(K.KV_ERR_ARG, K.kv_read_tokens, plan, 0, 2, read)
        K.kv_attn_plan_set(plan, K.make_seqs([]), None)
        K.kv_append_rotated(plan, 0, r, good_q, K.make_append_args(k, v, n_tokens=0), None)
        K.kv_append_rotated(plan, 0, r, good_q, good, None)
        K.kv_read_tokens(plan, 0, 2, read, None)
        K.kv_rotate_cached(c.handle, r, K.KV_TYPE_MX4, K.make_shifts([]), 0, 2)
        now, flat = c.now()
        assert torch.equal(flat, c.flat) and (out == 0).all() and (kk == 0).all()
