"""Attention over 4-bit pools on the GPU, element by element against 64 bits with the bounds derived in
tests/paged_reference.py: the cached values are what the rows stand for, so the bounds are those of 16-bit pools."""
from __future__ import annotations

import math

import numpy as np
import pytest
import torch

import paged_reference as ref
from paged_layout_transfer_amd import kvxfer as K
from rotated_harness import TYPES, Cache, deal, say, scale_of, seqs_of

pytestmark = pytest.mark.gpu


def attend_case(cache, lens, heads_q, *, window=0, full=False, softcap=0.0, slopes=False, seed=3, scale=None, layer=0, label="",
                plan=None):
    dim, scale = cache.dim, scale if scale is not None else scale_of(cache.dim)
    tables = deal(cache, lens)
    tables_d = [t.cuda() for t in tables]
    seqs, rows = seqs_of(tables_d, lens)
    gen = torch.Generator().manual_seed(seed)
    q_h = (torch.randn((rows + 3, heads_q + 2, dim), generator=gen) * 1.2).to(TYPES[cache.kind])
    q_d = q_h.cuda()
    wide = torch.full((rows + 3, heads_q * dim + 8), 7.0, dtype=TYPES[cache.kind], device="cuda")
    out = wide[:, :heads_q * dim].view(rows + 3, heads_q, dim)
    lse = torch.full((rows + 3, heads_q), 7.0, device="cuda")
    sl = (2.0 ** -torch.arange(1, heads_q + 1).float()) if slopes else None
    plan = plan or cache.plan(heads_q, max(1, len(lens)), max(1, rows), window, full)
    K.kv_attn_plan_set(plan, K.make_seqs(seqs), torch.cuda.current_stream())
    sl_d = sl.cuda() if slopes else None
    torch.cuda.synchronize()
    say("attend", label, "lens", lens[:8], "heads", heads_q, cache.heads, "dim", dim, "row", cache.row, "page", cache.page,
        cache.kind, "head_major", cache.head_major, "window", window, "full", full, "cap", softcap, "slopes", slopes)
    K.kv_attend(plan, layer, K.make_attend_args(q_d[:, :heads_q], out, lse, n_tokens=rows + 3, scale=scale, softcap=softcap,
                                                alibi_slopes=sl_d), torch.cuda.current_stream())
    torch.cuda.synchronize()
    got, got_lse = out.cpu().double(), lse.cpu().double()
    assert (wide[:, heads_q * dim:] == 7).all() and (out[rows:] == 7).all() and (lse[rows:] == 7).all(), \
        "wrote outside its rows"
    for t, (_, _, n, at, q_len, prefix) in zip(tables, seqs):
        # as the kernel reads them: rounded to the queries' type
        k, v = (cache.values(cache.rows(2 * layer + i, t, np.arange(n))).float().to(TYPES[cache.kind]).double() for i in (0, 1))
        want, z, tol, tol_z = ref.attend(q_h[at:at + q_len, :heads_q].double(), k, v, scale=scale, softcap=softcap, slopes=sl,
                                         window=window, prefix=prefix, full=full, kind=cache.kind)
        g, gz = got[at:at + q_len], got_lse[at:at + q_len]
        fin = torch.isfinite(want)
        assert torch.equal(torch.isnan(g), torch.isnan(want)), "NaN"
        # Rows of 4-bit values hold exact zeros, so a column's result can be all weights of almost nothing.  Weights below
        # the smallest normal number 2^-126 are zero (exponentials and products flush them; the largest is 1 or
        # more), and so is such a result: 2^-126 of each seen value and of the result, at most.
        if n:
            seen = ref.visible(q_len, n, window, prefix, full).double()
            va = torch.nan_to_num(v.abs(), nan=0.0).repeat_interleave(heads_q // cache.heads, 1)
            tol = tol + 2.0 ** -126 * (1 + torch.einsum("qn,nhd->qhd", seen, va))
        bad = (g - want).abs()[fin] > tol[fin]
        assert not bad.any(), "out: %d of %d off, worst %g" % (bad.sum(), bad.numel(), (g - want).abs()[fin].max())
        some = torch.isfinite(z)
        assert torch.equal(torch.isnan(gz), torch.isnan(z))
        assert torch.equal(gz[~some & ~torch.isnan(z)], z[~some & ~torch.isnan(z)])
        assert ((gz - z).abs()[some] <= tol_z[some]).all(), "lse: worst %g" % (gz - z).abs()[some].max()
    assert K.kv_pool_get_error(cache.handle) == 0
    return out, lse


FEW = [(1, 1), (1, 700), (2, 33), (0, 50), (3, 3), (1, 64), (1, 65), (1, 128), (2, 1000)]
MANY = [(70, 70), (1, 300), (40, 500), (130, 131), (0, 0), (64, 192), (33, 1000)]


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("dim", [64, 128, 256, 32, 96, 160, 192, 224])
@pytest.mark.parametrize("head_major", [False, True])
def test_types_dims_layouts(kind, dim, head_major):
    for lens, page in ((FEW, 16), (MANY, 24)):
        with Cache(heads=2, dim=dim, page=page, blocks=200, head_major=head_major, kind=kind, pad=32) as c:
            attend_case(c, lens, 8)


@pytest.mark.parametrize("page", [1, 3, 16, 64, 100])
@pytest.mark.parametrize("heads,heads_q", [(1, 1), (1, 16), (3, 3), (2, 10), (1, 40), (4, 28)])
def test_pages_and_groups(page, heads, heads_q):
    lens = [(1, 130), (5, 77), (2, 2), (19, 40), (1, 1), (60, 250)]
    with Cache(heads=heads, dim=64, page=page, blocks=600 // page + 20) as c:
        attend_case(c, lens, heads_q)


@pytest.mark.parametrize("heads,dim,row", [(4, 128, 68), (2, 128, 72), (1, 128, 80), (4, 64, 36), (4, 64, 48), (2, 256, 136)])
@pytest.mark.parametrize("head_major", [False, True])
def test_row_bytes(heads, dim, row, head_major):
    """Rows at every multiple of four bytes, with and without bytes to spare."""
    for lens in (FEW, MANY):
        with Cache(heads=heads, dim=dim, blocks=200, row=row, head_major=head_major) as c:
            attend_case(c, lens, heads * 2)


VARIANTS = [
    dict(window=1), dict(window=2**31 - 1), dict(window=7), dict(window=64), dict(window=200), dict(full=True), dict(softcap=5.0),
    dict(softcap=100.0), dict(slopes=True), dict(window=50, softcap=20.0, slopes=True), dict(full=True, slopes=True, softcap=3.0),
    dict(scale=0.0), dict(scale=-0.2), dict(scale=4.0),
]


@pytest.mark.parametrize("variant", VARIANTS, ids=str)
@pytest.mark.parametrize("kind,dim", [("f16", 64), ("bf16", 128), ("bf16", 256)])
def test_variants(variant, kind, dim):
    lens = [(1, 400, 0), (1, 400, 30), (3, 90, 90), (100, 300, 17), (60, 60, 200), (5, 2, 1), (4, 0), (90, 20, 0),
            (1, 129, 65), (80, 700, 64)]
    with Cache(heads=2, dim=dim, page=16, blocks=200, kind=kind) as c:
        attend_case(c, lens, 6, **variant)


@pytest.mark.parametrize("full", [False, True])
def test_every_query_sees_the_keys_its_masks_leave(full):
    """Queries of zeros weigh what they see alike, so exp(lse) counts the keys."""
    rng = np.random.default_rng(3)
    with Cache(heads=1, dim=64, page=16, blocks=200) as c:
        for window in (0,) if full else (0, 1, 2, 31, 33, 64, 100):
            lens = [(1, n, 0) for n in (1, 31, 32, 33, 63, 64, 65, 100, 390)] + [(20, 100, 3), (2, 400, 200), (150, 300, 40)]
            lens += [(int(q), int(q + rng.integers(0, 90)), int(rng.integers(0, 90))) for q in rng.integers(1, 40, 6)]
            tables = [t.cuda() for t in deal(c, lens)]
            seqs, rows = seqs_of(tables, lens)
            plan = c.plan(2, len(lens), rows, window=window, full=full)
            q, lse = torch.zeros(rows, 2, 64, device="cuda").bfloat16(), torch.zeros(rows, 2, device="cuda")
            K.kv_attn_plan_set(plan, K.make_seqs(seqs))
            say("counted keys, window", window, "full", full)
            K.kv_attend(plan, 0, K.make_attend_args(q, torch.empty_like(q), lse, n_tokens=rows, scale=0.1))
            want = torch.cat([ref.visible(a, n, window, p, full).sum(-1) for a, n, p in lens])
            assert torch.equal(lse.exp().round().long().cpu(), want[:, None].expand(-1, 2))


@pytest.mark.parametrize("kind,dim", [("bf16", 128), ("f16", 64), ("bf16", 256)])
def test_split_over_the_keys(kind, dim):
    with Cache(heads=1, dim=dim, page=16, blocks=1400, kind=kind) as c:
        attend_case(c, [(1, 12001), (1, 3000), (1, 90)], 4)
        attend_case(c, [(70, 9000), (40, 5001)], 2)
        attend_case(c, [(1, 12001, 700), (30, 3000, 20)], 4, window=2000)


@pytest.mark.parametrize("kind,dim", [("bf16", 64), ("bf16", 128), ("f16", 96), ("bf16", 256)])
def test_enough_work_for_a_head_a_wave(kind, dim):
    """Token-major pages, heads a multiple of four, many or long sequences: cut and whole pieces."""
    with Cache(heads=4, dim=dim, page=16, blocks=6200, kind=kind) as c:
        attend_case(c, [(1, 60000), (1, 23000), (3, 9000), (1, 130), (0, 5), (2, 1)], 8)
        attend_case(c, [(1 + i % 3, 240 + i) for i in range(260)], 8, window=200 if dim == 64 else 0)


@pytest.mark.parametrize("n", [6, 34], ids=["half_pieces", "whole_pieces"])
@pytest.mark.parametrize("dim,kind", [(64, "f16"), (128, "bf16")])
def test_pieces_of_128_and_256_rows(n, dim, kind):
    lens = [(66 + i % 3, 66 + 7 * i) for i in range(1, n)] + [(66, 66)]
    with Cache(heads=8, dim=dim, page=16, blocks=40 + sum(x[1] // 16 + 1 for x in lens), kind=kind) as c:
        attend_case(c, lens, 32, label="pieces")
        attend_case(c, lens, 32, window=50, label="pieces")


@pytest.mark.parametrize("lens", [[(1, 700), (2, 300)], [(50, 400), (70, 100)]], ids=["few", "many"])
@pytest.mark.parametrize("kind,dim", [("bf16", 64), ("f16", 128), ("bf16", 256)])
def test_what_a_query_does_not_see_does_not_reach_it(lens, kind, dim):
    """Rows of NaN in unused pages, behind the last token, outside the window, and in the newest token (which
    earlier queries of the call do not see)."""
    for window in (0, 100):
        with Cache(heads=2, dim=dim, page=16, blocks=150, kind=kind) as c:
            keep = torch.zeros(c.blocks, c.page, dtype=torch.bool)
            for t, (q, n) in zip(deal(c, lens), lens):
                lo = max(0, n - q - window + 1) if window else 0
                j = torch.arange(lo, n)
                keep[t.long()[j // 16], j % 16] = True
                keep[int(t[(n - 1) // 16]), (n - 1) % 16] = False
            c.bytes[:, ~keep] = 0xff
            c.upload()
            attend_case(c, lens, 4, window=window, label="poison")


@pytest.mark.parametrize("lens", [[(1, 20), (3, 300)], [(50, 60), (70, 400)]], ids=["few", "many"])
@pytest.mark.parametrize("window", [0, 40])
def test_nan_groups_reach_the_queries_that_see_them(lens, window):
    with Cache(heads=2, dim=96, page=16, blocks=60) as c:
        for t, (q, n) in zip(deal(c, lens), lens):
            for j, head, group in ((0, 0, 0), (n // 2, 1, 2), (n - 1, 1, 1)):     # values of single tokens
                c.view(1)[int(t[j // 16]), j % 16, head, 48 + group] = 255
        c.upload()
        attend_case(c, lens, 4, window=window, label="NaN groups")
    for long in ([(1, 257), (1, 1), (2, 1500)], [(70, 1025)]):
        with Cache(heads=2, dim=64, page=16, blocks=150) as c:
            for t, (q, n) in zip(deal(c, long), long):
                c.view(0)[int(t[(n - 1) // 16]), (n - 1) % 16, 1, 33] = 255       # a key alone in its stretch
            c.upload()
            attend_case(c, long, 4, window=1 if len(long) > 1 else 0, label="NaN key")


@pytest.mark.parametrize("kind,gain", [("bf16", 2.0 ** 40), ("bf16", 2.0 ** -60), ("f16", 2.0 ** 9), ("f16", 2.0 ** -18)])
def test_scales_over_the_types_range(kind, gain):
    """Small and large scale bytes; halves that widen to subnormal numbers."""
    with Cache(heads=2, dim=64, page=16, blocks=150, kind=kind, gain=gain) as c:
        attend_case(c, [(1, 700), (70, 300)], 4, scale=0.1 / gain, label="gain")


@pytest.mark.parametrize("lens", [[(1, 300), (1, 200)], [(40, 300), (40, 200)]], ids=["few", "many"])
def test_a_bad_block_id_is_reported_and_stays_in_its_sequence(lens):
    with Cache(heads=2, dim=64, page=16, blocks=64) as c:
        good, _ = attend_case(c, lens, 4)
        tables_d = [t.cuda() for t in deal(c, lens)]
        tables_d[0][3] = 64
        seqs, rows = seqs_of(tables_d, lens)
        plan = c.plan(4, 2, rows)
        gen = torch.Generator().manual_seed(3)
        q = (torch.randn((rows + 3, 6, 64), generator=gen) * 1.2).bfloat16().cuda()
        out = torch.empty(rows, 4, 64, dtype=torch.bfloat16, device="cuda")
        K.kv_attn_plan_set(plan, K.make_seqs(seqs))
        say("bad block id", lens)
        K.kv_attend(plan, 0, K.make_attend_args(q[:, :4], out, n_tokens=rows, scale=0.125))
        assert K.kv_pool_get_error(c.handle) == K.KV_DEVERR_BLOCK_RANGE
        first = seqs[1][3]
        assert torch.equal(out[first:], good[first:rows])


def test_regions_past_32_bits_of_bytes():
    """A block id whose page lies over 4 GiB into its region, in both kernels."""
    H, D, page, row = 8, 128, 16, 68
    stride = page * H * row
    blocks = (5 << 30) // stride
    big = torch.zeros(2, blocks * stride, dtype=torch.uint8, device="cuda")
    gen = torch.Generator().manual_seed(2)
    import rotated_reference as rot
    pages = rot.random_rows((2, 8, page, H), D, row, gen)
    ids = torch.tensor([blocks - 1 - 7 * i for i in range(8)])
    for i in range(2):
        big[i].view(blocks, page, H, row)[ids.cuda()] = pages[i].cuda()
    pool = K.kv_pool_create(K.make_pool_desc(1, 2, H, row, 1, page, blocks, stride, [big[0], big[1]]))
    plan = K.kv_attn_plan_create(pool, K.make_attn_desc(16, K.KV_TYPE_BF16, K.KV_TYPE_MX4, 1, 40))
    table = ids.int().cuda()
    q = torch.randn(40, 16, D, generator=gen).bfloat16()
    k, v = (rot.unpack(pages[i].reshape(-1, H, row), D) for i in (0, 1))
    try:
        for new in (1, 40):
            out = torch.zeros(new, 16, D, dtype=torch.bfloat16, device="cuda")
            K.kv_attn_plan_set(plan, K.make_seqs([(table, 8, 125, 0, new)]), None)
            q_d = q[:new].cuda()
            torch.cuda.synchronize()
            say("far pages, new tokens", new)
            K.kv_attend(plan, 0, K.make_attend_args(q_d, out, n_tokens=new, scale=0.1), None)
            torch.cuda.synchronize()
            want, _, tol, _ = ref.attend(q[:new].double(), k[:125], v[:125], scale=0.1)
            assert ((out.cpu().double() - want).abs() <= tol).all() and K.kv_pool_get_error(pool) == 0
    finally:
        torch.cuda.synchronize()
        K.kv_attn_plan_destroy(plan)
        K.kv_pool_destroy(pool)
