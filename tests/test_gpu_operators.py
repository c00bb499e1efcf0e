"""The operators on a paged cache on the GPU, against plain 64-bit implementations
(tests/paged_reference.py): page copies, table rewriting, append, attention, and a run of
them together.  Every case is printed before its first launch."""
from __future__ import annotations

import ctypes
import math

import numpy as np
import pytest
import torch

import paged_reference as ref
from paged_layout_transfer_amd import kvxfer as K

pytestmark = pytest.mark.gpu

KIND = {"f16": K.KV_TYPE_F16, "bf16": K.KV_TYPE_BF16, "e4m3": K.KV_TYPE_E4M3}


def say(*what):
    print("[gpu]", *what, flush=True)


def words(t):
    """A tensor's bits, for exact comparison."""
    return t.contiguous().view(torch.uint8)


class Cache:
    """A pool of random pages on the GPU, its host copy, and a plan."""

    def __init__(self, *, layers=1, heads=2, dim=64, page=16, blocks=64, head_major=False, kind="bf16", cache=None,
                 seed=0, pad=0):
        self.cache = cache or kind
        self.kind, self.heads, self.dim, self.page, self.head_major = kind, heads, dim, page, head_major
        self.layers, self.blocks = layers, blocks
        gen = torch.Generator().manual_seed(seed)
        wide = 1 if self.cache == "e4m3" else 2
        self.k_scale, self.v_scale = (0.037, 0.021) if self.cache == "e4m3" else (1.0, 1.0)
        inner = (heads, page, dim) if head_major else (page, heads, dim)
        x = torch.randn((2 * layers, blocks) + inner, generator=gen)
        if self.cache == "e4m3":
            x = (x * 25).clamp(-448, 448)
        self.host = x.to(ref.TYPES[self.cache])
        # `pad` bytes between blocks, which nothing may touch
        self.stride = page * heads * dim * wide + pad
        self.flat = torch.full((2 * layers, blocks, self.stride), 0xA5, dtype=torch.uint8)
        self.flat[:, :, :self.stride - pad] = words(self.host).view(2 * layers, blocks, -1)
        self.dev = self.flat.cuda()
        self.handle = K.kv_pool_create(K.make_pool_desc(
            layers, 2, heads, dim, wide, page, blocks, self.stride,
            [self.dev.data_ptr() + i * self.dev.stride(0) for i in range(2 * layers)],
            K.KV_PAGE_HEAD_MAJOR if head_major else K.KV_PAGE_TOKEN_MAJOR))
        self.plans = []

    def upload(self):
        """The host copy's pages to the device, after a test changed it."""
        n = self.page * self.heads * self.dim * self.host.element_size()
        self.flat[:, :, :n] = words(self.host).view(2 * self.layers, self.blocks, -1)
        self.dev.copy_(self.flat)

    def plan(self, heads_q, max_seqs, max_tokens, window=0, full=False):
        h = K.kv_attn_plan_create(self.handle, K.make_attn_desc(
            heads_q, KIND[self.kind], KIND[self.cache], max_seqs, max_tokens, window, K.KV_ATTN_FULL if full else 0))
        self.plans.append(h)
        return h

    def region(self, layer, kv):
        return self.host[2 * layer + kv]

    def close(self):
        torch.cuda.synchronize()
        for h in self.plans:
            K.kv_attn_plan_destroy(h)
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


def seqs_of(tables_d, lens):
    out, at = [], 0
    for t, (q, n, *prefix) in zip(tables_d, lens):
        out.append((t, t.numel(), n, at, q, prefix[0] if prefix else 0))
        at += q
    return out, at


def attend_case(cache, lens, heads_q, *, window=0, full=False, softcap=0.0, slopes=False, seed=3, scale=None,
                layer=0, label=""):
    """Attention of random queries over the cache, compared element by element."""
    dim, scale = cache.dim, scale if scale is not None else 1 / math.sqrt(cache.dim)
    tables = deal(cache, lens)
    tables_d = [t.cuda() for t in tables]
    seqs, rows = seqs_of(tables_d, lens)
    gen = torch.Generator().manual_seed(seed)
    # queries inside a wider row, results with a gap between tokens, spare rows behind
    q_h = (torch.randn((rows + 3, heads_q + 2, dim), generator=gen) * 1.2).to(ref.TYPES[cache.kind])
    q_d = q_h.cuda()
    wide = torch.full((rows + 3, heads_q * dim + 8), 7.0, dtype=ref.TYPES[cache.kind], device="cuda")
    out = wide[:, :heads_q * dim].view(rows + 3, heads_q, dim)
    lse = torch.full((rows + 3, heads_q), 7.0, device="cuda")
    sl = (2.0 ** -torch.arange(1, heads_q + 1).float()) if slopes else None
    plan = cache.plan(heads_q, max(1, len(lens)), max(1, rows), window, full)
    K.kv_attn_plan_set(plan, K.make_seqs(seqs), torch.cuda.current_stream())
    sl_d = sl.cuda() if slopes else None
    args = K.make_attend_args(q_d[:, :heads_q], out, lse, n_tokens=rows + 3, scale=scale, softcap=softcap,
                              alibi_slopes=sl_d, k_scale=cache.k_scale, v_scale=cache.v_scale)
    torch.cuda.synchronize()
    say("attend", label, "lens", lens[:8], "heads", heads_q, cache.heads, "dim", dim, "page", cache.page,
        cache.kind, cache.cache, "window", window, "full", full, "cap", softcap, "slopes", slopes)
    K.kv_attend(plan, layer, args, torch.cuda.current_stream())
    torch.cuda.synchronize()
    got, got_lse = out.cpu().double(), lse.cpu().double()
    assert (wide[:, heads_q * dim:] == 7).all() and (out[rows:] == 7).all() and (lse[rows:] == 7).all(), \
        "wrote outside its rows"
    for t, (_, n_t, n, at, q_len, prefix) in zip(tables, seqs):
        k, v = (ref.cache_of(cache.region(layer, i), cache.head_major, t, n) for i in (0, 1))
        want, z, tol, tol_z = ref.attend(
            q_h[at:at + q_len, :heads_q].double(), k, v, scale=scale, softcap=softcap, slopes=sl, window=window,
            prefix=prefix, full=full, k_scale=float(np.float32(cache.k_scale)),
            v_scale=float(np.float32(cache.v_scale)), kind=cache.kind)
        g, gz = got[at:at + q_len], got_lse[at:at + q_len]
        fin = torch.isfinite(want)
        assert torch.equal(torch.isnan(g), torch.isnan(want)) and torch.equal(g[~fin & ~torch.isnan(want)],
                                                                              want[~fin & ~torch.isnan(want)])
        bad = (g - want).abs()[fin] > tol[fin]
        assert not bad.any(), "out: %d of %d off, worst %g of %g allowed" % (
            bad.sum(), bad.numel(), (g - want).abs()[fin].max(), tol[fin][(g - want).abs()[fin].argmax()])
        some = torch.isfinite(z)
        assert torch.equal(torch.isnan(gz), torch.isnan(z))
        assert torch.equal(gz[~some & ~torch.isnan(z)], z[~some & ~torch.isnan(z)])
        assert ((gz - z).abs()[some] <= tol_z[some]).all(), "lse: worst %g" % (gz - z).abs()[some].max()
    return plan, args, out, lse, (tables_d, q_d, sl_d)      # what the plan and the arguments point at


FEW = [(1, 1), (1, 700), (2, 33), (0, 50), (3, 3), (1, 64), (1, 65), (1, 128), (2, 1000)]
MANY = [(70, 70), (1, 300), (40, 500), (130, 131), (0, 0), (64, 192), (33, 1000)]
TYPES = [("bf16", "bf16"), ("f16", "f16"), ("bf16", "e4m3"), ("f16", "e4m3")]


@pytest.mark.parametrize("kind,held", TYPES)
@pytest.mark.parametrize("dim", [64, 128, 256, 80, 16])
@pytest.mark.parametrize("head_major", [False, True])
def test_attention_types_dims_layouts(kind, held, dim, head_major):
    for lens, page in ((FEW, 16), (MANY, 24)):
        with Cache(heads=2, dim=dim, page=page, blocks=200, head_major=head_major, kind=kind, cache=held, pad=32) as c:
            attend_case(c, lens, 8)


@pytest.mark.parametrize("page", [1, 3, 16, 64, 100])
@pytest.mark.parametrize("heads,heads_q", [(1, 1), (1, 16), (3, 3), (2, 10), (1, 40), (4, 28)])
def test_attention_pages_and_groups(page, heads, heads_q):
    lens = [(1, 130), (5, 77), (2, 2), (19, 40), (1, 1), (60, 250)]
    with Cache(heads=heads, dim=64, page=page, blocks=600 // page + 20, kind="bf16") as c:
        attend_case(c, lens, heads_q)


VARIANTS = [
    dict(window=1), dict(window=2**31 - 1), dict(window=7), dict(window=64), dict(window=200), dict(full=True), dict(softcap=5.0),
    dict(slopes=True), dict(window=50, softcap=20.0, slopes=True), dict(full=True, slopes=True, softcap=3.0),
    dict(scale=0.0), dict(scale=-0.2), dict(scale=4.0),
]


@pytest.mark.parametrize("variant", VARIANTS, ids=str)
@pytest.mark.parametrize("held", ["f16", "e4m3"])
def test_attention_variants(variant, held):
    lens = [(1, 400, 0), (1, 400, 30), (3, 90, 90), (100, 300, 17), (60, 60, 200), (5, 2, 1), (4, 0), (90, 20, 0),
            (1, 129, 65), (80, 700, 64)]
    with Cache(heads=2, dim=64, page=16, blocks=200, kind="f16", cache=held) as c:
        attend_case(c, lens, 6, **variant)


@pytest.mark.parametrize("softcap", [0.0, 20.0])
@pytest.mark.parametrize("full", [False, True])
def test_every_query_sees_the_keys_its_masks_leave(softcap, full):
    """Queries of zeros weigh what they see alike, so exp(lse) counts the keys."""
    rng = np.random.default_rng(3)
    with Cache(heads=1, dim=64, page=16, blocks=200, kind="bf16") as c:
        for window in (0,) if full else (0, 1, 2, 5, 10, 16, 31, 33, 50, 64, 100):
            lens = [(1, n, 0) for n in (1, 31, 32, 33, 64, 100, 390)] + [(20, 100, 3), (2, 400, 200), (150, 300, 40)]
            lens += [(int(q), int(q + rng.integers(0, 90)), int(rng.integers(0, 90))) for q in rng.integers(1, 40, 6)]
            tables = [t.cuda() for t in deal(c, lens)]
            seqs, rows = seqs_of(tables, lens)
            plan = c.plan(2, len(lens), rows, window=window, full=full)
            q, lse = torch.zeros(rows, 2, 64, device="cuda").bfloat16(), torch.zeros(rows, 2, device="cuda")
            K.kv_attn_plan_set(plan, K.make_seqs(seqs))
            say("counted keys, window", window, "cap", softcap, "full", full)
            K.kv_attend(plan, 0, K.make_attend_args(q, torch.empty_like(q), lse, n_tokens=rows, scale=0.1,
                                                    softcap=softcap))
            want = torch.cat([ref.visible(a, n, window, p, full).sum(-1) for a, n, p in lens])
            assert torch.equal(lse.exp().round().long().cpu(), want[:, None].expand(-1, 2))


@pytest.mark.parametrize("kind,held,dim", [("bf16", "bf16", 128), ("f16", "e4m3", 64), ("bf16", "bf16", 256)])
def test_attention_split_over_the_keys(kind, held, dim):
    with Cache(heads=1, dim=dim, page=16, blocks=1400, kind=kind, cache=held) as c:
        attend_case(c, [(1, 12001), (1, 3000), (1, 90)], 4)
        attend_case(c, [(70, 9000), (40, 5001)], 2)
        attend_case(c, [(1, 12001, 700), (30, 3000, 20)], 4, window=2000)


@pytest.mark.parametrize("kind,held,dim", [("bf16", "bf16", 64), ("f16", "e4m3", 64), ("bf16", "bf16", 128),
                                           ("f16", "f16", 80), ("bf16", "bf16", 256)])
def test_attention_of_enough_work_for_a_head_a_wave(kind, held, dim):
    """Token-major pages, heads a multiple of four, many or long sequences: cut and whole pieces."""
    with Cache(heads=4, dim=dim, page=16, blocks=6200, kind=kind, cache=held) as c:
        attend_case(c, [(1, 60000), (1, 23000), (3, 9000), (1, 130), (0, 5), (2, 1)], 8)
        attend_case(c, [(1 + i % 3, 240 + i) for i in range(260)], 8, window=200 if dim == 64 else 0)


@pytest.mark.parametrize("lens", [[(1, 700), (2, 300)], [(50, 400), (70, 100)]], ids=["few", "many"])
@pytest.mark.parametrize("held", ["bf16", "e4m3"])
@pytest.mark.parametrize("poison", [math.nan, math.inf])
def test_what_a_query_does_not_see_does_not_reach_it(lens, held, poison):
    """NaN or infinities in unused pages, behind the last token, outside the window, and in
    the newest token (which earlier queries of the call do not see)."""
    if held == "e4m3" and poison == math.inf:
        pytest.skip("e4m3 has no infinity")
    for window in (0, 100):
        with Cache(heads=2, dim=64, page=16, blocks=150, kind="bf16", cache=held) as c:
            tables = deal(c, lens)
            view = c.host.transpose(2, 3) if c.head_major else c.host
            keep = torch.zeros(c.blocks, c.page, dtype=torch.bool)
            for t, (q, n) in zip(tables, lens):
                lo = max(0, n - q - window + 1) if window else 0
                j = torch.arange(lo, n)
                keep[t.long()[j // 16], j % 16] = True
                keep[int(t[(n - 1) // 16]), (n - 1) % 16] = False
            bits = view.view(torch.uint8) if held == "e4m3" else view.view(torch.int16)
            bits[:, ~keep] = torch.tensor([poison]).to(view.dtype).view(bits.dtype)
            c.upload()
            attend_case(c, lens, 4, window=window, label="poison %s" % poison)


@pytest.mark.parametrize("lens", [[(1, 20), (3, 300)], [(50, 60), (70, 400)]], ids=["few", "many"])
@pytest.mark.parametrize("window", [0, 40])
def test_infinite_and_nan_values_reach_the_queries_that_see_them(lens, window):
    """Values (not keys) of single cached tokens: the first one, one in the middle and the
    newest, an infinity of either sign, both in one column, NaN."""
    with Cache(heads=2, dim=64, page=16, blocks=60, kind="bf16") as c:
        for t, (q, n) in zip(deal(c, lens), lens):
            at = lambda j: c.host[1][int(t[j // 16]), j % 16]       # noqa: E731
            at(0)[0, 3] = math.inf
            at(n // 2)[0, 5] = -math.inf
            at(n - 1)[1, 7] = math.nan
            at(n - 1)[0, 9] = math.inf
            at(n - 2)[0, 9] = -math.inf
            at(n - 2)[1, 11] = math.inf
        c.upload()
        attend_case(c, lens, 4, window=window, label="infinite values")


@pytest.mark.parametrize("n", [6, 34], ids=["half_pieces", "whole_pieces"])
@pytest.mark.parametrize("dim,kind,cache", [(64, "f16", "f16"), (128, "bf16", "e4m3")])
def test_pieces_of_128_and_256_rows(n, dim, kind, cache):
    """A step that does not fill the chip is planned in pieces of half the rows."""
    lens = [(66 + i % 3, 66 + 7 * i) for i in range(1, n)] + [(66, 66)]
    with Cache(heads=8, dim=dim, page=16, blocks=40 + sum(x[1] // 16 + 1 for x in lens), kind=kind,
               cache=cache) as c:
        attend_case(c, lens, 32, label="pieces")
        attend_case(c, lens, 32, window=50, label="pieces")


def test_a_nan_key_reaches_the_queries_that_see_it():
    """Alone in its stretch of keys, so that the wave or part that meets it has no other score."""
    for lens in ([(1, 257), (1, 1), (2, 1500)], [(70, 1025)]):
        with Cache(heads=2, dim=64, page=16, blocks=150, kind="bf16") as c:
            for t, (q, n) in zip(deal(c, lens), lens):
                c.host[0][int(t[(n - 1) // 16]), (n - 1) % 16, 1] = math.nan
            c.upload()
            attend_case(c, lens, 4, window=1 if len(lens) > 1 else 0, label="NaN key")
            attend_case(c, lens, 4, label="NaN key")


def test_tables_of_unseen_pages_may_hold_anything():
    with Cache(heads=1, dim=64, page=16, blocks=64, kind="bf16") as c:
        lens = [(1, 600, 20), (30, 300, 0)]
        tables = deal(c, lens)
        for t, (q, n, prefix) in zip(tables, lens):
            for pg in range(-(-n // 16)):
                if pg * 16 >= prefix and (pg + 1) * 16 <= n - q - 64 + 1:
                    t[pg] = -1
        tables_d = [t.cuda() for t in tables]
        seqs, rows = seqs_of(tables_d, lens)
        plan = c.plan(2, 2, rows, window=64)
        q = torch.randn(rows, 2, 64, device="cuda", dtype=torch.bfloat16)
        out = torch.empty_like(q)
        K.kv_attn_plan_set(plan, K.make_seqs(seqs))
        say("stale table entries outside the window")
        K.kv_attend(plan, 0, K.make_attend_args(q, out, n_tokens=rows, scale=0.125))
        assert K.kv_pool_get_error(c.handle) == 0
        clean = deal(c, lens)
        for t, (_, _, n, at, q_len, prefix) in zip(clean, seqs):
            k, v = (ref.cache_of(c.region(0, i), False, t, n) for i in (0, 1))
            want, _, tol, _ = ref.attend(q[at:at + q_len].cpu().double(), k, v, scale=0.125, window=64, prefix=prefix)
            assert ((out[at:at + q_len].cpu().double() - want).abs() <= tol).all()


@pytest.mark.parametrize("lens", [[(1, 300), (1, 200)], [(40, 300), (40, 200)]], ids=["few", "many"])
def test_a_bad_block_id_is_reported_and_stays_in_its_sequence(lens):
    with Cache(heads=2, dim=64, page=16, blocks=64, kind="bf16") as c:
        tables = deal(c, lens)
        tables_d = [t.cuda() for t in tables]
        tables_d[0][3] = 64
        seqs, rows = seqs_of(tables_d, lens)
        plan = c.plan(4, 2, rows)
        q = torch.randn(rows, 4, 64, device="cuda", dtype=torch.bfloat16)
        out = torch.empty_like(q)
        K.kv_attn_plan_set(plan, K.make_seqs(seqs))
        say("bad block id", lens)
        K.kv_attend(plan, 0, K.make_attend_args(q, out, n_tokens=rows, scale=0.125))
        assert K.kv_pool_get_error(c.handle) == K.KV_DEVERR_BLOCK_RANGE
        assert K.kv_pool_get_error(c.handle) == 0
        at, n = seqs[1][3], seqs[1][2]
        k, v = (ref.cache_of(c.region(0, i), False, tables[1], n) for i in (0, 1))
        want, _, tol, _ = ref.attend(q[at:].cpu().double(), k, v, scale=0.125)
        assert ((out[at:].cpu().double() - want).abs() <= tol).all()
        # appended tokens: the bad page is skipped, the others arrive
        tables_d[0][-3] = -1
        before = c.dev.clone()
        x = torch.randn(rows, 2, 64, device="cuda", dtype=torch.bfloat16)
        K.kv_append_tokens(plan, 0, K.make_append_args(x, x, n_tokens=rows))
        assert K.kv_pool_get_error(c.handle) == K.KV_DEVERR_BLOCK_RANGE
        changed = (c.dev != before).any(-1).any(0).nonzero().flatten().tolist()
        allowed = {int(i) for t, (q_len, n) in zip(tables, lens) for i in t[(n - q_len) // 16:-(-n // 16)]}
        assert set(changed) <= allowed - {int(tables[0][-3])} and changed


def test_attention_far_into_a_large_pool():
    """Block offsets past 2^32 bytes; the pages that are read sit at both ends of the region."""
    page, heads, dim = 64, 8, 128
    stride = page * heads * dim * 2
    blocks = (5 << 30) // stride
    buf = torch.zeros(2 * blocks * stride, dtype=torch.uint8, device="cuda")
    pool = K.kv_pool_create(K.make_pool_desc(1, 2, heads, dim, 2, page, blocks, stride,
                                             [buf.data_ptr(), buf.data_ptr() + blocks * stride]))
    view = buf.view(torch.bfloat16).view(2, blocks, page, heads, dim)
    ids = [blocks - 1, 0, blocks - 2, 4097, blocks // 2]
    n = 5 * page - 7
    gen = torch.Generator().manual_seed(5)
    k, v = (torch.randn(5 * page, heads, dim, generator=gen).bfloat16() for _ in range(2))
    table = torch.tensor(ids, dtype=torch.int32, device="cuda")
    for i, b in enumerate(ids):     # all but the newest 40 tokens are there; those are appended
        view[0, b], view[1, b] = k[i * page:(i + 1) * page].cuda(), v[i * page:(i + 1) * page].cuda()
    new = 40
    view[0, ids[-1]] = 0
    view[1, ids[-1]] = 0
    view[:, ids[-1], :page - 7 - new] = torch.stack([k, v])[:, 4 * page:n - new].cuda()
    plan = K.kv_attn_plan_create(pool, K.make_attn_desc(16, K.KV_TYPE_BF16, K.KV_TYPE_BF16, 1, new))
    K.kv_attn_plan_set(plan, K.make_seqs([(table, 5, n, 0, new)]))
    q = torch.randn(new, 16, dim, generator=gen).bfloat16()
    qd, out = q.cuda(), torch.empty(new, 16, dim, dtype=torch.bfloat16, device="cuda")
    kd, vd = k[n - new:n].cuda(), v[n - new:n].cuda()
    say("5 GiB regions")
    K.kv_append_tokens(plan, 0, K.make_append_args(kd, vd, n_tokens=new))
    K.kv_attend(plan, 0, K.make_attend_args(qd, out, n_tokens=new, scale=0.09))
    K.kv_copy_pages(pool, K.make_page_copies([(blocks - 1, blocks // 2 + 1, 64)]), 0, 1)
    assert K.kv_pool_get_error(pool) == 0
    want, _, tol, _ = ref.attend(q.double(), k[:n].double(), v[:n].double(), scale=0.09)
    assert ((out.cpu().double() - want).abs() <= tol).all()
    assert torch.equal(view[:, blocks // 2 + 1].cpu(), torch.stack([k, v])[:, :page])
    K.kv_attn_plan_destroy(plan)
    K.kv_pool_destroy(pool)


def test_attention_is_the_same_from_run_to_run_and_on_another_stream():
    with Cache(heads=2, dim=128, page=16, blocks=600, kind="bf16") as c:
        for lens in ([(1, 3000), (2, 500)], [(100, 4000), (3, 77)]):
            plan, args, out, lse, _held = attend_case(c, lens, 8)
            first = out.clone(), lse.clone()
            side = torch.cuda.Stream()
            torch.cuda.synchronize()
            for stream in (torch.cuda.current_stream(), side):
                out.fill_(5), lse.fill_(5)
                torch.cuda.synchronize()
                K.kv_attend(plan, 0, args, stream)
                torch.cuda.synchronize()
                rows = sum(q for q, _ in lens)
                assert torch.equal(words(out[:rows]), words(first[0][:rows]))
                assert torch.equal(words(lse[:rows]), words(first[1][:rows]))


def test_the_result_may_take_the_queries_place():
    with Cache(heads=2, dim=64, page=16, blocks=300, kind="bf16") as c:
        lens = [(1, 700), (2, 3), (60, 900), (1, 3000)]
        tables = [t.cuda() for t in deal(c, lens)]
        seqs, rows = seqs_of(tables, lens)
        plan = c.plan(8, len(lens), rows)
        K.kv_attn_plan_set(plan, K.make_seqs(seqs))
        q = torch.randn(rows, 8, 64, device="cuda").bfloat16()
        out = torch.empty_like(q)
        say("in place")
        K.kv_attend(plan, 0, K.make_attend_args(q, out, n_tokens=rows, scale=0.125))
        K.kv_attend(plan, 0, K.make_attend_args(q, q, n_tokens=rows, scale=0.125))
        torch.cuda.synchronize()
        assert torch.equal(words(q), words(out))


def test_a_captured_step_works_on_the_plan_that_is_set_when_it_runs():
    """Append and attend of two layers captured once; each replay after another plan, with
    eager work in between, against the same calls made eagerly."""
    steps = [[(1, 40), (1, 700), (2, 90)], [(1, 41), (1, 701), (2, 92)], [(1, 6000), (0, 5), (3, 3)],
             [(60, 200), (1, 1), (3, 30)], [(1, 2)], []]
    with Cache(layers=2, heads=2, dim=64, page=16, blocks=500, kind="f16") as c:
        most = 64
        plan = c.plan(8, 3, most)
        gen = torch.Generator(device="cuda").manual_seed(2)
        x = torch.randn(2, most, 12, 64, device="cuda", generator=gen).half()
        out = torch.zeros(2, most, 8, 64, device="cuda", dtype=torch.float16)
        lse = torch.zeros(2, most, 8, device="cuda")
        at = [K.make_attend_args(x[i, :, :8], out[i], lse[i], n_tokens=most, scale=0.125) for i in range(2)]
        ap = [K.make_append_args(x[i, :, 8:10], x[i, :, 10:], n_tokens=most) for i in range(2)]

        def step(stream):
            for i in range(2):
                K.kv_append_tokens(plan, i, ap[i], stream)
                K.kv_attend(plan, i, at[i], stream)

        def seqs(lens):
            tables = [t.cuda() for t in deal(c, lens, seed=8)]
            torch.cuda.synchronize()
            return K.make_seqs(seqs_of(tables, lens)[0]), tables

        graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        held = [seqs(lens) for lens in steps]
        K.kv_attn_plan_set(plan, held[0][0], side)
        torch.cuda.synchronize()
        say("capture of two layers")
        with torch.cuda.graph(graph, stream=side):
            with pytest.raises(K.KvError) as e:
                K.kv_attn_plan_set(plan, held[1][0], side)
            assert e.value.code == K.KV_ERR_CAPTURE
            step(side)
        start = c.dev.clone()
        for round in range(2):
            for lens, (s, _) in zip(steps, held):
                got = []
                for replay in (False, True):
                    c.dev.copy_(start)
                    out.fill_(3), lse.fill_(3), x.normal_(generator=torch.Generator(device="cuda").manual_seed(9))
                    torch.cuda.synchronize()
                    K.kv_attn_plan_set(plan, s, torch.cuda.current_stream())
                    if replay:
                        torch.cuda.synchronize()
                        say("replay", lens)
                        graph.replay()
                    else:
                        step(torch.cuda.current_stream())
                    torch.cuda.synchronize()
                    got.append([words(t).clone() for t in (c.dev, out, lse)])
                assert all(torch.equal(a, b) for a, b in zip(*got)), lens
        # a replay whose plan has more rows than the captured arrays writes none past them
        del graph


def test_a_replay_stays_within_the_captured_arrays():
    with Cache(heads=1, dim=64, page=16, blocks=64, kind="bf16") as c:
        plan = c.plan(2, 2, 64)
        short = [(1, 30), (3, 50)]
        tables = [t.cuda() for t in deal(c, [(40, 200), (10, 50)])]
        q = torch.randn(8, 2, 64, device="cuda").bfloat16()
        out, kv = torch.zeros_like(q), torch.randn(8, 1, 64, device="cuda").bfloat16()
        args = K.make_attend_args(q[:4], out[:4], n_tokens=4, scale=0.125)
        app = K.make_append_args(kv[:4], kv[:4], n_tokens=4)
        side = torch.cuda.Stream()
        K.kv_attn_plan_set(plan, K.make_seqs(seqs_of(tables, short)[0]), side)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            K.kv_append_tokens(plan, 0, app, side)
            K.kv_attend(plan, 0, args, side)
        K.kv_attn_plan_set(plan, K.make_seqs(seqs_of(tables, [(40, 200), (10, 50)])[0]), side)
        torch.cuda.synchronize()
        with pytest.raises(K.KvError) as e:
            K.kv_attend(plan, 0, args)
        assert e.value.code == K.KV_ERR_RANGE
        before = c.dev.clone()
        say("replay on a plan of more rows")
        graph.replay()
        torch.cuda.synchronize()
        assert (out[4:] == 0).all() and (out[:4] != 0).any()
        changed = (c.dev != before).any(-1)
        assert set(changed.any(0).nonzero().flatten().tolist()) == {int(tables[0][10])}


@pytest.mark.parametrize("kind,held", TYPES)
@pytest.mark.parametrize("head_major,dim,page", [(False, 128, 16), (True, 64, 24), (True, 80, 1), (False, 16, 100)])
def test_append(kind, held, head_major, dim, page):
    heads, lens = 3, [(1, 1), (40, 90), (0, 10), (17, 17), (1, 333), (33, 64)]
    with Cache(layers=2, heads=heads, dim=dim, page=page, blocks=800 // page + 20, head_major=head_major, kind=kind,
               cache=held, pad=16) as c:
        tables = deal(c, lens)
        tables_d = [t.cuda() for t in tables]
        seqs, rows = seqs_of(tables_d, lens)
        plan = c.plan(heads, len(lens), rows)
        x = torch.randn(rows + 2, 2 * heads + 1, dim, generator=torch.Generator().manual_seed(4)) * 5
        x[1, 0, 0], x[2, 1, 3], x[3, 2, 5], x[4, 4, 7] = math.nan, math.inf, -math.inf, 1e-9
        x = x.to(ref.TYPES[kind])
        xd = x.cuda()
        k, v = xd[:, :heads], xd[:, heads:2 * heads]
        K.kv_attn_plan_set(plan, K.make_seqs(seqs))
        say("append", kind, held, "head-major" if head_major else "token-major", dim, page)
        K.kv_append_tokens(plan, 1, K.make_append_args(k, v, n_tokens=rows + 2, k_scale=c.k_scale, v_scale=c.v_scale))
        torch.cuda.synchronize()
        for kv, src, scale in ((0, x[:, :heads], c.k_scale), (1, x[:, heads:2 * heads], c.v_scale)):
            view = ref.paged(c.region(1, kv), head_major).view(torch.uint8)
            new = words(ref.appended(src, scale, held)).view(rows + 2, heads, -1)
            for t, (_, _, n, at, q_len, _) in zip(tables, seqs):
                for i in range(q_len):
                    p = n - q_len + i
                    view[int(t[p // page]), p % page] = new[at + i]
        n = c.stride - 16
        want = c.flat.clone()
        want[:, :, :n] = words(c.host).view(4, c.blocks, -1)
        got = c.dev.cpu()
        if held == "e4m3":      # a NaN keeps whatever sign the conversion gives it
            for t in (got, want):
                t[:, :, :n][(t[:, :, :n] & 0x7f) == 0x7f] = 0x7f
        assert torch.equal(got, want)


def test_append_and_attend_refusals():
    with Cache(heads=2, dim=64, page=16, blocks=64, kind="bf16", cache="e4m3") as c:
        table = torch.arange(8, dtype=torch.int32, device="cuda")
        plan = c.plan(4, 2, 16)
        ok = (table, 8, 100, 0, 4)

        def refused(code, fn, *args):
            with pytest.raises(K.KvError) as e:
                fn(*args)
            assert e.value.code == code

        def bad(code, *seqs):
            refused(code, K.kv_attn_plan_set, plan, K.make_seqs(seqs))

        bad(K.KV_ERR_ARG, ok, ok, ok)                                  # more sequences than the plan holds
        bad(K.KV_ERR_ARG, (table, 8, 100, 0, 17))                      # more rows
        bad(K.KV_ERR_ARG, (table, 8, -1, 0, 1))
        bad(K.KV_ERR_ARG, (table, 8, 100, -1, 1))
        bad(K.KV_ERR_ARG, (table, 8, 100, 0, -1))
        bad(K.KV_ERR_ARG, (table, 8, 100, 0, 1, -1))
        bad(K.KV_ERR_ARG, (0, 8, 100, 0, 1))
        bad(K.KV_ERR_ALIGN, (table.data_ptr() + 2, 7, 100, 0, 1))
        bad(K.KV_ERR_RANGE, (table, 6, 100, 0, 1))
        bad(K.KV_ERR_RANGE, (table, 1 << 31, 100, 0, 1))
        bad(K.KV_ERR_RANGE, (table, (1 << 31) - 1, (1 << 31) - 4096, 0, 1))
        bad(K.KV_ERR_RANGE, (table, 1 << 30, 100, 0, 1))               # past its allocation
        bad(K.KV_ERR_RANGE, (table, 8, 100, (1 << 31) - 2, 4))
        bad(K.KV_ERR_DUP, ok, (table, 8, 100, 3, 2))
        K.kv_attn_plan_set(plan, K.make_seqs([ok]))
        q = torch.zeros(4, 4, 64, dtype=torch.bfloat16, device="cuda")
        out, kv = torch.zeros_like(q), torch.zeros(4, 2, 64, dtype=torch.bfloat16, device="cuda")

        def attend(code, layer=0, **kw):
            a = dict(n_tokens=4, scale=0.1, q_strides=(256, 64), out_strides=(256, 64))
            qq, oo = kw.pop("q", q), kw.pop("out", out)
            a.update(kw)
            refused(code, K.kv_attend, plan, layer, K.make_attend_args(qq, oo, kw.get("lse"), **{
                k: v for k, v in a.items() if k != "lse"}))

        attend(K.KV_ERR_ARG, layer=1)
        attend(K.KV_ERR_ARG, layer=-1)
        attend(K.KV_ERR_RANGE, n_tokens=3)
        attend(K.KV_ERR_ARG, n_tokens=-1)
        attend(K.KV_ERR_ARG, scale=math.nan)
        attend(K.KV_ERR_ARG, softcap=-1.0)
        attend(K.KV_ERR_ARG, softcap=1e-42)                          # 2.9e41 times the dot product
        attend(K.KV_ERR_ARG, softcap=3e38)
        attend(K.KV_ERR_ARG, k_scale=0.0)
        attend(K.KV_ERR_ARG, v_scale=math.inf)
        attend(K.KV_ERR_ARG, q=0)
        attend(K.KV_ERR_ARG, out=0)
        attend(K.KV_ERR_ALIGN, q=q.data_ptr() + 8)
        attend(K.KV_ERR_ALIGN, q_strides=(257, 64))
        attend(K.KV_ERR_ALIGN, out_strides=(256, 68))
        attend(K.KV_ERR_ARG, q_strides=(-256, 64))
        attend(K.KV_ERR_ARG, out_strides=(0, 64))                      # rows of the result over each other
        attend(K.KV_ERR_ARG, out_strides=(64, 64))
        attend(K.KV_ERR_RANGE, q_strides=(1 << 40, 64))
        attend(K.KV_ERR_ALIGN, lse=out.data_ptr() + 2)
        attend(K.KV_ERR_ALIGN, alibi_slopes=out.data_ptr() + 1)
        for code, kw in ((K.KV_ERR_RANGE, dict(n_tokens=3)), (K.KV_ERR_ARG, dict(k_scale=-1.0)),
                         (K.KV_ERR_ARG, dict(v_scale=math.nan))):
            a = dict(n_tokens=4)
            a.update(kw)
            refused(code, K.kv_append_tokens, plan, 0, K.make_append_args(kv, kv, **a))
        K.kv_attn_plan_set(plan, K.make_seqs([(table, 8, 3, 0, 4)]))   # more new tokens than cached ones
        refused(K.KV_ERR_ARG, K.kv_append_tokens, plan, 0, K.make_append_args(kv, kv, n_tokens=4))
        assert (out == 0).all() and torch.equal(c.dev.cpu(), c.flat)


@pytest.mark.parametrize("head_major,heads,dim,kind", [(False, 8, 128, "bf16"), (True, 8, 128, "bf16"), (True, 16, 12, "f16"),
                                                       (True, 100, 6, "f16"), (False, 3, 16, "e4m3"), (True, 4, 16, "e4m3")])
@pytest.mark.parametrize("n", [1, 40, 300])
def test_page_copies(head_major, heads, dim, kind, n):
    rng = np.random.default_rng(n)
    with Cache(layers=3, heads=heads, dim=dim, page=16, blocks=700, head_major=head_major, kind=kind, pad=48) as c:
        ids = rng.permutation(700)
        dst = ids[:n]
        src = rng.choice(ids[n:], n)            # a source may be copied twice
        tok = np.where(rng.random(n) < 0.5, 16, rng.integers(1, 17, n))
        K.kv_copy_pages(c.handle, K.make_page_copies(zip(src, dst, tok)), 1, 3)
        say("copies", n, "head-major" if head_major else "token-major", heads, dim)
        torch.cuda.synchronize()
        for kv in range(2, 6):
            view = ref.paged(c.host[kv], head_major).view(torch.uint8)
            for s, d, k in zip(src, dst, tok):
                view[int(d), :k] = view[int(s), :k]
        want = c.flat.clone()
        want[:, :, :c.stride - 48] = words(c.host).view(6, c.blocks, -1)
        assert torch.equal(c.dev.cpu(), want)


@pytest.mark.parametrize("n", [0, 1, 256, 257, 4096, 5000])
@pytest.mark.parametrize("in_place", [False, True])
def test_remapped_tables(n, in_place):
    rng = np.random.default_rng(n)
    with Cache(heads=1, dim=16, page=1, blocks=12000, kind="bf16") as c:
        src = rng.permutation(12000)[:n].astype(np.int32)
        dst = rng.integers(0, 12000, n).astype(np.int32)
        t = rng.integers(-3, 12010, 70001).astype(np.int32)
        t[:len(src)] = src
        want = t.copy()
        m = dict(zip(src.tolist(), dst.tolist()))
        want[:] = [m.get(x, x) for x in t.tolist()]
        d = torch.from_numpy(t).cuda()
        out = d if in_place else torch.full_like(d, -9)
        torch.cuda.synchronize()
        say("remap", n)
        K.kv_remap_tables(c.handle, K.make_page_copies([(a, b, 1) for a, b in zip(src, dst)]), d, out, 70000)
        torch.cuda.synchronize()
        want[70000:] = t[70000:] if in_place else -9
        assert np.array_equal(out.cpu().numpy(), want)


def test_copies_and_remaps_captured():
    with Cache(heads=2, dim=64, page=16, blocks=600, kind="bf16") as c:
        few = K.make_page_copies([(i, 200 + i, 16 - i % 3) for i in range(100)])
        lots = K.make_page_copies([(i, 300 + i, 16) for i in range(257)])
        t = torch.arange(400, dtype=torch.int32, device="cuda")
        out = torch.zeros_like(t)
        side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
        K.kv_copy_pages(c.handle, few, 0, 1, side)
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=side):
            for fn, args in ((K.kv_copy_pages, (lots, 0, 1)), (K.kv_remap_tables, (lots, t, out, 400))):
                with pytest.raises(K.KvError) as e:
                    fn(c.handle, *args, side)
                assert e.value.code == K.KV_ERR_CAPTURE
            K.kv_copy_pages(c.handle, few, 0, 1, side)
            K.kv_remap_tables(c.handle, few, t, out, 400, side)
        for k in range(3):
            c.dev[:, :100].random_(0, 255)
            c.dev[:, 200:] = k
            out.fill_(0)
            torch.cuda.synchronize()
            want = c.dev.clone()
            for i in range(100):
                n = (16 - i % 3) * 256
                want[:, 200 + i, :n] = want[:, i, :n]
            say("replay", k)
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(c.dev, want)
            assert out.tolist() == [200 + i if i < 100 else i for i in range(400)]


@pytest.mark.parametrize("kind,held", [("bf16", "bf16"), ("f16", "e4m3")])
def test_a_request_forks_grows_is_compacted_and_answers_the_same(kind, held):
    """The operators as a serving program uses them together: a prompt is appended and
    attended to; two children fork off it and each grows by one token; the pool is compacted and
    the tables rewritten; the next token's attention is what it is without the compaction."""
    with Cache(layers=2, heads=2, dim=64, page=16, blocks=64, kind=kind, cache=held, seed=6) as c:
        stream = torch.cuda.current_stream()
        gen = torch.Generator().manual_seed(1)
        rows = lambda n: torch.randn(2, n, 8, 64, generator=gen).to(ref.TYPES[kind])    # noqa: E731
        scales = dict(k_scale=c.k_scale, v_scale=c.v_scale)
        plan = c.plan(4, 3, 128)
        hole = K.kv_pool_alloc_blocks(c.handle, 20)
        parent = K.kv_pool_alloc_blocks(c.handle, 7)
        K.kv_pool_free_blocks(c.handle, hole)
        tables = torch.zeros(3, 8, dtype=torch.int32, device="cuda")
        tables[0, :7] = torch.from_numpy(parent)
        held_rows = [[torch.zeros(0, 2, 64) for _ in range(2)] for _ in range(2)]       # [layer][k, v] of the parent

        def step(x, seqs):
            K.kv_attn_plan_set(plan, K.make_seqs(seqs), stream)
            out = torch.zeros(2, x.shape[1], 4, 64, dtype=x.dtype, device="cuda")
            for i in range(2):
                K.kv_append_tokens(plan, i, K.make_append_args(x[i, :, 4:6], x[i, :, 6:], n_tokens=x.shape[1],
                                                               **scales), stream)
                K.kv_attend(plan, i, K.make_attend_args(x[i, :, :4], out[i], n_tokens=x.shape[1], scale=0.125,
                                                        **scales), stream)
            return out

        def check(x, out, at, layer, k, v, q_len=1):
            want, _, tol, _ = ref.attend(x[layer, at:at + q_len, :4].double(), k.double(), v.double(), scale=0.125,
                                         k_scale=float(np.float32(c.k_scale)), v_scale=float(np.float32(c.v_scale)),
                                         kind=kind)
            assert ((out[layer, at:at + q_len].cpu().double() - want).abs() <= tol).all()

        prompt = rows(100)
        say("prompt")
        out = step(prompt.cuda(), [(tables[0], 8, 100, 0, 100)])
        hold = lambda x, a: (ref.appended(x[:, 4:6], c.k_scale, held).float(),          # noqa: E731
                             ref.appended(x[:, 6:], c.v_scale, held).float())[a]
        for i in range(2):
            held_rows[i] = [hold(prompt[i], 0), hold(prompt[i], 1)]
            check(prompt, out, 0, i, *held_rows[i], q_len=100)
        kids, tails = [], []
        for n in range(2):
            child, tail = K.kv_pool_fork_blocks(c.handle, 100, parent)
            kids.append(child)
            tails.append(tail)
            tables[n + 1, :7] = torch.from_numpy(child)
        K.kv_copy_pages(c.handle, K.make_page_copies(tails), 0, 2, stream)
        grown = rows(3)
        say("fork")
        out = step(grown.cuda(), [(tables[n], 8, 101, n, 1) for n in range(3)])
        for i in range(2):
            for n in range(3):
                k, v = (torch.cat([held_rows[i][a], hold(grown[i], a)[n:n + 1]]) for a in range(2))
                check(grown, out, n, i, k, v)
        again = rows(3)
        plain = step(again.cuda(), [(tables[n], 8, 102, n, 1) for n in range(3)])
        torch.cuda.synchronize()
        moves = K.kv_pool_plan_compact(c.handle, 64)
        assert moves._n == 9 - 2        # two tails sit in the holes already
        K.kv_copy_pages(c.handle, moves, 0, 2, stream)
        K.kv_remap_tables(c.handle, moves, tables, tables, tables.numel(), stream)
        torch.cuda.synchronize()
        K.kv_pool_free_blocks(c.handle, [m.src for m in moves[:moves._n]])
        assert K.kv_pool_free_count(c.handle) == 64 - 9 and int(tables[:, :7].max()) < 9
        c.dev[:, 9:] = 0xff             # NaN in what was freed
        say("compacted")
        out = step(again.cuda(), [(tables[n], 8, 102, n, 1) for n in range(3)])
        assert torch.equal(words(out), words(plain))
        assert K.kv_pool_get_error(c.handle, stream) == 0


def test_a_pool_destroyed_behind_its_page_copies():
    """Copies and rewritten tables have no event of their own: destroy waits for the device."""
    region = torch.arange(64 * 4096, dtype=torch.int32, device="cuda").view(64, 4096)    # 16 KiB pages
    want, table = region.clone(), torch.arange(64, dtype=torch.int32, device="cuda")
    side, big = torch.cuda.Stream(), torch.ones(1 << 26, device="cuda")
    pool = K.kv_pool_create(K.make_pool_desc(1, 1, 8, 128, 1, 16, 64, 16384, [region]))
    torch.cuda.synchronize()
    copies = K.make_page_copies([(i, 32 + i, 16) for i in range(8)])
    say("copies behind other work, then destroy")
    with torch.cuda.stream(side):
        for _ in range(20):
            big.mul_(1.0)
        K.kv_copy_pages(pool, copies, 0, 1, side)
        K.kv_remap_tables(pool, copies, table, table, 64, side)
    K.kv_pool_destroy(pool)
    assert side.query()
    want[32:40] = want[:8]
    assert torch.equal(region, want) and table[:8].tolist() == list(range(32, 40)) and table[8:].tolist() == list(range(8, 64))


def test_a_plan_is_ready_on_every_stream_when_create_returns():
    """Made behind work on the null stream, set and used on another at once."""
    with Cache(heads=2, dim=64, page=16, blocks=64, kind="bf16") as c:
        lens = [(1, 300), (2, 90)]
        tables = [t.cuda() for t in deal(c, lens)]
        seqs, rows = seqs_of(tables, lens)
        q = torch.randn(rows, 4, 64, device="cuda").bfloat16()
        out, want = torch.zeros_like(q), torch.zeros_like(q)
        args = [K.make_attend_args(q, o, n_tokens=rows, scale=0.125) for o in (out, want)]
        plan = c.plan(4, 2, rows)
        K.kv_attn_plan_set(plan, K.make_seqs(seqs))
        K.kv_attend(plan, 0, args[1])
        side, big = torch.cuda.Stream(), torch.ones(1 << 28, device="cuda")
        torch.cuda.synchronize()
        say("a plan made behind other work")
        for _ in range(60):
            big.mul_(1.0)
        plan = c.plan(4, 2, rows)
        assert torch.cuda.current_stream().query()      # the header's promise: it waits for the device
        K.kv_attn_plan_set(plan, K.make_seqs(seqs), side)
        K.kv_attend(plan, 0, args[0], side)
        torch.cuda.synchronize()
        assert (want != 0).any() and torch.equal(words(out), words(want))


def test_an_error_right_after_the_last_one_was_read_is_not_lost():
    """Reading clears the error word before it returns: calls on a stream of their own, behind work on
    the null stream that waits for none of them."""
    with Cache(heads=2, dim=64, page=16, blocks=64, kind="bf16") as c:
        side = torch.cuda.Stream()
        table = torch.full((20,), 64, dtype=torch.int32, device="cuda")
        q = torch.randn(1, 4, 64, device="cuda").bfloat16()
        out, big = torch.zeros_like(q), torch.ones(1 << 22, device="cuda")
        plan = c.plan(4, 1, 1)
        K.kv_attn_plan_set(plan, K.make_seqs([(table, 20, 300, 0, 1)]), side)
        args = K.make_attend_args(q, out, n_tokens=1, scale=0.125)
        say("errors one after another")
        for _ in range(100):
            K.kv_attend(plan, 0, args, side)
            big.mul_(1.0)
            assert K.kv_pool_get_error(c.handle, side) == K.KV_DEVERR_BLOCK_RANGE
        assert K.kv_pool_get_error(c.handle, side) == 0


@pytest.mark.parametrize("mode", [0, 2], ids=["global", "relaxed"])
def test_nothing_is_freed_that_cannot_be_waited_for(mode):
    """While a stream captures the device cannot be waited for: a plan, and a pool with copies in flight, then
    stay as they are."""
    region = torch.arange(64 * 4096, dtype=torch.int32, device="cuda").view(64, 4096)    # 16 KiB pages
    regions = [region, region.clone()]
    want = [r.clone() for r in regions]
    pool = K.kv_pool_create(K.make_pool_desc(1, 2, 8, 64, 2, 16, 64, 16384, regions))
    plan = K.kv_attn_plan_create(pool, K.make_attn_desc(8, K.KV_TYPE_BF16, K.KV_TYPE_BF16, 1, 1))
    side, other, big = torch.cuda.Stream(), torch.cuda.Stream(), torch.ones(1 << 26, device="cuda")
    graph = ctypes.c_void_p()
    torch.cuda.synchronize()
    say("destroy while a stream captures, mode", mode)
    with torch.cuda.stream(other):
        for _ in range(20):
            big.mul_(1.0)
        K.kv_copy_pages(pool, K.make_page_copies([(i, 32 + i, 16) for i in range(8)]), 0, 1, other)
    begun = K._lib.hipStreamBeginCapture(ctypes.c_void_p(side.cuda_stream), mode)
    codes = [K._lib.kv_attn_plan_destroy(ctypes.c_void_p(plan)), K._lib.kv_pool_destroy(ctypes.c_void_p(pool))]
    K._lib.hipStreamEndCapture(ctypes.c_void_p(side.cuda_stream), ctypes.byref(graph))
    K._lib.hipGetLastError()
    torch.cuda.synchronize()
    assert begun == 0 and codes == [K.KV_ERR_HIP, K.KV_ERR_HIP]
    K.kv_copy_pages(pool, K.make_page_copies([(i, 40 + i, 16) for i in range(8)]), 0, 1, other)
    torch.cuda.synchronize()
    for r, w in zip(regions, want):
        w[32:40], w[40:48] = w[:8], w[:8]
        assert torch.equal(r, w)
    K.kv_attn_plan_destroy(plan)
    K.kv_pool_destroy(pool)
