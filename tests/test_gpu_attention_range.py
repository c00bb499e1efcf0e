"""Attention over its arguments' whole range, on the GPU against 64 bits: caps far above the scores,
tails far below the largest score, infinite and NaN values at every padded width."""
from __future__ import annotations

import math

import pytest
import torch

import paged_reference as ref
from paged_layout_transfer_amd import kvxfer as K
from test_gpu_operators import Cache, attend_case, deal, say, seqs_of, words

pytestmark = pytest.mark.gpu

F = 2.0 ** -24      # half a unit in the last place of 32 bits


def run(c, lens, heads_q, q, **kw):
    """out and lse of one call, on the host in 64 bits, with each sequence's rows and cache."""
    tables = deal(c, lens)
    on_gpu = [t.cuda() for t in tables]
    seqs, rows = seqs_of(on_gpu, lens)
    plan = c.plan(heads_q, len(lens), rows, kw.pop("window", 0))
    K.kv_attn_plan_set(plan, K.make_seqs(seqs))
    qd = q.cuda()
    out, lse = torch.zeros_like(qd), torch.zeros(rows, heads_q, device="cuda")
    K.kv_attend(plan, 0, K.make_attend_args(qd, out, lse, n_tokens=rows, k_scale=c.k_scale, v_scale=c.v_scale, **kw))
    torch.cuda.synchronize()
    held = [(at, q_len, *(ref.cache_of(c.region(0, i), False, t, n) for i in (0, 1)))
            for t, (_, _, n, at, q_len, _) in zip(tables, seqs)]
    return out.cpu().double(), lse.cpu().double(), held


CAPS = [0.5, 30.0, 64.0, 65.0, 1e3, 1e4, 1e5, 1e6, 1e7, 1e20, 2e38]


@pytest.mark.parametrize("softcap", CAPS)
@pytest.mark.parametrize("lens", [[(1, 700), (3, 90)], [(70, 400)]], ids=["few", "many"])
@pytest.mark.parametrize("kind,held,dim", [("f16", "f16", 64), ("bf16", "e4m3", 128)])
def test_a_cap_is_exact_however_large(softcap, lens, kind, held, dim):
    """The bound is relative to the score for caps over 64, 2^-21 of the cap below.  With f = 2^-24: the products' sum as in
    paged_reference.attend, f (dim + 8) scale sum|q k|, which a cap only shrinks; then of c tanh(s / c)
    = s P(u) / Q(u), u = (s / c)^2, at most 24 roundings: scale and base 2, s / c 3 (u twice that and its
    own, worth half in the quotient, 4), P and Q 5 each with their coefficients, reciprocal 2, two
    products 2, the quotient's own error and the edge's 2 (2^-23.8 and 2^-26.2).  A weight is off by twice the
    worst error of a score, as is their sum."""
    with Cache(heads=2, dim=dim, page=16, blocks=60, kind=kind, cache=held) as c:
        gen = torch.Generator().manual_seed(7)
        rows = sum(x[0] for x in lens)
        # scores of standard deviation 3 to 4
        q = (torch.randn((rows, 4, dim), generator=gen) * 3).to(ref.TYPES[kind])
        scale = 1 / math.sqrt(dim)
        say("cap", softcap, lens, kind, held, dim)
        out, lse, seqs = run(c, lens, 4, q, scale=scale, softcap=softcap)
        u = torch.finfo(ref.TYPES[kind]).eps / 2
        ks, vs = (float(torch.tensor(x, dtype=torch.float32)) for x in (c.k_scale, c.v_scale))
        for at, n_q, k, v in seqs:
            n = k.shape[0]
            seen = ref.visible(n_q, n)
            for x in range(4):
                qq, kk, vv = q[at:at + n_q, x].double(), k[:, x // 2] * ks, v[:, x // 2] * vs
                s = softcap * torch.tanh(qq @ kk.t() * scale / softcap)
                ds = F * (dim + 8) * scale * (qq.abs() @ kk.abs().t())
                ds = ds + (24 * F * s.abs() if softcap > 64 else 8 * F * s.abs() + 2.0 ** -21 * softcap)
                e = torch.where(seen, ds, 0.0).amax(-1)
                s = torch.where(seen, s, -math.inf)
                z = torch.logsumexp(s, -1)
                w = torch.exp(s - z[:, None])
                want, a = w @ vv, w @ vv.abs()
                rel = (2 * e + (4 * n + 64) * F)[:, None]
                small = 2.0 ** -25 * (seen.double() @ vv.abs()) if kind == "f16" else 0.0
                tol = a * (u + rel) + small + want.abs() * (u + rel) + torch.finfo(ref.TYPES[kind]).smallest_normal * 2 * u
                got, got_z = out[at:at + n_q, x], lse[at:at + n_q, x]
                off = (got - want).abs() / tol
                assert off.max() <= 1, "out: %g of what is allowed" % off.max()
                off = (got_z - z).abs() / (e + (4 * n + 64) * F + 8 * F * z.abs())
                assert off.max() <= 1, "lse: %g of what is allowed" % off.max()


@pytest.mark.parametrize("lens", [[(1, 40)], [(40, 80)]], ids=["few", "many"])
def test_a_capped_score_that_is_infinite_or_nan(lens):
    """An infinite score is at the cap; NaN stays NaN."""
    with Cache(heads=1, dim=64, page=16, blocks=20, kind="bf16") as c:
        for t, (_, n) in zip(deal(c, lens), lens):
            at = lambda j: c.host[0][int(t[j // 16]), j % 16, 0]       # noqa: E731
            at(3)[0] = math.inf
            at(7)[0] = -math.inf
            at(n - 1)[1] = math.nan
        c.upload()
        rows = lens[0][0]
        q = torch.rand(rows, 1, 64, generator=torch.Generator().manual_seed(1)).bfloat16() + 0.1
        say("infinite capped scores", lens)
        out, lse, seqs = run(c, lens, 1, q, scale=0.125, softcap=5.0)
        (_, n_q, k, v), = seqs
        s = 5 * torch.tanh(q[:, 0].double() @ k[:, 0].t() * 0.125 / 5)
        assert (s[:, 3] == 5).all() and (s[:, 7] == -5).all()
        s = torch.where(ref.visible(n_q, k.shape[0]), s, -math.inf)
        z = torch.logsumexp(s, -1)
        assert torch.equal(torch.isnan(lse[:, 0]), torch.isnan(z)) and torch.isnan(z[-1])
        assert torch.equal(torch.isnan(out[:, 0]), torch.isnan(z)[:, None].expand(-1, 64))
        fine = ~torch.isnan(z)
        # scores below 5: their products' sums 72 roundings of at most 20, the cap 24 of 5; the sum 4 n + 64
        assert ((lse[:, 0] - z).abs()[fine] <= F * (72 * 20 + 24 * 5 + 4 * 80 + 64 + 64)).all()


@pytest.mark.parametrize("lens", [[(1, 700)], [(2, 9000), (1, 5000)], [(40, 5000)], [(66, 3000)] * 12],
                         ids=["few", "few_cut", "many", "many_whole"])
@pytest.mark.parametrize("kind,held,dim", [("f16", "f16", 64), ("f16", "f16", 256), ("f16", "e4m3", 128), ("bf16", "bf16", 64)])
def test_a_long_tail_far_below_the_first_key(lens, kind, held, dim):
    """The first key's score lies 17.5 above the others', which hold all of the values (none is negative, so
    the sum of absolute values is the result).  The bounds are those of paged_reference.attend, one product a
    score, but half weights lose 2^-32 of the largest one: they are scaled by 2^7, and the largest is at
    least 1 before that."""
    heads = 2
    with Cache(heads=heads, dim=dim, page=16, blocks=sum(n // 16 + 1 for _, n in lens), kind=kind, cache=held) as c:
        c.k_scale = c.v_scale = 1.0
        gen = torch.Generator().manual_seed(9)
        c.host[0] = 0
        c.host[0][..., 0] = (torch.rand(c.host[0].shape[:-1], generator=gen) * 2 - 1).to(c.host.dtype)
        c.host[1] = (torch.rand(c.host[1].shape, generator=gen) * 8 + 8).to(c.host.dtype)
        for t in deal(c, lens):
            c.host[0][int(t[0]), 0, :, 0] = torch.tensor(17.5).to(c.host.dtype)      # 18 in e4m3
            c.host[1][int(t[0]), 0] = 0
        c.upload()
        rows = sum(x[0] for x in lens)
        q = torch.zeros(rows, 4 * heads, dim)
        q[..., 0] = 8
        q = q.to(ref.TYPES[kind])
        say("long tail", lens[:3], kind, held, dim)
        out, lse, seqs = run(c, lens, 4 * heads, q, scale=0.125)
        u = torch.finfo(ref.TYPES[kind]).eps / 2
        for at, n_q, k, v in seqs:
            want, z, _, tol_z = ref.attend(q[at:at + n_q].double(), k, v, scale=0.125, kind=kind)
            n = k.shape[0]
            e = F * (dim + 16) * 18
            tol = 2 * want * (u + 2 * e + (4 * n + 64) * F) + torch.finfo(ref.TYPES[kind]).smallest_normal * 2 * u
            if kind == "f16":
                seen = ref.visible(n_q, n).double()
                tol = tol + 2.0 ** -32 * torch.stack([seen @ v[:, x // 4] for x in range(4 * heads)], 1)
            off = (out[at:at + n_q] - want).abs() / tol
            assert off.max() <= 1, "out: %g of what is allowed, %g for %g" % (off.max(), out[at:at + n_q].flatten()[off.argmax()], want.flatten()[off.argmax()])
            off = (lse[at:at + n_q] - z).abs() / tol_z
            assert off.max() <= 1, "lse: %g of what is allowed" % off.max()


@pytest.mark.parametrize("lens", [[(1, 300), (3, 900)], [(1, 9000)], [(70, 600), (40, 2000)], [(66, 700)] * 20],
                         ids=["few", "few_cut", "many", "many_whole"])
@pytest.mark.parametrize("kind,held,dim,apart", [("f16", "f16", 64, 40), ("bf16", "bf16", 128, 40), ("bf16", "bf16", 64, 200),
                                                 ("f16", "f16", 256, 200), ("f16", "e4m3", 128, 40), ("bf16", "bf16", 80, 200)])
def test_a_seen_infinity_counts_however_small_its_weight(lens, kind, held, dim, apart):
    """Infinite and NaN values of keys whose scores lie `apart` below those of every 32nd key, which come before
    them in whatever order the keys are taken: their weights are small, or zero in 32 bits, but positive.  In
    stretches of keys that every query sees, and nothing of it reaches the other columns and heads."""
    heads = 2
    with Cache(heads=heads, dim=dim, page=16, blocks=sum(n // 16 + 1 for _, n in lens), kind=kind, cache=held) as c:
        c.host[0] = 0
        for t, (q, n) in zip(deal(c, lens), lens):
            for j in range(0, n, 32):
                c.host[0][int(t[j // 16]), j % 16, :, 0] = torch.tensor(16.0).to(c.host.dtype)
            at = lambda j: c.host[1][int(t[j // 16]), j % 16]       # noqa: E731
            at(0)[0, 3] = math.nan
            if held != "e4m3":
                at(1)[0, 5] = math.inf
                at(70)[1, 9] = -math.inf
                at(5)[1, dim - 1], at(100)[1, dim - 1] = math.inf, math.inf
                at(6)[0, 11], at(130)[0, 11] = math.inf, -math.inf
        c.upload()
        rows = sum(x[0] for x in lens)
        q = torch.zeros(rows, 4 * heads, dim)
        q[..., 0] = apart / 16 / c.k_scale
        q = q.to(ref.TYPES[kind])
        say("infinities of small weight", lens[:3], kind, held, dim, apart)
        out, lse, seqs = run(c, lens, 4 * heads, q, scale=1.0)
        assert torch.isfinite(lse).all()
        ks, vs = (float(torch.tensor(x, dtype=torch.float32)) for x in (c.k_scale, c.v_scale))
        for at, n_q, k, v in seqs:
            want, _, tol, _ = ref.attend(q[at:at + n_q].double(), k, v, scale=1.0, kind=kind, k_scale=ks, v_scale=vs)
            got = out[at:at + n_q]
            assert torch.equal(torch.isnan(got), torch.isnan(want)) and torch.isnan(got).any()
            inf = torch.isinf(want)
            assert torch.equal(torch.isinf(got), inf) and torch.equal(got[inf], want[inf])
            assert inf.any() or held == "e4m3"
            fin = torch.isfinite(want)
            assert ((got - want).abs()[fin] <= tol[fin]).all()


# a head to each wave of the few-rows kernel: heads a multiple of four, and work enough
FORMS = {"few": (2, [(1, 700), (2, 300)]), "many": (2, [(50, 400), (70, 100), (130, 135)]),
         "a_head_a_wave": (4, [(1 + i % 3, 240 + i) for i in range(260)])}


@pytest.mark.parametrize("form", list(FORMS))
@pytest.mark.parametrize("dim", [80, 128, 192, 256])
@pytest.mark.parametrize("kind,held", [("bf16", "bf16"), ("f16", "e4m3")])
def test_what_a_query_does_not_see_does_not_reach_it_at_other_widths(form, dim, kind, held):
    """NaN, and infinities where the type has them, in unused pages, behind the last token, outside the
    window, and in the newest token, which earlier queries of the call do not see."""
    heads, lens = FORMS[form]
    for window, poison in ((0, math.nan), (100, math.nan), (100, math.inf)):
        if held == "e4m3" and poison == math.inf:
            continue
        with Cache(heads=heads, dim=dim, page=16, blocks=20 + sum(n // 16 + 1 for _, n in lens), kind=kind, cache=held) as c:
            keep = torch.zeros(c.blocks, c.page, dtype=torch.bool)
            for t, (q, n) in zip(deal(c, lens), lens):
                j = torch.arange(max(0, n - q - window + 1) if window else 0, n)
                keep[t.long()[j // 16], j % 16] = True
                keep[int(t[(n - 1) // 16]), (n - 1) % 16] = False
            bits = c.host.view(torch.uint8 if held == "e4m3" else torch.int16)
            bits[:, ~keep] = torch.tensor([poison]).to(c.host.dtype).view(bits.dtype)
            c.upload()
            attend_case(c, lens, 2 * heads, window=window, label="poison %s" % poison)


SHAPES = [dict(), dict(window=40, softcap=200.0), dict(window=40), dict(softcap=30.0, slopes=True)]
SPECIAL = [(form, dim, kind, held, shape) for form in FORMS for dim in (80, 128, 192, 256)
           for kind, held in (("bf16", "bf16"), ("f16", "f16"), ("bf16", "e4m3")) for shape in SHAPES
           if form != "a_head_a_wave" or (kind == held == "bf16" and shape in SHAPES[:2])]      # 60 times the reference's work


@pytest.mark.parametrize("form,dim,kind,held,shape", SPECIAL, ids=str)
def test_infinite_and_nan_values_at_other_widths(form, dim, kind, held, shape):
    """Values of single cached tokens: the first one, one in the middle and the newest, an infinity of either
    sign, both in one column, NaN, in the first and the last columns."""
    heads, lens = FORMS[form]
    with Cache(heads=heads, dim=dim, page=16, blocks=20 + sum(n // 16 + 1 for _, n in lens), kind=kind, cache=held) as c:
        for t, (q, n) in zip(deal(c, lens), lens):
            at = lambda j: c.host[1][int(t[j // 16]), j % 16]       # noqa: E731
            at(n - 1)[1, 7], at(n // 3)[heads - 1, dim - 2] = math.nan, math.nan
            if held != "e4m3":
                at(0)[0, 3] = math.inf
                at(n // 2)[0, 5] = -math.inf
                at(n - 1)[0, 9], at(n - 2)[0, 9] = math.inf, -math.inf
                at(n - 2)[heads - 1, dim - 1] = math.inf
        c.upload()
        attend_case(c, lens, 2 * heads, label="infinite values", **shape)


@pytest.mark.parametrize("kind,held", [("bf16", "bf16"), ("f16", "f16"), ("bf16", "e4m3"), ("f16", "e4m3")])
@pytest.mark.parametrize("dim", [136, 192, 240, 96, 48])
@pytest.mark.parametrize("head_major", [False, True])
def test_widths_between_those_of_the_kernels(kind, held, dim, head_major):
    if held == "e4m3" and dim % 16:
        dim += 8
    lens = [(1, 700), (2, 33), (70, 70), (1, 300), (40, 500), (130, 131), (3, 3)]
    with Cache(heads=2, dim=dim, page=24, blocks=200, head_major=head_major, kind=kind, cache=held, pad=32) as c:
        attend_case(c, lens, 8)
        attend_case(c, lens, 4, window=60, softcap=100.0, slopes=True)


@pytest.mark.parametrize("softcap", [0.0, 200.0])
def test_infinities_and_a_large_cap_captured(softcap):
    """A graph of both kernels and the join, replayed between eager calls, against the eager result; every other
    replay with no infinity in the cache."""
    lens = [(1, 9000), (2, 300), (70, 600)]
    with Cache(heads=2, dim=128, page=16, blocks=700, kind="f16") as c:
        c.host[0] = 0
        tables = deal(c, lens)
        for t, (_, n) in zip(tables, lens):
            for j in range(0, n, 32):
                c.host[0][int(t[j // 16]), j % 16, :, 0] = 16.0
        clean = c.host.clone()
        for t in tables:
            c.host[1][int(t[4]), 6, 1, 9] = math.inf
            c.host[1][int(t[5]), 3, 0, 127] = -math.inf
        caches = []
        for h in (c.host.clone(), clean):
            c.host = h
            c.upload()
            caches.append(c.dev.clone())
        on_gpu = [t.cuda() for t in tables]
        seqs, rows = seqs_of(on_gpu, lens)
        plan = c.plan(8, len(lens), rows)
        q = torch.zeros(rows, 8, 128, device="cuda", dtype=torch.float16)
        q[..., 0] = 40 / 16
        out, lse = torch.zeros_like(q), torch.zeros(rows, 8, device="cuda")
        args = K.make_attend_args(q, out, lse, n_tokens=rows, scale=1.0, softcap=softcap)
        side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
        K.kv_attn_plan_set(plan, K.make_seqs(seqs), side)
        torch.cuda.synchronize()
        say("captured infinities, cap", softcap)
        with torch.cuda.graph(graph, stream=side):
            K.kv_attend(plan, 0, args, side)
        for i in range(4):
            c.dev.copy_(caches[i % 2])
            got = []
            for call in (lambda: K.kv_attend(plan, 0, args, torch.cuda.current_stream()), graph.replay):
                out.fill_(3), lse.fill_(3)
                torch.cuda.synchronize()
                call()
                torch.cuda.synchronize()
                got.append((words(out).clone(), words(lse).clone()))
            assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])
            assert torch.isinf(out).any() == (i % 2 == 0) and not torch.isnan(out).any()
