"""The rotated operators together, as a serving program makes them: steps over 4-bit pools, captured and replayed steps,
streams of their own, and 4-bit pools moved by the library's transfers."""
from __future__ import annotations

import math

import numpy as np
import pytest
import torch

import paged_reference as ref
import rotated_reference as rot
from paged_layout_transfer_amd import kvxfer as K
from rotated_harness import KIND, TYPES, Cache, check_between, frequencies, rounded, say, scale_of

pytestmark = pytest.mark.gpu


def words(t):
    return t.contiguous().view(torch.uint8)


class Model:
    """One attention layer after another over a pool; remembers what each cached token was."""

    def __init__(self, cache, heads_q, adjacent=False):
        self.c, self.heads_q, self.adjacent = cache, heads_q, adjacent
        self.freq = frequencies(cache.dim // 2)
        self.rotation = cache.rotation(self.freq, adjacent)
        self.gen = torch.Generator().manual_seed(8)

    def new(self, n):
        c = self.c
        return torch.randn((c.layers, n, self.heads_q + 2 * c.heads, c.dim), generator=self.gen).to(TYPES[c.kind]).cuda()

    def step(self, plan, seqs, x, stream, positions=None):
        """Plan, rotated append, attention, layer by layer; the rotated queries and the results."""
        c, n = self.c, x.shape[1]
        scales = dict(k_scale=c.k_scale, v_scale=c.v_scale)
        q, k, v = x.split([self.heads_q, c.heads, c.heads], dim=2)
        turned, out = torch.zeros_like(q), torch.zeros_like(q)
        if seqs is not None:
            K.kv_attn_plan_set(plan, K.make_seqs(seqs), stream)
        for i in range(c.layers):
            K.kv_append_rotated(plan, i, self.rotation, K.make_rotate_args(q[i], turned[i], positions),
                                K.make_append_args(k[i], v[i], n_tokens=n, **scales), stream)
            K.kv_attend(plan, i, K.make_attend_args(turned[i], out[i], n_tokens=n, scale=scale_of(c.dim), **scales), stream)
        return turned, out


@pytest.mark.parametrize("kind,store", [("bf16", "mx4"), ("f16", "mx4"), ("bf16", "e4m3"), ("f16", "f16")])
@pytest.mark.parametrize("head_major", [False, True])
def test_prompt_decode_drop_the_middle_and_go_on(kind, store, head_major):
    """A prompt in two chunks, decoded tokens, a page dropped from the middle and the keys behind it turned
    back by a page, the next token: after every call the attention is that over the cached values (read back),
    and those are the tokens' own, turned to their places."""
    with Cache(layers=2, heads=2, dim=64, page=16, blocks=40, head_major=head_major, kind=kind, cache=store) as c:
        m, stream = Model(c, 4), torch.cuda.current_stream()
        plan = c.plan(4, 2, 96)
        ids = K.kv_pool_alloc_blocks(c.handle, 8)
        table = torch.from_numpy(ids).cuda()
        known = []      # of each token of the cache: its k and v by layer

        def check(x, turned, out, total):
            n = x.shape[1]
            for i in range(2):
                k, v = x[i, :, 4:6].cpu().double(), x[i, :, 6:].cpu().double()
                known.extend([] if i else [([], []) for _ in range(n)])
                for j in range(n):
                    known[len(known) - n + j][0].append(k[j])
                    known[len(known) - n + j][1].append(v[j])
            # the whole cache, read back
            reader = c.plan(4, 1, 128)
            K.kv_attn_plan_set(reader, K.make_seqs([(table, len(table), total, 0, total)]), stream)
            got = [torch.zeros(2, total, 2, 64, dtype=TYPES[kind], device="cuda") for _ in range(2)]
            K.kv_read_tokens(reader, 0, 2, K.make_read_args(*got, n_tokens=total, k_scale=c.k_scale, v_scale=c.v_scale), stream)
            torch.cuda.synchronize()
            cs, sn = rot.turned_by(range(total - n, total), m.freq)
            for i in range(2):
                kk, vv = (g[i].cpu().double() for g in got)
                want, size = rot.rotate(x[i, :, :4].cpu().double(), cs, sn, False)
                check_between(turned[i].cpu().double(), *rounded(kind, want, size, 1.0), "q")
                want, _, tol, _ = ref.attend(turned[i].cpu().double(), kk, vv, scale=scale_of(64), kind=kind)
                # an e4m3 cache is attended before its scale rounds: half a step of the read values more
                if store == "e4m3":
                    u = torch.finfo(TYPES[kind]).eps / 2
                    tol = tol + 4 * u * (vv.abs().amax() + (turned[i].cpu().double().abs().amax() * kk.abs().amax() * 8 * vv.abs().amax()))
                assert ((out[i].cpu().double() - want).abs() <= tol).all()
            return got

        say("prompt", kind, store)
        for at, n in ((0, 50), (50, 40), (90, 1), (91, 1)):
            x = m.new(n)
            turned, out = m.step(plan, [(table, 8, at + n, 0, n)], x, stream)
            check(x, turned, out, at + n)
        say("drop a page and turn the rest back")
        before = [torch.zeros(2, 92, 2, 64, dtype=TYPES[kind], device="cuda") for _ in range(2)]
        reader = c.plan(4, 1, 128)
        K.kv_attn_plan_set(reader, K.make_seqs([(table, 8, 92, 0, 92)]), stream)
        K.kv_read_tokens(reader, 0, 2, K.make_read_args(*before, n_tokens=92, k_scale=c.k_scale, v_scale=c.v_scale), stream)
        torch.cuda.synchronize()
        K.kv_pool_free_blocks(c.handle, ids[2:3])
        table = torch.from_numpy(np.delete(ids, 2)).cuda()
        del known[32:48]
        K.kv_rotate_cached(c.handle, m.rotation, KIND[store], K.make_shifts([(table, 7, 32, 76, -16)]), 0, 2, stream)
        x = m.new(1)
        turned, out = m.step(plan, [(table, 7, 77, 0, 1)], x, stream)
        after = check(x, turned, out, 77)
        cs, sn = rot.turned_by([-16], m.freq)
        for i in range(2):
            assert torch.equal(words(after[0][i, :32]), words(before[0][i, :32]))
            assert torch.equal(words(after[1][i, 32:76]), words(before[1][i, 48:92]))
            old = before[0][i, 48:92].cpu().double()
            want, size = rot.rotate(old, cs.expand(44, -1), sn.expand(44, -1), False)
            g = after[0][i, 32:76].cpu().double()
            # one more rounding of the cache's type (and, read back, of e4m3's scale): half a step each
            step = {"mx4": None, "e4m3": 2.0 ** -4, "f16": 2.0 ** -11}[store]
            if step is None:
                codes, e = rot.mx4_of(want)
                assert torch.equal(g, rot.unpack(rot.pack(codes, e, 40), 64))
            else:
                assert ((g - want).abs() <= want.abs() * step * 1.01 + size * 2.0 ** -7 * (store == "e4m3") + size * 2.0 ** -20 +
                        2.0 ** -9 * c.k_scale * (store == "e4m3")).all()
        # and the tokens are their own: 4-bit groups within half a step of their largest, and another turn's
        cs, sn = rot.turned_by(range(77), m.freq)
        worst = {"mx4": 0.5, "e4m3": 2.0 ** -2, "f16": 2.0 ** -8}[store]
        for i in range(2):
            own = torch.stack([t[0][i] for t in known])
            want, size = rot.rotate(own, cs, sn, False)
            most = size.amax(-1, keepdim=True)
            assert ((after[0][i].cpu().double() - want).abs() <= worst * most).all()
        assert K.kv_pool_get_error(c.handle, stream) == 0


@pytest.mark.parametrize("store", ["bf16", "e4m3", "mx4"])
def test_captured_steps_are_replayed_on_other_plans(store):
    """A graph of a rotated append, a read, a shift and an attention: replays on what the last set gave, with the
    program's own work between them, give the bits of the same calls made eagerly."""
    with Cache(layers=1, heads=2, dim=64, page=16, blocks=64, cache=store) as c, \
            Cache(layers=1, heads=2, dim=64, page=16, blocks=64, cache=store) as e:
        stream = torch.cuda.Stream()
        rows = 48
        ms = [Model(c, 4), Model(e, 4)]
        plans = [x.plan(4, 4, rows) for x in (c, e)]
        x = torch.zeros(1, rows, 8, 64, dtype=torch.bfloat16, device="cuda")
        pos = torch.zeros(rows, dtype=torch.int32, device="cuda")
        table = torch.randperm(64, generator=torch.Generator().manual_seed(1)).int().cuda().view(4, 16)
        shift = K.make_shifts([(table[3], 16, 40, 100, 77)])
        out = [{k: torch.zeros(1, rows, n, 64, dtype=torch.bfloat16, device="cuda") for k, n in
                (("q", 4), ("out", 4), ("k", 2), ("v", 2))} for _ in range(2)]

        def calls(i, s):
            cc, o, scales = (c, e)[i], out[i], dict(k_scale=c.k_scale, v_scale=c.v_scale)
            K.kv_append_rotated(plans[i], 0, ms[i].rotation, K.make_rotate_args(x[0, :, :4], o["q"][0], pos),
                                K.make_append_args(x[0, :, 4:6], x[0, :, 6:], n_tokens=rows, **scales), s)
            K.kv_attend(plans[i], 0, K.make_attend_args(o["q"][0], o["out"][0], n_tokens=rows, scale=0.125, **scales), s)
            K.kv_rotate_cached(cc.handle, ms[i].rotation, KIND[store], shift, 0, 1, s)
            K.kv_read_tokens(plans[i], 0, 1, K.make_read_args(o["k"], o["v"], n_tokens=rows, **scales), s)

        first = K.make_seqs([(table[0], 16, 33, 0, 1)])
        for i in range(2):
            K.kv_attn_plan_set(plans[i], first, stream)
        torch.cuda.synchronize()
        say("capture", store)
        with torch.cuda.stream(stream):
            calls(0, stream), calls(1, stream)      # once outside: the device state is there
            stream.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=stream):
                calls(0, stream)
        steps = [[(1, 34), (1, 60)], [(20, 70), (0, 9), (5, 5)], [(1, 1), (1, 200), (16, 48), (30, 100)], [(48, 60)], []]
        gen = torch.Generator().manual_seed(2)
        for step in steps:
            with torch.cuda.stream(stream):
                x.copy_(torch.randn(x.shape, generator=gen))
                pos.copy_(torch.randint(-1000, 100000, (rows,), generator=gen, dtype=torch.int32))
                at, seqs = 0, []
                for i, (q, n) in enumerate(step):
                    seqs.append((table[i], 16, n, at, q))
                    at += q
                for p in plans:
                    K.kv_attn_plan_set(p, K.make_seqs(seqs), stream)
                graph.replay()
                calls(1, stream)
            torch.cuda.synchronize()
            for name in out[0]:
                assert torch.equal(words(out[0][name]), words(out[1][name])), (step, name)
            assert torch.equal(c.dev, e.dev), step
            torch.ones(1 << 20, device="cuda").sum().item()
        assert K.kv_pool_get_error(c.handle, stream) == 0
        del graph


def test_calls_that_cannot_be_captured_are_refused():
    with Cache(heads=2, dim=64, blocks=64) as c, Cache(heads=2, dim=64, blocks=64, seed=1) as fresh:
        r = c.rotation(frequencies(32))
        table = torch.arange(16, dtype=torch.int32, device="cuda")
        stream = torch.cuda.Stream()
        K.kv_rotate_cached(c.handle, r, K.KV_TYPE_MX4, K.make_shifts([(table, 16, 0, 3, 5)]), 0, 1, stream)
        one, many = K.make_shifts([(table, 16, 3, 9, 5)]), K.make_shifts([(table, 16, 3 * i, 3 * i + 2, 5) for i in range(65)])
        torch.cuda.synchronize()
        say("refused while a stream captures")
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.stream(stream), torch.cuda.graph(graph, stream=stream):
            for pool, shifts in ((c, many), (fresh, one)):
                with pytest.raises(K.KvError) as e:
                    K.kv_rotate_cached(pool.handle, r, K.KV_TYPE_MX4, shifts, 0, 1, stream)
                assert e.value.code == K.KV_ERR_CAPTURE
            K.kv_rotate_cached(c.handle, r, K.KV_TYPE_MX4, one, 0, 1, stream)
        torch.cuda.synchronize()
        before, _ = c.now()
        graph.replay()
        torch.cuda.synchronize()
        now, _ = c.now()
        assert not torch.equal(now, before)
        del graph


def test_two_streams_and_a_rotation_destroyed_behind_its_calls():
    """Pools and plans on streams of their own share one rotation; destroying it waits for the calls that read it."""
    with Cache(heads=2, dim=128, blocks=300, seed=1) as a, Cache(heads=2, dim=128, blocks=300, seed=2) as b:
        lens = [(40, 4000)]
        streams = [torch.cuda.Stream() for _ in range(2)]
        r = K.kv_rotation_create(K.make_rotation_desc(frequencies(64)))
        x = torch.randn(40, 8, 128, device="cuda").bfloat16()
        table = torch.arange(300, dtype=torch.int32, device="cuda")
        big = torch.ones(1 << 26, device="cuda")
        outs, want = [], []
        torch.cuda.synchronize()
        say("two streams")
        for c, s in zip((a, b), streams):
            plan = c.plan(4, 1, 40)
            turned, out = torch.zeros_like(x[:, :4]), torch.zeros_like(x[:, :4])
            torch.cuda.synchronize()
            with torch.cuda.stream(s):
                for _ in range(10):
                    big.mul_(1.0)
            K.kv_attn_plan_set(plan, K.make_seqs([(table, 300, 4000, 0, 40)]), s)
            K.kv_append_rotated(plan, 0, r, K.make_rotate_args(x[:, :4], turned), K.make_append_args(x[:, 4:6], x[:, 6:], n_tokens=40), s)
            K.kv_attend(plan, 0, K.make_attend_args(turned, out, n_tokens=40, scale=0.1), s)
            outs.append((turned, out, plan))
        K.kv_rotation_destroy(r)
        assert all(s.query() for s in streams)
        q = x.cpu().double()
        cs, sn = rot.turned_by(range(3960, 4000), frequencies(64))
        turned, size = rot.rotate(q[:, :4], cs, sn, False)
        new_k, _ = rot.rotate(q[:, 4:6], cs, sn, False)
        for c, (t, out, _) in zip((a, b), outs):
            check_between(t.cpu().double(), *rounded("bf16", turned, size, 1.0), "q")
            j = np.arange(4000)
            tab = torch.arange(300)
            k, v = (c.values(c.rows(i, tab, j)) for i in (0, 1))
            k[3960:] = rot.unpack(rot.pack(*rot.mx4_of(new_k), 72), 128)
            v[3960:] = rot.unpack(rot.pack(*rot.mx4_of(q[:, 6:]), 72), 128)
            ref_out, _, tol, _ = ref.attend(t.cpu().double(), k, v, scale=0.1)
            assert ((out.cpu().double() - ref_out).abs() <= tol).all()


@pytest.mark.parametrize("head_major", [False, True])
def test_a_4_bit_pool_is_offloaded_and_reloaded(head_major):
    """Gathered into chunks and scattered into other pages of another pool: the next token's attention has the same bits."""
    with Cache(layers=2, heads=4, dim=64, page=16, blocks=40, head_major=head_major, row=36) as c, \
            Cache(layers=2, heads=4, dim=64, page=16, blocks=40, head_major=not head_major, row=36, seed=9) as d:
        tok = 4 * 36
        src, dst = (torch.from_numpy(np.random.default_rng(i).permutation(40)[:20].astype(np.int32)).cuda() for i in (1, 2))
        n, stream = 300, torch.cuda.current_stream()
        slot = 2 * 2 * 320 * tok
        chunk = torch.zeros(slot, dtype=torch.uint8, device="cuda")
        spec = K.make_chunk_spec(K.KV_LAYER_FIRST, 2, 320, 0, 2, chunk, slot, 1)
        torch.cuda.synchronize()
        say("offload and reload")
        K.kv_gather_chunks(c.handle, K.make_spans([(src, 20, 0, n, 0)]), spec, stream)
        K.kv_scatter_chunks(d.handle, K.make_spans([(dst, 20, 0, n, 0)]), spec, stream)
        x = torch.randn(1, 16, 64, device="cuda").bfloat16()
        outs = []
        for cache, table in ((c, src), (d, dst)):
            m, plan = Model(cache, 8), cache.plan(8, 1, 1)
            outs.append(m.step(plan, [(table, 20, n + 1, 0, 1)], x.expand(2, 1, 16, 64).contiguous(), stream)[1])
        torch.cuda.synchronize()
        assert (outs[0] != 0).any() and torch.equal(words(outs[0]), words(outs[1]))


def test_compaction_of_a_4_bit_pool_changes_no_answer():
    with Cache(layers=2, heads=2, dim=128, page=16, blocks=64) as c:
        m, stream = Model(c, 8), torch.cuda.current_stream()
        plan = c.plan(8, 2, 2)
        K.kv_pool_alloc_blocks(c.handle, 30)
        ids = K.kv_pool_alloc_blocks(c.handle, 20)
        K.kv_pool_free_blocks(c.handle, list(range(30)))
        tables = torch.from_numpy(ids.reshape(2, 10)).cuda()
        x = m.new(2)
        seqs = lambda: [(tables[i], 10, 140 + i, i, 1) for i in range(2)]      # noqa: E731
        want = m.step(plan, seqs(), x, stream)
        moves = K.kv_pool_plan_compact(c.handle, 64)
        assert moves._n == 20
        say("compact")
        K.kv_copy_pages(c.handle, moves, 0, 2, stream)
        K.kv_remap_tables(c.handle, moves, tables, tables, 20, stream)
        torch.cuda.synchronize()
        K.kv_pool_free_blocks(c.handle, [mv.src for mv in moves[:moves._n]])
        c.dev[:, 20:] = 0xff
        got = m.step(plan, seqs(), x, stream)
        torch.cuda.synchronize()
        assert int(tables.max()) < 20
        for a, b in zip(got, want):
            assert (b != 0).any() and torch.equal(words(a), words(b))


def test_the_same_call_gives_the_same_bits():
    with Cache(heads=2, dim=128, page=16, blocks=700) as c:
        m, stream = Model(c, 8), torch.cuda.current_stream()
        plan = c.plan(8, 2, 65)
        table = torch.randperm(700, generator=torch.Generator().manual_seed(3)).int().cuda()
        x = m.new(65)
        seqs = [(table[:600], 600, 9000, 0, 1), (table[600:], 100, 1500, 1, 64)]
        say("twice the same")
        runs = [m.step(plan, seqs, x, stream) for _ in range(3)]
        torch.cuda.synchronize()
        for a, b in zip(runs[0], runs[1]):
            assert torch.equal(words(a), words(b))
        for a, b in zip(runs[0], runs[2]):
            assert torch.equal(words(a), words(b))
