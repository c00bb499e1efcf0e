"""Rotated appends, reads and shifts of sizes at which a workgroup takes more tokens or layers, and regions past 32 bits
of bytes."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import rotated_reference as rot
from paged_layout_transfer_amd import kvxfer as K
from rotated_harness import KIND, TYPES, Cache, deal, frequencies, say, seqs_of
from test_gpu_rotate import append_case, new_tokens, shift_case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("with_q", [True, False])
@pytest.mark.parametrize("store", ["bf16", "mx4"])
def test_a_long_prompt(store, with_q):
    """More than 512 runs of eight tokens, the last one short."""
    with Cache(heads=2, dim=64, page=16, blocks=280, kind="bf16", cache=store) as c:
        append_case(c, [(4133, 4133), (9, 25), (1, 1)], 4, frequencies(32), with_q=with_q)


def test_a_long_prompt_without_a_rotation():
    """kv_append_tokens into a 4-bit pool: the values' own rounding."""
    lens = [(4133, 4140), (5, 5)]
    with Cache(heads=3, dim=96, page=16, blocks=280, kind="f16", cache="mx4", pad=16) as c:
        tables = deal(c, lens)
        seqs, rows = seqs_of([t.cuda() for t in tables], lens)
        x = new_tokens(rows, 3, 3, 96, "f16", 8)
        x_d = x.cuda()
        plan = c.plan(3, 2, rows)
        K.kv_attn_plan_set(plan, K.make_seqs(seqs), None)
        torch.cuda.synchronize()
        say("append of", rows)
        K.kv_append_tokens(plan, 0, K.make_append_args(x_d[:, 3:6], x_d[:, 6:], n_tokens=rows), None)
        assert K.kv_pool_get_error(c.handle) == 0
        at = 0
        for t, (q, n) in zip(tables, lens):
            for region, first in ((0, 3), (1, 6)):
                old = c.rows(region, t, np.arange(n - q, n))
                packed = rot.pack(*rot.mx4_of(x[at:at + q, first:first + 3].double()), c.row)
                packed[..., 51:] = old[..., 51:]
                c.put(region, t, np.arange(n - q, n), packed)
            at += q
        assert torch.equal(c.now()[0], c.bytes)


@pytest.mark.parametrize("store", ["bf16", "e4m3", "mx4"])
@pytest.mark.parametrize("both", [True, False])
def test_reads_of_many_layers(store, both):
    """A workgroup takes some layers of its tokens; the last takes what is left."""
    layers, lens = 7, [(1501, 1501), (700, 1000), (1, 3)]
    with Cache(layers=layers, heads=2, dim=64, page=16, blocks=170, head_major=both, kind="bf16", cache=store) as c:
        tables = deal(c, lens)
        seqs, rows = seqs_of([t.cuda() for t in tables], lens)
        plan = c.plan(2, len(lens), rows)
        K.kv_attn_plan_set(plan, K.make_seqs(seqs), None)
        k, v = (torch.full((layers - 1, rows + 1, 2, 64), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        torch.cuda.synchronize()
        say("read", store, "layers", layers - 1, "rows", rows)
        K.kv_read_tokens(plan, 1, layers, K.make_read_args(k if both else None, v, n_tokens=rows + 1, k_scale=c.k_scale,
                                                           v_scale=c.v_scale), None)
        assert K.kv_pool_get_error(c.handle) == 0
        for region, got, scale in ((0, k, c.k_scale), (1, v, c.v_scale)):
            if region == 0 and not both:
                assert (got == 7).all()
                continue
            assert (got[:, rows:] == 7).all()
            for layer in range(1, layers):
                y = torch.cat([c.values(c.rows(2 * layer + region, t, np.arange(n - q, n))) for t, (q, n) in zip(tables, lens)])
                x = got[layer - 1, :rows].cpu().double()
                if store == "e4m3":     # the product in 32 bits, then the type's rounding
                    assert ((x - y * scale).abs() <= (y * scale).abs() * (2.0 ** -8 + 2.0 ** -23)).all()
                else:
                    assert torch.equal(torch.nan_to_num(x, 2.0 ** 100), torch.nan_to_num(y, 2.0 ** 100).to(torch.bfloat16).double())


@pytest.mark.parametrize("adjacent", [False, True], ids=["halves", "adjacent"])
@pytest.mark.parametrize("store", ["bf16", "e4m3", "mx4"])
@pytest.mark.parametrize("heads,dim,pairs", [(2, 64, 32), (1, 96, 12)])
def test_shifts_of_many_layers(store, adjacent, heads, dim, pairs):
    """A workgroup takes some layers of its tokens; the last takes what is left."""
    with Cache(layers=12, heads=heads, dim=dim, page=16, blocks=280, kind="bf16", cache=store, pad=16) as c:
        shift_case(c, [(0, 3001, 12345), (5, 1300, -7)], frequencies(pairs), adjacent, (1, 12))


@pytest.mark.parametrize("store", ["bf16", "e4m3", "mx4"])
def test_regions_past_32_bits_of_bytes(store):
    """Block ids whose pages lie over 4 GiB into their region give the bytes that near pages give."""
    H, D, page = 2, 128, 16
    with Cache(heads=H, dim=D, page=page, blocks=8, kind="bf16", cache=store) as c:
        stride = c.stride
        blocks = (5 << 30) // stride
        big = torch.zeros(2, blocks * stride, dtype=torch.uint8, device="cuda")
        near, far = torch.arange(8), blocks - 1 - 5 * torch.arange(8)
        pages = big.view(2, blocks, stride)
        pages[:, far.cuda()] = c.dev[:, near.cuda()]
        pool = K.kv_pool_create(K.make_pool_desc(1, 2, H, c.row // c.wide, c.wide, page, blocks, stride, [big[0], big[1]]))
        plan = K.kv_attn_plan_create(pool, K.make_attn_desc(4, K.KV_TYPE_BF16, KIND[store], 1, 128))
        r = c.rotation(frequencies(64))
        x = new_tokens(100, 4, H, D, "bf16", 3).cuda()
        q, k, v = x.split([4, H, H], dim=1)
        got = []
        try:
            for p, h, ids in ((c.plan(4, 1, 128), c.handle, near), (plan, pool, far)):
                table = ids.int().cuda()
                out, read = torch.zeros_like(q), torch.zeros(2, 100, H, D, dtype=torch.bfloat16, device="cuda")
                K.kv_attn_plan_set(p, K.make_seqs([(table, 8, 125, 0, 100)]), None)
                torch.cuda.synchronize()
                say("pages", int(ids[-1]), "of", stride, "bytes,", store)
                K.kv_append_rotated(p, 0, r, K.make_rotate_args(q, out), K.make_append_args(
                    k, v, n_tokens=103, k_scale=c.k_scale, v_scale=c.v_scale), None)
                K.kv_rotate_cached(h, r, KIND[store], K.make_shifts([(table, 8, 3, 120, -50)]), 0, 1, None)
                K.kv_read_tokens(p, 0, 1, K.make_read_args(read[0], read[1], n_tokens=100, k_scale=c.k_scale,
                                                           v_scale=c.v_scale), None)
                torch.cuda.synchronize()
                assert K.kv_pool_get_error(h) == 0
                got.append((out.view(torch.int16), read.view(torch.int16)))
            assert all(torch.equal(a, b) for a, b in zip(*got)) and got[0][1].any()
            assert torch.equal(pages[:, far.cuda()], c.dev[:, near.cuda()])
            pages[:, far.cuda()] = 0
            assert not big[:, -64 * stride:].any() and not big[:, :64 * stride].any()
        finally:
            torch.cuda.synchronize()
            K.kv_attn_plan_destroy(plan)
            K.kv_pool_destroy(pool)
