"""Rotated appends, shifts and reads at the ends of their ranges on the GPU, against the same plain 64-bit implementations
as tests/test_gpu_rotate.py.  Every case is printed before its first launch."""
from __future__ import annotations

import math

import numpy as np
import pytest
import torch

import rotated_reference as rot
from paged_layout_transfer_amd import kvxfer as K
from rotated_harness import KIND, TYPES, Cache, check_between, deal, frequencies, round_to, say, seqs_of
from test_gpu_rotate import SPECIAL, append_case, shift_case

pytestmark = pytest.mark.gpu

MOST = 7 * 2.0 ** 127       # what the largest scale holds; turned keys may pass it, and are cut to it


@pytest.fixture
def cut(monkeypatch):
    """The 4-bit reference with finite values cut to the largest scale's."""
    plain = rot.mx4_of
    monkeypatch.setattr(rot, "mx4_of", lambda x: plain(torch.where(torch.isfinite(x), x.double().clamp(-MOST, MOST), x.double())))


# ---- 4-bit groups that a turn makes larger than 32 bits hold ------------------------------------

@pytest.mark.parametrize("adjacent", [False, True], ids=["halves", "adjacent"])
@pytest.mark.parametrize("amplitude", [1.0, 1.5, 2.0 ** 20, 3e38])
@pytest.mark.parametrize("kind", ["bf16", "f16"])
def test_turned_keys_past_the_range_of_32_bits(kind, amplitude, adjacent, cut):
    """Keys up to the type's largest in groups with small and zero ones, infinities and NaN in others: 4-bit rows bit by bit."""
    lens = [(40, 43)]
    gen = torch.Generator().manual_seed(6)
    most = torch.finfo(TYPES[kind]).max
    x = torch.randn((43, 4 + 2 * 2, 64), generator=gen) * (most / 3)
    x[::3] *= torch.exp2(-torch.randint(0, 20, x[::3].shape, generator=gen).float())
    x[1::5, :, :32] = most
    x[2::5, :, 32:] = -most
    x[3, :, 7], x[8, :, 40], x[13, :, 0] = math.inf, -math.inf, math.nan
    x[18:20, :, ::2] = 0.0
    x = x.clamp(-most, most).to(TYPES[kind])
    x[3, :, 7], x[8, :, 40] = math.inf, -math.inf
    with Cache(heads=2, dim=64, blocks=8, kind=kind) as c:
        append_case(c, lens, 4, frequencies(32), adjacent=adjacent, amplitude=float(np.float32(amplitude)), x=x, with_q=False)


@pytest.mark.parametrize("pairs", [32, 12])
@pytest.mark.parametrize("adjacent", [False, True], ids=["halves", "adjacent"])
@pytest.mark.parametrize("top", [251, 252, 253, 254])
def test_shifts_of_the_largest_scales(top, adjacent, pairs, cut):
    """Groups up to each of the largest scales, whose values or whose turned values 32 bits do not hold, and NaN groups."""
    with Cache(layers=2, heads=3, dim=64, page=16, blocks=12, gain=2.0 ** (top - 127)) as c:
        c.view(0)[3, 5, 1, 32] = 255
        c.view(2)[:, ::7, 0, 33] = 255
        c.view(0)[:, 1::7, :, 32] = 0
        c.upload()
        shift_case(c, [(0, 61, 5), (3, 4, -77777), (7, 40, 2 ** 31 - 1), (0, 16, 0)], frequencies(pairs), adjacent, (0, 2))


@pytest.mark.parametrize("adjacent", [False, True], ids=["halves", "adjacent"])
@pytest.mark.parametrize("kind", ["bf16", "f16"])
def test_special_values_of_a_turned_group(kind, adjacent, cut):
    """The groups at the edges of the format, as keys that turn."""
    extra = [[2.0 ** -126 * i for i in range(32)], [3e38, -3e38] + [1e37] * 30, [2.0 ** 100] * 32,
             [3.3e38] * 32, [3.3e38 * (-1) ** i for i in range(32)]] if kind == "bf16" else []
    groups = torch.tensor(SPECIAL + extra)
    rows = len(groups)
    x = torch.zeros(rows + 3, 6, 64)
    x[:rows, 2, :32], x[:rows, 2, 32:] = groups, groups.flip(0)
    x[:rows, 3, :32], x[:rows, 3, 32:] = groups.flip(0), groups * 0.5
    x[:rows, 4], x[:rows, 5] = x[:rows, 2].flip(1), x[:rows, 3].flip(1)
    x = x.to(TYPES[kind])
    for pairs in (32, 16, 4):
        with Cache(heads=2, dim=64, blocks=8, kind=kind) as c:
            append_case(c, [(rows, rows + 3)], 2, frequencies(pairs), adjacent=adjacent, x=x, with_q=False)


# ---- the slowest frequencies ---------------------------------------------------------------------

@pytest.mark.parametrize("adjacent", [False, True], ids=["halves", "adjacent"])
@pytest.mark.parametrize("kind", ["bf16", "f16"])
def test_pairs_of_the_slowest_frequencies_turn(kind, adjacent):
    """Pairs (x, 0): the second element becomes x sin a, good relative to itself.  Before the rounding to the type: the
    frequency as a fraction of 64 bits (a half of 2^-64 turns of 1.6e-12 or more: 2^-25), the two parts of the rest, their sum and
    its product with 2 pi / 2^32 (4 * 2^-24 with that constant's rounding), the series' last step and the product (2 * 2^-24):
    under 2^-21 in all."""
    n, t = 8, TYPES[kind]
    freq = [1e-11, 3e-11, 1e-10, 7e-10, 1e-9, 2e-8, 5e-7, 3e-6] if kind == "bf16" else [3e-9, 1e-8, 2e-8, 1e-7, 3e-7, 1e-6, 3e-6, 1e-5]
    first = list(range(0, 2 * n, 2)) if adjacent else list(range(n))
    second = [i + 1 for i in first] if adjacent else [i + n for i in first]
    gen = torch.Generator().manual_seed(8)
    x = torch.zeros(60, 4, 32)
    x[:, :, first] = (torch.rand((60, 4, n), generator=gen) + 1) * (1 if kind == "bf16" else 30000)
    x = x.to(t)
    pos = [int(p) for p in torch.randint(-300, 300, (60,), generator=gen)]
    pos[:4] = [1, -1, 2, 0]
    with Cache(heads=1, dim=32, blocks=8, kind=kind, cache=kind) as c:
        table = torch.arange(8, dtype=torch.int32).cuda()
        plan, r = c.plan(2, 1, 60), c.rotation(freq, adjacent)
        K.kv_attn_plan_set(plan, K.make_seqs([(table, 8, 60, 0, 60)]), None)
        x_d, pos_d = x.cuda(), torch.tensor(pos, dtype=torch.int32).cuda()
        out, k, moved = (torch.zeros(60, h, 32, dtype=t, device="cuda") for h in (2, 1, 1))
        torch.cuda.synchronize()
        say("slow pairs", kind, "adjacent", adjacent)
        K.kv_append_rotated(plan, 0, r, K.make_rotate_args(x_d[:, :2], out, pos_d),
                            K.make_append_args(x_d[:, 2:3], x_d[:, 3:], n_tokens=60), None)
        K.kv_read_tokens(plan, 0, 1, K.make_read_args(k, None, n_tokens=60), None)
        K.kv_append_tokens(plan, 0, K.make_append_args(x_d[:, 2:3], x_d[:, 3:], n_tokens=60), None)
        K.kv_rotate_cached(c.handle, r, KIND[kind], K.make_shifts([(table, 8, 0, 60, -3)]), 0, 1, None)
        K.kv_read_tokens(plan, 0, 1, K.make_read_args(moved, None, n_tokens=60), None)
        torch.cuda.synchronize()
        for got, heads, at in ((out, slice(0, 2), pos), (k, slice(2, 3), pos), (moved, slice(2, 3), [-3])):
            _, sn = rot.turned_by(at, freq)
            y = x[:, heads][..., first].double() * sn[:, None]
            a, b = round_to(y * (1 - 2.0 ** -21), t), round_to(y * (1 + 2.0 ** -21), t)
            check_between(got.cpu()[..., second].double(), torch.minimum(a, b), torch.maximum(a, b), "x sin a")


# ---- reads into arrays of any order ------------------------------------------------------------------

@pytest.mark.parametrize("store", ["bf16", "e4m3", "mx4"])
@pytest.mark.parametrize("order", ["tlhd", "lthd", "thld", "hltd", "htld", "lhtd"])
def test_reads_into_arrays_of_any_order(order, store):
    """[tokens][layers][heads][dim] (the order of page-first chunks) and the others give what [layers][tokens][heads][dim]
    gives, and leave what lies between untouched."""
    lens, L, H, D = [(21, 21), (3, 40), (1, 1)], 3, 2, 64
    with Cache(layers=L, heads=H, dim=D, blocks=8, cache=store) as c:
        tables = [t.cuda() for t in deal(c, lens)]
        seqs, rows = seqs_of(tables, lens)
        plan = c.plan(H, len(lens), rows)
        K.kv_attn_plan_set(plan, K.make_seqs(seqs), None)
        n = rows + 2
        plain = torch.full((2, L, n, H, D), 7.0, dtype=torch.bfloat16, device="cuda")
        # k and v side by side, and eight elements to spare behind each
        sizes = {"t": n, "l": L, "h": H, "d": D + 8}
        both = torch.full([sizes[x] for x in order[:-1]] + [2, D + 8], 7.0, dtype=torch.bfloat16, device="cuda")
        k, v = (both[..., i, :D].permute([order.index(x) for x in "lthd"]) for i in (0, 1))
        torch.cuda.synchronize()
        say("read", order, store)
        scales = dict(n_tokens=n, k_scale=c.k_scale, v_scale=c.v_scale)
        K.kv_read_tokens(plan, 0, L, K.make_read_args(plain[0], plain[1], **scales), None)
        K.kv_read_tokens(plan, 0, L, K.make_read_args(k, v, k_strides=k.stride()[:3], v_strides=v.stride()[:3], **scales), None)
        assert K.kv_pool_get_error(c.handle) == 0
        assert torch.equal(k, plain[0]) and torch.equal(v, plain[1]) and not (plain[:, :, :rows] == 7).all()
        assert (both[..., D:] == 7).all()


def test_reads_into_arrays_that_overlap_are_refused():
    with Cache(layers=2, heads=2, dim=64, blocks=8) as c:
        table = torch.zeros(4, dtype=torch.int32, device="cuda")
        plan = c.plan(2, 1, 8)
        K.kv_attn_plan_set(plan, K.make_seqs([(table, 4, 8, 0, 8)]), None)
        x = torch.zeros(8, 2, 2, 64, dtype=torch.bfloat16, device="cuda")
        say("overlapping reads")
        # (layer, token, head): a layer within a head's step, within a token's, on the heads, behind its own start, nowhere
        for strides, code in (((64, 256, 64), K.KV_ERR_ARG), ((192, 256, 64), K.KV_ERR_ARG), ((56, 256, 64), K.KV_ERR_ARG),
                              ((-128, 256, 64), K.KV_ERR_ARG), ((0, 256, 64), K.KV_ERR_ARG), ((132, 256, 64), K.KV_ERR_ALIGN),
                              ((1 << 40, 256, 64), K.KV_ERR_RANGE), ((1 << 60, 256, 64), K.KV_ERR_ARG)):
            with pytest.raises(K.KvError) as e:
                K.kv_read_tokens(plan, 0, 2, K.make_read_args(x, None, n_tokens=8, k_strides=strides), None)
            assert e.value.code == code, strides
        K.kv_read_tokens(plan, 0, 2, K.make_read_args(x, None, n_tokens=8, k_strides=(128, 256, 64)), None)
        K.kv_read_tokens(plan, 0, 2, K.make_read_args(x, None, n_tokens=8, k_strides=(64, 256, 128)), None)


# ---- the arithmetic of e4m3 reads ----------------------------------------------------------------------

@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("scale", [0.037, 1.0, 1.2345678e-3, 3.0e4])
def test_e4m3_elements_are_read_as_a_32_bit_product_rounded(kind, scale):
    """Every e4m3 code, bit by bit (NaN as NaN)."""
    with Cache(heads=2, dim=64, page=16, blocks=4, kind=kind, cache="e4m3") as c:
        codes = torch.arange(256, dtype=torch.uint8)
        c.bytes.view(2, -1)[:] = codes.repeat(c.bytes[0].numel() // 256)
        c.upload()
        table = torch.arange(4, dtype=torch.int32).cuda()
        plan = c.plan(2, 1, 64)
        K.kv_attn_plan_set(plan, K.make_seqs([(table, 4, 64, 0, 64)]), None)
        k, v = (torch.zeros(64, 2, 64, dtype=TYPES[kind], device="cuda") for _ in range(2))
        torch.cuda.synchronize()
        say("e4m3 read", kind, scale)
        K.kv_read_tokens(plan, 0, 1, K.make_read_args(k, v, n_tokens=64, k_scale=scale, v_scale=scale / 3), None)
        torch.cuda.synchronize()
        values = codes.view(torch.float8_e4m3fn).float().repeat(32)
        for got, by in ((k, scale), (v, scale / 3)):
            want = (values * torch.tensor(by, dtype=torch.float32)).to(TYPES[kind])
            got = got.cpu().flatten()
            assert torch.equal(torch.isnan(got), torch.isnan(want))
            fine = ~torch.isnan(want)
            assert torch.equal(got[fine].view(torch.int16), want[fine].view(torch.int16))


# ---- amplitudes of 4-bit appends -------------------------------------------------------------------------

@pytest.mark.parametrize("adjacent", [False, True], ids=["halves", "adjacent"])
@pytest.mark.parametrize("amplitude", [1.0948, 0.7071, 3.0e-3])
@pytest.mark.parametrize("shape", [(8, 2, 128, 64), (3, 3, 96, 20), (5, 1, 256, 128)])
def test_4_bit_appends_with_an_amplitude(shape, amplitude, adjacent):
    """Bit by bit, the amplitude as the 32-bit number that the descriptor holds."""
    heads_q, heads, dim, pairs = shape
    lens = [(5, 21), (0, 9), (1, 1), (33, 33), (8, 24)]
    for kind in ("bf16", "f16"):
        with Cache(heads=heads, dim=dim, blocks=20, kind=kind, pad=32) as c:
            append_case(c, lens, heads_q, frequencies(pairs, 500000.0), adjacent=adjacent, amplitude=float(np.float32(amplitude)))
