"""Host side of rotations and 4-bit pools (no GPU): sizes, and the arguments each entry point refuses before it
needs a device."""
from __future__ import annotations

import ctypes
import math

import numpy as np
import pytest
import torch

import rotated_reference as rot
from paged_layout_transfer_amd import kvxfer as K

FAKE = 0x7F0000000000


def _pool(N=64, bs=16, H=2, R=72, E=1, KV=2, L=2, page_layout=0):
    tok = H * R * E
    return K.kv_pool_create(K.make_pool_desc(L, KV, H, R, E, bs, N, bs * tok,
                                             [FAKE + i * (1 << 30) for i in range(L * KV)], page_layout))


def _refused(code, fn, *args):
    with pytest.raises(K.KvError) as e:
        fn(*args)
    assert e.value.code == code


@pytest.mark.parametrize("dim", range(32, 257, 32))
@pytest.mark.parametrize("heads", [1, 2, 3, 4, 5, 8, 16])
def test_row_bytes_make_tokens_of_whole_vectors(dim, heads):
    row = K.kv_mx4_row_bytes(dim, heads)
    assert row == rot.row_bytes(dim, heads)
    assert row % 4 == 0 and row * heads % 16 == 0 and row // 17 * 32 == dim
    assert not any(r * heads % 16 == 0 for r in range(-(-dim * 17 // 32 // 4) * 4, row, 4))
    K.kv_pool_destroy(_pool(H=heads, R=row))
    K.kv_pool_destroy(_pool(H=heads, R=row, page_layout=K.KV_PAGE_HEAD_MAJOR))


@pytest.mark.parametrize("dim,heads", [(0, 1), (-32, 1), (16, 1), (33, 1), (288, 1), (128, 0), (128, -1)])
def test_row_bytes_refusals(dim, heads):
    _refused(K.KV_ERR_ARG, K.kv_mx4_row_bytes, dim, heads)


def _desc(heads=8, q=K.KV_TYPE_BF16, kv=K.KV_TYPE_MX4, seqs=4, tokens=64, window=0, flags=0):
    return K.make_attn_desc(heads, q, kv, seqs, tokens, window, flags)


@pytest.mark.parametrize("pool,desc,code", [
    (dict(), dict(q=K.KV_TYPE_MX4), K.KV_ERR_ARG),
    (dict(), dict(kv=4), K.KV_ERR_ARG),
    (dict(), dict(kv=-1), K.KV_ERR_ARG),
    (dict(E=2), dict(), K.KV_ERR_ARG),                  # elements of two bytes
    (dict(R=16), dict(), K.KV_ERR_ARG),                 # no group
    (dict(R=160), dict(), K.KV_ERR_ARG),                # 9 groups: 288 wide
    (dict(H=16, R=71), dict(heads=16), K.KV_ERR_ALIGN),
    (dict(KV=1), dict(), K.KV_ERR_ARG),
    (dict(), dict(heads=3), K.KV_ERR_ARG),
    (dict(R=1 << 26, H=1, N=1, bs=1), dict(), K.KV_ERR_ARG),
    (dict(R=68, H=1 << 20, N=1, bs=1), dict(heads=1 << 20, tokens=1), K.KV_ERR_ARG),    # 2^28 elements of a token
])
def test_plan_refusals(pool, desc, code):
    p = _pool(**pool)
    _refused(code, K.kv_attn_plan_create, p, _desc(**desc))
    K.kv_pool_destroy(p)


@pytest.mark.parametrize("kw,code", [
    (dict(inv_freq=[]), K.KV_ERR_ARG),
    (dict(inv_freq=[0.1] * 132), K.KV_ERR_ARG),
    (dict(inv_freq=[0.1] * 6), K.KV_ERR_ALIGN),
    (dict(inv_freq=[0.1] * 3), K.KV_ERR_ALIGN),
    (dict(inv_freq=[0.1] * 4, pairing=2), K.KV_ERR_ARG),
    (dict(inv_freq=[0.1] * 4, pairing=-1), K.KV_ERR_ARG),
    (dict(inv_freq=[0.1] * 4, amplitude=0.0), K.KV_ERR_ARG),
    (dict(inv_freq=[0.1] * 4, amplitude=-1.0), K.KV_ERR_ARG),
    (dict(inv_freq=[0.1] * 4, amplitude=math.inf), K.KV_ERR_ARG),
    (dict(inv_freq=[0.1] * 4, amplitude=math.nan), K.KV_ERR_ARG),
    (dict(inv_freq=[0.1, 0.1, math.nan, 0.1]), K.KV_ERR_ARG),
    (dict(inv_freq=[0.1, 0.1, math.inf, 0.1]), K.KV_ERR_ARG),
    (dict(inv_freq=[0.1, 0.1, -0.1, 0.1]), K.KV_ERR_ARG),
    (dict(inv_freq=[0.1, 0.1, 2.0 ** 20 + 1, 0.1]), K.KV_ERR_ARG),
])
def test_rotation_refusals(kw, code):
    _refused(code, K.kv_rotation_create, K.make_rotation_desc(**kw))


def test_null_handles():
    assert K._lib.kv_rotation_destroy(None) == K.KV_OK
    assert K._lib.kv_rotation_create(None, None) == K.KV_ERR_ARG
    h = ctypes.c_void_p(7)
    assert K._lib.kv_rotation_create(None, ctypes.byref(h)) == K.KV_ERR_ARG and h.value is None
    none = K.kv_rotation_desc(4, 0, 1.0, None)
    assert K._lib.kv_rotation_create(ctypes.byref(none), ctypes.byref(h)) == K.KV_ERR_ARG
    assert K._lib.kv_append_rotated(None, 0, None, None, None, None) == K.KV_ERR_ARG
    assert K._lib.kv_read_tokens(None, 0, 1, None, None) == K.KV_ERR_ARG
    assert K._lib.kv_rotate_cached(None, None, 0, None, 0, 0, 1, None) == K.KV_ERR_ARG
    p = _pool()
    assert K._lib.kv_rotate_cached(p, None, K.KV_TYPE_MX4, None, 0, 0, 1, None) == K.KV_ERR_ARG
    assert K._lib.kv_mx4_row_bytes(64, 1, None) == K.KV_ERR_ARG
    K.kv_pool_destroy(p)


def test_row_arrays_need_packed_heads():
    x = torch.zeros(2, 4, 2, 8, 2)[..., 0]
    for make in (lambda: K.make_rotate_args(x[0], x[0]), lambda: K.make_read_args(x, x, n_tokens=4),
                 lambda: K.make_read_args(x[0], None, n_tokens=4)):
        with pytest.raises(ValueError):
            make()


def test_descriptors_hold_what_they_are_given():
    k = torch.zeros(3, 5, 2, 8)
    a = K.make_read_args(k, None, n_tokens=5)
    assert (a.k_layer_stride, a.k_token_stride, a.k_head_stride, a.v) == (80, 16, 8, None)
    a = K.make_read_args(None, k[0], n_tokens=5)
    assert (a.v_layer_stride, a.v_token_stride, a.v_head_stride, a.k) == (0, 16, 8, None)
    d = K.make_rotation_desc(np.array([1.0, 0.5, 0.25, 0.125]), K.KV_ROT_ADJACENT, 1.5)
    assert (d.pairs, d.pairing, d.amplitude, d.inv_freq[2]) == (4, 1, 1.5, 0.25)
    s = K.make_shifts([(FAKE, 7, 3, 9, -5)])
    assert (s._n, s[0].block_table, s[0].table_len, s[0].t_begin, s[0].t_end, s[0].delta) == (1, FAKE, 7, 3, 9, -5)


def test_the_reference_rounds_to_nearest():
    """The 4-bit reference against every value a group can hold, and its ties."""
    for k in (-20, 0, 30):
        x = torch.tensor([g * 2.0 ** k for g in rot.GRID] + [-g * 2.0 ** k for g in rot.GRID] + [0.0] * 16).double()
        codes, e = rot.mx4_of(x)
        assert e.item() == 127 + k and (rot.unpack(rot.pack(codes, e, 20), 32) == x).all()
        ties = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.0, 6.999] + [0.0] * 23).double() * 2.0 ** k
        codes, e = rot.mx4_of(ties)
        assert e.item() == 127 + k and codes[:9].tolist() == [0, 2, 2, 4, 4, 6, 6, 7, 7]
        over = torch.tensor([7.0000001] + [0.0] * 31, dtype=torch.float64) * 2.0 ** k
        assert rot.mx4_of(over)[1].item() == 128 + k
    c, s = rot.turned_by([0, 1, -3, 2 ** 31 - 1], [1.0, 0.25, 2.0 ** -40])
    assert torch.allclose(c[:3], torch.cos(torch.tensor([[0.0], [1], [-3]]).double() * torch.tensor([1.0, 0.25, 2.0 ** -40]).double()),
                          rtol=0, atol=1e-15)
    assert torch.allclose(c * c + s * s, torch.ones_like(c), rtol=0, atol=1e-15)


def test_plans_over_4_bit_pools_walk_every_visible_key_once(tmp_path):
    """tests/plan_walk_mx4.cpp under AddressSanitizer and UBSan (host code only)."""
    import os
    import subprocess

    from paged_layout_transfer_amd import _build

    rocm = os.path.dirname(os.path.dirname(os.path.realpath(_build.HIPCC)))
    out = str(tmp_path / "plan_walk_mx4")
    subprocess.run(["g++", "-std=c++17", "-O2", "-g", "-Wall", "-fsanitize=address,undefined",
                    "-fno-sanitize-recover=undefined", "-D__HIP_PLATFORM_AMD__", "-I", os.path.join(rocm, "include"),
                    "-I", os.path.join(_build.ROOT, "include"), "-I", _build.CSRC,
                    os.path.join(os.path.dirname(__file__), "plan_walk_mx4.cpp"), "-o", out],
                   check=True, capture_output=True)
    r = subprocess.run([out], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout[-1000:] + r.stderr[-2000:]
