"""Host side of the operators on a paged cache (no GPU): references, forks, compaction plans,
and the arguments each entry point refuses before any HIP call."""
from __future__ import annotations

import ctypes

import numpy as np
import pytest

from paged_layout_transfer_amd import kvxfer as K

FAKE = 0x7F0000000000


def _pool(N=64, bs=16, H=2, D=64, E=2, KV=2, L=2, page_layout=0):
    tok = H * D * E
    return K.kv_pool_create(K.make_pool_desc(L, KV, H, D, E, bs, N, bs * tok,
                                             [FAKE + i * (1 << 30) for i in range(L * KV)], page_layout))


def _refused(code, fn, *args):
    with pytest.raises(K.KvError) as e:
        fn(*args)
    assert e.value.code == code


def test_references_keep_a_block_until_the_last_one_goes():
    p = _pool()
    ids = K.kv_pool_alloc_blocks(p, 4)
    assert [K.kv_pool_block_refs(p, i) for i in (0, 3, 4)] == [1, 1, 0]
    K.kv_pool_share_blocks(p, [0, 1, 1])
    assert [K.kv_pool_block_refs(p, i) for i in range(4)] == [2, 3, 1, 1]
    K.kv_pool_free_blocks(p, ids)
    assert K.kv_pool_free_count(p) == 62
    assert [K.kv_pool_block_refs(p, i) for i in range(4)] == [1, 2, 0, 0]
    _refused(K.KV_ERR_RANGE, K.kv_pool_free_blocks, p, [1, 0, 1])   # twice in one call: nothing freed
    assert [K.kv_pool_block_refs(p, i) for i in range(2)] == [1, 2]
    _refused(K.KV_ERR_RANGE, K.kv_pool_share_blocks, p, [0, 2])
    _refused(K.KV_ERR_RANGE, K.kv_pool_share_blocks, p, [0, 64])
    _refused(K.KV_ERR_RANGE, K.kv_pool_share_blocks, p, [-1])
    assert [K.kv_pool_block_refs(p, i) for i in range(3)] == [1, 2, 0]
    K.kv_pool_free_blocks(p, [0, 1])
    K.kv_pool_free_blocks(p, [1])
    assert K.kv_pool_free_count(p) == 64
    assert K.kv_pool_alloc_blocks(p, 3).tolist() == [0, 1, 2]
    _refused(K.KV_ERR_RANGE, K.kv_pool_block_refs, p, 64)
    K.kv_pool_destroy(p)


@pytest.mark.parametrize("tokens,tail", [(0, None), (1, 1), (16, None), (33, 1), (47, 15), (48, None)])
def test_fork_shares_whole_pages_and_copies_the_tail(tokens, tail):
    p = _pool()
    ids = K.kv_pool_alloc_blocks(p, -(-tokens // 16))
    child, copy = K.kv_pool_fork_blocks(p, tokens, ids)
    whole = tokens // 16
    assert child[:whole].tolist() == ids[:whole].tolist()
    assert all(K.kv_pool_block_refs(p, int(i)) == 2 for i in ids[:whole])
    if tail is None:
        assert copy is None
    else:
        assert copy == (int(ids[-1]), int(child[-1]), tail) and child[-1] not in ids
        assert K.kv_pool_block_refs(p, int(ids[-1])) == 1
    K.kv_pool_free_blocks(p, ids)
    K.kv_pool_free_blocks(p, child)
    assert K.kv_pool_free_count(p) == 64
    K.kv_pool_destroy(p)


def test_fork_refuses_and_changes_nothing():
    p = _pool(N=3)
    ids = K.kv_pool_alloc_blocks(p, 3)
    _refused(K.KV_ERR_OOM, K.kv_pool_fork_blocks, p, 47, ids)     # no block for the tail
    _refused(K.KV_ERR_DUP, K.kv_pool_fork_blocks, p, 48, [0, 1, 1])
    _refused(K.KV_ERR_RANGE, K.kv_pool_fork_blocks, p, 16, [3])
    _refused(K.KV_ERR_RANGE, K.kv_pool_fork_blocks, p, 1 << 40, ids)
    _refused(K.KV_ERR_ARG, K.kv_pool_fork_blocks, p, -1, ids)
    assert [K.kv_pool_block_refs(p, i) for i in range(3)] == [1, 1, 1]
    K.kv_pool_destroy(p)


@pytest.mark.parametrize("bs", [1, 16, 24])
@pytest.mark.parametrize("tokens", [2**63 - 1, 2**63 - 16, 2**62, 65 * 24])
def test_a_fork_of_more_tokens_than_the_pool_holds_is_out_of_range(bs, tokens):
    p = _pool(bs=bs)
    ids, child = np.zeros(64, np.int32), np.full(64, -1, np.int32)
    tail = K.kv_page_copy()
    rc = K._lib.kv_pool_fork_blocks(p, tokens, ids.ctypes.data, child.ctypes.data, ctypes.byref(tail))
    assert rc == K.KV_ERR_RANGE and (child == -1).all()
    K.kv_pool_destroy(p)


def test_a_fork_takes_as_many_ids_as_the_tokens_have_pages():
    p = _pool()
    ids = K.kv_pool_alloc_blocks(p, 5)
    for few in ([], ids[:2]):
        with pytest.raises(ValueError):
            K.kv_pool_fork_blocks(p, 40, few)
    child, tail = K.kv_pool_fork_blocks(p, 40, ids)     # the parent has room for more tokens
    assert child.tolist() == [0, 1, 5] and tail == (2, 5, 8)
    child, tail = K.kv_pool_fork_blocks(p, 0, ids)
    assert child.size == 0 and tail is None
    assert [K.kv_pool_block_refs(p, i) for i in range(6)] == [2, 2, 1, 1, 1, 1]
    K.kv_pool_destroy(p)


@pytest.mark.parametrize("N,live,most", [(64, 20, 100), (64, 64, 8), (64, 0, 8), (200, 90, 7), (1000, 333, 1000), (1, 1, 1)])
def test_compaction_pairs_highest_pages_with_lowest_holes(N, live, most):
    rng = np.random.default_rng(N + live)
    p = _pool(N=N)
    K.kv_pool_alloc_blocks(p, N)
    keep = np.sort(rng.permutation(N)[:live])
    gone = np.setdiff1d(np.arange(N), keep)
    K.kv_pool_free_blocks(p, gone)
    shared = keep[::3].astype(np.int32)
    K.kv_pool_share_blocks(p, shared)
    want, have, holes = [], list(keep), list(gone)
    while len(want) < most and have and holes and holes[0] < have[-1]:
        want.append((have.pop(), holes.pop(0)))
    moves = K.kv_pool_plan_compact(p, most)
    got = [(m.src, m.dst, m.n_tokens) for m in moves[:moves._n]]
    assert got == [(int(a), int(b), 16) for a, b in reversed(want)]
    assert K.kv_pool_free_count(p) == N - live - len(want)
    for a, b in want:
        assert K.kv_pool_block_refs(p, int(a)) == 1
        assert K.kv_pool_block_refs(p, int(b)) == (2 if a in shared else 1)
    K.kv_pool_free_blocks(p, [a for a, _ in want])
    assert K.kv_pool_free_count(p) == N - live
    K.kv_pool_destroy(p)


@pytest.mark.parametrize("N,most", [(16, 2), (200, 7), (300, 64)])
def test_a_pool_is_compacted_a_few_pages_at_a_time(N, most):
    """Plans made one after another, no source freed in between: every move is of another page."""
    rng = np.random.default_rng(N)
    p = _pool(N=N)
    K.kv_pool_alloc_blocks(p, N)
    gone = np.sort(rng.permutation(N)[:N // 2])
    keep = np.setdiff1d(np.arange(N), gone)
    K.kv_pool_free_blocks(p, gone)
    K.kv_pool_share_blocks(p, keep[::2])
    refs = {int(i): K.kv_pool_block_refs(p, int(i)) for i in keep}
    where, moved = {i: i for i in refs}, []       # a page's place by its first one
    have, holes = [int(i) for i in keep], [int(i) for i in gone]
    while True:
        want = []
        while len(want) < most and have and holes and holes[0] < have[-1]:
            want.append((have.pop(), holes.pop(0)))
        moves = K.kv_pool_plan_compact(p, most)
        got = [(m.src, m.dst) for m in moves[:moves._n]]
        assert got == want[::-1]
        if not got:
            break
        for src, dst in got:
            assert where.pop(src) == src
            where[dst] = src
            moved.append(src)
        assert K.kv_pool_free_count(p) == len(gone) - len(moved)
    assert len(set(moved)) == len(moved) > most
    assert all(K.kv_pool_block_refs(p, at) == refs[first] for at, first in where.items())
    assert all(K.kv_pool_block_refs(p, i) == 1 for i in moved)
    K.kv_pool_free_blocks(p, moved)
    assert K.kv_pool_free_count(p) == len(gone)
    # freed sources are ordinary blocks again: handed out and moved like any other
    again = K.kv_pool_alloc_blocks(p, K.kv_pool_free_count(p))
    assert set(moved) <= set(again.tolist())
    K.kv_pool_free_blocks(p, [i for i in again if i != max(moved)])
    moves = K.kv_pool_plan_compact(p, most)
    assert [(m.src, m.dst) for m in moves[:moves._n]] == [(max(moved), len(keep))]
    K.kv_pool_destroy(p)


COPIES = [
    ([(0, 64, 1)], K.KV_ERR_RANGE), ([(-1, 2, 1)], K.KV_ERR_RANGE), ([(0, 1, 0)], K.KV_ERR_ARG),
    ([(0, 1, 17)], K.KV_ERR_ARG), ([(0, 1, 4), (2, 1, 4)], K.KV_ERR_DUP), ([(0, 1, 4), (1, 2, 4)], K.KV_ERR_DUP),
    ([(5, 5, 16)], K.KV_ERR_DUP),
]


@pytest.mark.parametrize("copies,code", COPIES)
def test_copy_refusals(copies, code):
    p = _pool()
    _refused(code, K.kv_copy_pages, p, K.make_page_copies(copies), 0, 2)
    K.kv_pool_destroy(p)


def test_copy_and_remap_ranges():
    p = _pool()
    one = K.make_page_copies([(0, 1, 16)])
    for lo, hi in ((-1, 1), (0, 3), (1, 1), (2, 1)):
        _refused(K.KV_ERR_ARG, K.kv_copy_pages, p, one, lo, hi)
    K.kv_copy_pages(p, K.make_page_copies([]), 0, 2)     # nothing to do: no GPU needed
    t = np.zeros(8, np.int32).ctypes.data & ~15
    _refused(K.KV_ERR_ARG, K.kv_remap_tables, p, one, 0, t, 4)
    _refused(K.KV_ERR_ALIGN, K.kv_remap_tables, p, one, t + 2, t + 2, 4)
    _refused(K.KV_ERR_ARG, K.kv_remap_tables, p, one, t, t + 4, 4)     # overlapping, not in place
    _refused(K.KV_ERR_ARG, K.kv_remap_tables, p, one, t, t, -1)
    _refused(K.KV_ERR_DUP, K.kv_remap_tables, p, K.make_page_copies([(3, 1, 1), (3, 2, 1)]), t, t, 4)
    _refused(K.KV_ERR_RANGE, K.kv_remap_tables, p, K.make_page_copies([(3, 64, 1)]), t, t, 4)
    K.kv_remap_tables(p, one, t, t, 0)
    many = (K.kv_page_copy * (K.KV_MAX_PAGE_COPIES + 1))()
    many._n = K.KV_MAX_PAGE_COPIES + 1
    _refused(K.KV_ERR_ARG, K.kv_copy_pages, p, many, 0, 2)
    _refused(K.KV_ERR_ARG, K.kv_remap_tables, p, many, t, t, 4)
    _refused(K.KV_ERR_ARG, K.kv_pool_plan_compact, p, K.KV_MAX_PAGE_COPIES + 1)
    K.kv_pool_destroy(p)


def _desc(heads=8, q=K.KV_TYPE_BF16, kv=K.KV_TYPE_BF16, seqs=4, tokens=64, window=0, flags=0):
    return K.make_attn_desc(heads, q, kv, seqs, tokens, window, flags)


PLANS = [
    (dict(), dict(heads=3), K.KV_ERR_ARG),                              # not a multiple of the pool's heads
    (dict(), dict(heads=0), K.KV_ERR_ARG),
    (dict(), dict(q=K.KV_TYPE_E4M3, kv=K.KV_TYPE_E4M3), K.KV_ERR_ARG),
    (dict(), dict(q=K.KV_TYPE_F16), K.KV_ERR_ARG),                      # two 16-bit types
    (dict(), dict(kv=K.KV_TYPE_E4M3), K.KV_ERR_ARG),                    # a pool of 2-byte elements
    (dict(E=1), dict(), K.KV_ERR_ARG),
    (dict(KV=1), dict(), K.KV_ERR_ARG),
    (dict(D=264), dict(), K.KV_ERR_ARG),
    (dict(D=4, H=2), dict(), K.KV_ERR_ALIGN),
    (dict(D=8, H=2, E=1), dict(kv=K.KV_TYPE_E4M3), K.KV_ERR_ALIGN),
    (dict(), dict(window=-1), K.KV_ERR_ARG),
    (dict(), dict(window=5, flags=K.KV_ATTN_FULL), K.KV_ERR_ARG),
    (dict(), dict(flags=2), K.KV_ERR_ARG),
    (dict(), dict(seqs=0), K.KV_ERR_ARG),
    (dict(), dict(seqs=K.KV_MAX_SEQS + 1), K.KV_ERR_ARG),
    (dict(), dict(tokens=0), K.KV_ERR_ARG),
    (dict(), dict(tokens=(1 << 24) + 1), K.KV_ERR_ARG),
    (dict(), dict(heads=1024, tokens=1 << 22), K.KV_ERR_ARG),           # rows past 31 bits
]


@pytest.mark.parametrize("pool,desc,code", PLANS)
def test_plan_refusals(pool, desc, code):
    p = _pool(**pool)
    _refused(code, K.kv_attn_plan_create, p, _desc(**desc))
    K.kv_pool_destroy(p)


def test_null_handles():
    assert K._lib.kv_attn_plan_destroy(None) == K.KV_OK
    assert K._lib.kv_attn_plan_create(None, None, None) == K.KV_ERR_ARG
    assert K._lib.kv_attn_plan_set(None, None, 0, None) == K.KV_ERR_ARG
    assert K._lib.kv_append_tokens(None, 0, None, None) == K.KV_ERR_ARG
    assert K._lib.kv_attend(None, 0, None, None) == K.KV_ERR_ARG
    assert K._lib.kv_copy_pages(None, None, 0, 0, 1, None) == K.KV_ERR_ARG
    assert K._lib.kv_remap_tables(None, None, 0, None, None, 0, None) == K.KV_ERR_ARG
    assert K._lib.kv_pool_share_blocks(None, 0, None) == K.KV_ERR_ARG
    assert K._lib.kv_pool_fork_blocks(None, 0, None, None, ctypes.byref(K.kv_page_copy())) == K.KV_ERR_ARG
    assert K._lib.kv_pool_plan_compact(None, 0, None, None) == K.KV_ERR_ARG


def test_row_arrays_need_packed_heads():
    import torch

    x = torch.zeros(4, 2, 8, 2)[..., 0]
    with pytest.raises(ValueError):
        K.make_append_args(x, x, 4)


def test_plans_walk_every_visible_key_once(tmp_path):
    """tests/plan_walk.cpp under AddressSanitizer and UBSan (host code only)."""
    import os
    import subprocess

    from paged_layout_transfer_amd import _build

    rocm = os.path.dirname(os.path.dirname(os.path.realpath(_build.HIPCC)))
    out = str(tmp_path / "plan_walk")
    subprocess.run(["g++", "-std=c++17", "-O2", "-g", "-Wall", "-fsanitize=address,undefined",
                    "-fno-sanitize-recover=undefined", "-D__HIP_PLATFORM_AMD__", "-I", os.path.join(rocm, "include"),
                    "-I", os.path.join(_build.ROOT, "include"), "-I", _build.CSRC,
                    os.path.join(os.path.dirname(__file__), "plan_walk.cpp"), "-o", out],
                   check=True, capture_output=True)
    r = subprocess.run([out], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout[-1000:] + r.stderr[-2000:]
