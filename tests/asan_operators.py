"""Runs the host code of the operators on a paged cache under AddressSanitizer and UBSan (no GPU, no torch).

Started by tests/test_operators_sanitizers.py in a child process whose LD_PRELOAD holds the sanitizer
runtime; argv[1] is a build of the library's host files with host-side instrumentation, the operators'
launches left out.  Drives references, forks and compactions against a model of plain dicts, and the arguments that
the device calls refuse before they need a GPU.  Prints "ok" at the end; any sanitizer report aborts the process.
"""
from __future__ import annotations

import ctypes
import os
import sys

import numpy as np

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from paged_layout_transfer_amd import _abi as A  # noqa: E402

lib = ctypes.CDLL(sys.argv[1])
P, I32, I64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
for name, args in dict(kv_pool_alloc_blocks=[P, I32, P], kv_pool_free_blocks=[P, I32, P], kv_pool_share_blocks=[P, I32, P],
                       kv_pool_block_refs=[P, I32, P], kv_pool_fork_blocks=[P, I64, P, P, P], kv_pool_free_count=[P, P],
                       kv_pool_plan_compact=[P, I32, P, P], kv_copy_pages=[P, P, I32, I32, I32, P],
                       kv_remap_tables=[P, P, I32, P, P, I64, P], kv_attn_plan_create=[P, P, P],
                       kv_pool_create=[P, P], kv_pool_destroy=[P]).items():
    getattr(lib, name).argtypes = args


def pool_of(n, page=16):
    tok = 2 * 64 * 2
    desc = A.make_pool_desc(1, 2, 2, 64, 2, page, n, page * tok, [0x7F0000000000, 0x7F8000000000])
    h = P()
    assert lib.kv_pool_create(ctypes.byref(desc), ctypes.byref(h)) == 0
    return h


def ids_of(x):
    return np.ascontiguousarray(x, dtype=np.int32)


def model(seed: int) -> None:
    """Random calls; refs maps each allocated block to its references, moved holds the sources of compactions."""
    rng = np.random.default_rng(seed)
    n = int(rng.integers(1, 300))
    h, refs, moved = pool_of(n), {}, set()

    def drop(ids):
        for i in ids:
            refs[i] -= 1
            if refs[i] == 0:
                del refs[i]
                moved.discard(i)

    for _ in range(400):
        what, held = int(rng.integers(0, 6)), sorted(refs)
        if what == 0:
            k = int(rng.integers(0, n // 3 + 2))
            out = np.empty(max(1, k), np.int32)
            rc = lib.kv_pool_alloc_blocks(h, k, out.ctypes.data)
            free = [i for i in range(n) if i not in refs]
            assert rc == (0 if k <= len(free) else A.KV_ERR_OOM)
            if rc == 0:
                assert out[:k].tolist() == free[:k]
                refs.update((i, 1) for i in free[:k])
        elif what == 1 and held:
            ids = [int(i) for i in rng.permutation(held)[:int(rng.integers(1, len(held) + 1))]]
            bad = int(rng.integers(0, 8))
            x = ids + [[ids[0]], [n], [-1]][bad] if bad < 3 else ids
            a = ids_of(x)
            rc = lib.kv_pool_free_blocks(h, a.size, a.ctypes.data)
            assert rc == (A.KV_ERR_RANGE if bad < 3 else 0)
            if rc == 0:
                drop(ids)
        elif what == 2 and held:
            ids = [int(i) for i in rng.choice(held, int(rng.integers(1, 9)))]
            a = ids_of(ids)
            assert lib.kv_pool_share_blocks(h, a.size, a.ctypes.data) == 0
            for i in ids:
                refs[i] += 1
        elif what == 3 and held:
            ids = [int(i) for i in rng.permutation(held)[:int(rng.integers(1, len(held) + 1))]]
            tokens = 16 * len(ids) - int(rng.integers(0, 16))
            a, child, tail = ids_of(ids), np.empty(len(ids), np.int32), A.kv_page_copy()
            rc = lib.kv_pool_fork_blocks(h, tokens, a.ctypes.data, child.ctypes.data, ctypes.byref(tail))
            free = [i for i in range(n) if i not in refs]
            part = tokens % 16 != 0
            assert rc == (A.KV_ERR_OOM if part and not free else 0)
            if rc == 0:
                assert child.tolist() == ids[:-1] + [free[0]] if part else child.tolist() == ids
                for i in ids[:-1] if part else ids:
                    refs[i] += 1
                if part:
                    refs[free[0]] = 1
        elif what == 4:
            most = int(rng.integers(0, n + 2))
            moves, count = (A.kv_page_copy * max(1, most))(), I32()
            assert lib.kv_pool_plan_compact(h, most, moves, ctypes.byref(count)) == 0
            high = [i for i in sorted(refs, reverse=True) if i not in moved]
            low = [i for i in range(n) if i not in refs]
            want = [(a, b) for a, b in zip(high, low) if b < a][:most]
            assert [(m.src, m.dst) for m in moves[:count.value]] == want[::-1]
            for a, b in want:
                refs[b], refs[a] = refs[a], 1
                moved.add(a)
        elif what == 5 and moved:
            ids = [i for i in moved if refs[i] == 1]
            a = ids_of(ids)
            assert lib.kv_pool_free_blocks(h, a.size, a.ctypes.data) == 0
            drop(ids)
        count = I64()
        assert lib.kv_pool_free_count(h, ctypes.byref(count)) == 0 and count.value == n - len(refs)
        for i in rng.integers(0, n, 5):
            got = I32()
            assert lib.kv_pool_block_refs(h, int(i), ctypes.byref(got)) == 0 and got.value == refs.get(int(i), 0)
    assert lib.kv_pool_destroy(h) == 0


def refusals() -> None:
    h = pool_of(64)
    tail, count = A.kv_page_copy(), I32()
    a, child = ids_of(range(4)), np.empty(4, np.int32)
    for tokens in (-1, 65 * 16, 2**62, 2**63 - 1):
        assert lib.kv_pool_fork_blocks(h, tokens, a.ctypes.data, child.ctypes.data, ctypes.byref(tail)) < 0
    assert lib.kv_pool_fork_blocks(h, 0, None, None, ctypes.byref(tail)) == 0
    assert lib.kv_pool_plan_compact(h, A.KV_MAX_PAGE_COPIES + 1, None, ctypes.byref(count)) < 0
    for copies in ([(0, 64, 1)], [(-1, 2, 1)], [(0, 1, 0)], [(0, 1, 4), (2, 1, 4)], [(0, 1, 4), (1, 2, 4)]):
        c = A.make_page_copies(copies)
        assert lib.kv_copy_pages(h, c, len(copies), 0, 1, None) < 0
        assert lib.kv_remap_tables(h, c, len(copies), 0x1000, 0x1004, 4, None) < 0
    one = A.make_page_copies([(0, 1, 16)])
    for n in (-1, A.KV_MAX_PAGE_COPIES + 1):
        assert lib.kv_copy_pages(h, one, n, 0, 1, None) < 0 and lib.kv_remap_tables(h, one, n, None, None, 0, None) < 0
    assert lib.kv_remap_tables(h, one, 1, 0x1000, 0x1000, 2**62, None) < 0
    plan = P()
    for kw in (dict(num_q_heads=3), dict(max_seqs=0), dict(max_tokens=1 << 25), dict(window=-1), dict(flags=6),
               dict(num_q_heads=1 << 30, max_tokens=1 << 24)):
        d = dict(num_q_heads=4, q_type=A.KV_TYPE_BF16, kv_type=A.KV_TYPE_BF16, max_seqs=2, max_tokens=4)
        d.update(kw)
        desc = A.make_attn_desc(**d)
        assert lib.kv_attn_plan_create(h, ctypes.byref(desc), ctypes.byref(plan)) < 0 and not plan.value
    assert lib.kv_pool_destroy(h) == 0


for seed in range(30):
    model(seed)
refusals()
print("ok")
