"""Runs the host code of rotations under AddressSanitizer and UBSan (no GPU, no torch).

Started by tests/test_rotate_sanitizers.py in a child process whose LD_PRELOAD holds the sanitizer runtime; argv[1] is
a build of the library's host files with host-side instrumentation, the launches left out.  Drives row
sizes, frequencies of every size and the arguments that are refused before a GPU is needed.  Prints "ok" at the end; any
sanitizer report aborts the process.
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
for name, args in dict(kv_mx4_row_bytes=[I32, I32, P], kv_rotation_create=[P, P], kv_rotation_destroy=[P],
                       kv_rotate_cached=[P, P, I32, P, I32, I32, I32, P], kv_append_rotated=[P, I32, P, P, P, P],
                       kv_read_tokens=[P, I32, I32, P, P], kv_attn_plan_create=[P, P, P], kv_pool_create=[P, P],
                       kv_pool_destroy=[P]).items():
    getattr(lib, name).argtypes = args


def rows() -> None:
    out = I32()
    for dim in range(-64, 400):
        for heads in (-1, 0, 1, 2, 3, 5, 7, 8, 13, 64, 65536, 2**31 - 1):
            rc = lib.kv_mx4_row_bytes(dim, heads, ctypes.byref(out))
            assert (rc == 0) == (dim > 0 and dim % 32 == 0 and dim <= A.KV_MAX_ATTN_DIM and heads > 0)
            if rc == 0:
                assert out.value // 17 == dim // 32 and out.value % 4 == 0 and out.value * heads % 16 == 0
    assert lib.kv_mx4_row_bytes(64, 1, None) < 0


def rotations() -> None:
    """No GPU: each ends in an error, those in range after their frequencies were worked out."""
    rng, h = np.random.default_rng(4), P()
    fs = [0.0, 5e-324, 2.0**-1022, 1e-300, 2.0**-70, 2.0**-11, 1.0, np.pi, 2 * np.pi, 1024.5, 2.0**20 - 1e-9, 2.0**20]
    fs += np.exp(rng.uniform(-700, 13, 500)).tolist()
    for i in range(0, len(fs) - 4, 4):
        desc = A.make_rotation_desc(fs[i:i + 4], A.KV_ROT_HALVES, 1.0)
        assert lib.kv_rotation_create(ctypes.byref(desc), ctypes.byref(h)) == A.KV_ERR_HIP and not h.value
    for f, amplitude in (([1.0] * 128, 1.0), ([1.0] * 132, 1.0), ([1.0] * 3, 1.0), ([-1.0] * 4, 1.0), ([2.0**21] * 4, 1.0),
                         ([float("nan")] * 4, 1.0), ([float("inf")] * 4, 1.0), ([1.0] * 4, 0.0), ([1.0] * 4, float("nan"))):
        desc = A.make_rotation_desc(f, A.KV_ROT_ADJACENT, amplitude)
        assert lib.kv_rotation_create(ctypes.byref(desc), ctypes.byref(h)) < 0 and not h.value
    assert lib.kv_rotation_create(None, ctypes.byref(h)) < 0 and lib.kv_rotation_create(ctypes.byref(desc), None) < 0
    assert lib.kv_rotation_destroy(None) == 0


def shifts() -> None:
    desc = A.make_pool_desc(2, 2, 2, 64, 2, 16, 64, 16 * 256, [0x7F0000000000 + (i << 28) for i in range(4)])
    h = P()
    assert lib.kv_pool_create(ctypes.byref(desc), ctypes.byref(h)) == 0
    no_rotation = ctypes.create_string_buffer(256)     # reads as one of no pairs, of device 0
    table = 0x7E0000000000

    def call(records, n=None, kind=A.KV_TYPE_BF16, layers=(0, 2)):
        s = (A.kv_shift * max(1, len(records)))(*[A.kv_shift(*r) for r in records])
        return lib.kv_rotate_cached(h, ctypes.byref(no_rotation), kind, s, len(records) if n is None else n, *layers, None)

    assert call([]) == 0 and call([(None, 0, 5, 5, 1)]) == 0
    assert call([(table + 4096 * i, 64, 0, 1000, 7) for i in range(300)]) == A.KV_ERR_HIP     # all taken, then no device
    assert call([(table, 64, 500, 1000, 7), (table, 64, 0, 500, 3)]) == A.KV_ERR_HIP           # side by side
    assert call([(table, 64, 499, 1000, 7), (table + 64, 64, 0, 9, 1), (table, 64, 0, 500, 3)]) == A.KV_ERR_DUP
    assert call([(table, 64, 0, 5, 7)] * 2) == A.KV_ERR_DUP
    for bad in ((None, 4, 0, 60, 1), (table + 2, 4, 0, 60, 1), (table, 3, 0, 60, 1), (table, 4, -1, 60, 1), (table, 4, 61, 60, 1),
                (table, 2**31, 0, 60, 1), (table, 2**40, 0, 2**31, 1), (table, 2**62, 2**62, 2**63 - 1, 1)):
        assert call([(table, 64, 0, 10, 7), bad]) < 0
    most = 2**31 - 4097
    assert call([(table, most // 16 + 1, 0, most, 1)] * 40) < 0       # more pieces than a grid counts
    assert call([], -1) < 0 and call([], A.KV_MAX_SHIFTS + 1) < 0
    for layers in ((0, 0), (1, 1), (-1, 1), (0, 3), (2, 1)):
        assert call([(table, 64, 0, 10, 7)], layers=layers) < 0
    for kind in (A.KV_TYPE_E4M3, A.KV_TYPE_MX4, -1, 9):
        assert call([(table, 64, 0, 10, 7)], kind=kind) < 0
    assert lib.kv_rotate_cached(h, None, A.KV_TYPE_BF16, None, 0, 0, 1, None) < 0
    assert lib.kv_rotate_cached(None, ctypes.byref(no_rotation), A.KV_TYPE_BF16, None, 0, 0, 1, None) < 0
    assert lib.kv_append_rotated(None, 0, None, None, None, None) < 0 and lib.kv_read_tokens(None, 0, 1, None, None) < 0
    assert lib.kv_pool_destroy(h) == 0
    for heads, code in ((1 << 20, A.KV_ERR_HIP), (1 << 21, A.KV_ERR_ARG)):     # 2^27 elements of a token's k and v, 2^28
        desc = A.make_pool_desc(1, 2, heads, 64, 2, 1, 64, heads * 128, [0x7F0000000000, 0x7F8000000000])
        assert lib.kv_pool_create(ctypes.byref(desc), ctypes.byref(h)) == 0
        assert call([(table, 64, 0, 10, 7)], layers=(0, 1)) == code
        assert lib.kv_pool_destroy(h) == 0


rows()
rotations()
shifts()
print("ok")
