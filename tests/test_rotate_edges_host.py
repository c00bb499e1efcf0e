"""Host side of rotations and 4-bit pools at the ends of their ranges (no GPU)."""
from __future__ import annotations

import os
import subprocess

from paged_layout_transfer_amd import _build


def _run_cpp(name, tmp_path):
    """A C++ test under AddressSanitizer and UBSan (host code only)."""
    rocm = os.path.dirname(os.path.dirname(os.path.realpath(_build.HIPCC)))
    out = str(tmp_path / name)
    subprocess.run(["g++", "-std=c++17", "-O2", "-g", "-Wall", "-fsanitize=address,undefined",
                    "-fno-sanitize-recover=undefined", "-D__HIP_PLATFORM_AMD__", "-I", os.path.join(rocm, "include"),
                    "-I", os.path.join(_build.ROOT, "include"), "-I", _build.CSRC,
                    os.path.join(os.path.dirname(__file__), name + ".cpp"), "-o", out],
                   check=True, capture_output=True)
    r = subprocess.run([out], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout[-1000:] + r.stderr[-2000:]


def test_shifts_of_as_many_items_as_a_call_may_have_end(tmp_path):
    """tests/shift_walk.cpp: a workgroup's last step passes 31 bits."""
    _run_cpp("shift_walk", tmp_path)


def test_arrays_in_any_order_of_their_dimensions_are_taken(tmp_path):
    """tests/apart_walk.cpp: outputs of layers, tokens and heads."""
    _run_cpp("apart_walk", tmp_path)


def test_the_split_search_counts_equal_parts_together(tmp_path):
    """tests/plan_spans.cpp: the same spans as parts dealt one by one, and few runs for steps of unequal token counts."""
    _run_cpp("plan_spans", tmp_path)
