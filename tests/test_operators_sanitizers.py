"""The operators' host code under AddressSanitizer and UBSan (CPU only): kvxfer.cpp, kvxfer_ops.cpp and the
allocator, built with host-side instrumentation and driven by tests/asan_operators.py in a child process that
preloads the sanitizer runtime.  Launches are left out: nothing here reaches one."""
from __future__ import annotations

import os
import subprocess
import sys

import pytest

from paged_layout_transfer_amd import _build
from test_host_sanitizers import _runtime

HERE = os.path.dirname(os.path.abspath(__file__))

NO_LAUNCHES = """
#include <hip/hip_runtime.h>
#include "kvxfer_ops.h"
namespace kvx {
int launch_copy_pages(const CopyLaunch &, hipStream_t) { return 1; }
int launch_remap(const RemapLaunch &, hipStream_t) { return 1; }
int padded_dim(int dim) { return dim <= 64 ? 64 : dim <= 128 ? 128 : 256; }
int launch_attend(const AttnLaunch &, int, int, int, uint32_t, hipStream_t) { return 1; }
int launch_join(const AttnLaunch &, int, uint32_t, hipStream_t) { return 1; }
int launch_append(const AttnLaunch &, int, int, uint32_t, hipStream_t) { return 1; }
}
"""


@pytest.mark.timeout(600)
def test_the_operators_host_code_is_clean_under_asan_and_ubsan(tmp_path):
    rt = _runtime()
    if rt is None:
        pytest.skip("no sanitizer runtime next to the compiler")
    stubs, out = tmp_path / "no_launches.cpp", str(tmp_path / "libops_asan.so")
    stubs.write_text(NO_LAUNCHES)
    flags = [f for f in _build.FLAGS if f != "-fvisibility=hidden"]
    cmd = [_build.HIPCC, *flags,
           "-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
           "-Xarch_host", "-fno-sanitize-recover=undefined", "-Xarch_host", "-fno-omit-frame-pointer",
           "-shared-libsan", "-I", os.path.join(_build.ROOT, "include"), "-I", _build.CSRC,
           *_build.SOURCES, os.path.join(_build.CSRC, "kvxfer_ops.cpp"), str(stubs), "-o", out]
    subprocess.run(cmd, check=True, capture_output=True)
    env = dict(os.environ, LD_PRELOAD=rt, ASAN_OPTIONS="detect_leaks=0:abort_on_error=1",
               UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1")
    r = subprocess.run([sys.executable, os.path.join(HERE, "asan_operators.py"), out], env=env,
                       capture_output=True, text=True, timeout=500)
    assert r.returncode == 0 and r.stdout.strip().endswith("ok"), r.stdout[-2000:] + r.stderr[-4000:]
    assert "runtime error" not in r.stderr, r.stderr[-4000:]
