"""What the compiler reports of kernels whose times depend on how many waves run at once (no GPU)."""
from __future__ import annotations

import os
import re
import subprocess

import pytest

from paged_layout_transfer_amd import _build


def _report(tmp_path, lines):
    """{kernel: {figure: value}} of instantiations, one explicit instantiation a line."""
    source = tmp_path / "kernels.hip"
    source.write_text('#include "kvxfer_attn.h"\nnamespace kvx {\n' + "\n".join(lines) + "\n}\n")
    flags = [f for f in _build.FLAGS if f != "-shared"]
    r = subprocess.run([_build.HIPCC, *flags, "--cuda-device-only", "-I", os.path.join(_build.ROOT, "include"), "-I", _build.CSRC,
                        "-Rpass-analysis=kernel-resource-usage", "-c", str(source), "-o", os.devnull],
                       check=True, capture_output=True, text=True)
    out, name = {}, None
    for line in r.stderr.splitlines():
        m = re.search(r"(Function Name|VGPRs|ScratchSize \[bytes/lane\]|Occupancy \[waves/SIMD\]): (\S+)", line)
        if m and m[1] == "Function Name":
            name = m[2]
            out[name] = {}
        elif m and "AGPRs" not in line:
            out[name][m[1].split()[0]] = int(m[2])
    return out


@pytest.mark.timeout(300)
def test_few_rows_over_64_wide_e4m3_heads_keep_four_waves(tmp_path):
    report = _report(tmp_path, ["template __global__ void attend_few<%s, kE4m3, 64, %d>(const AttnLaunch);" % (t, shaped)
                                for t in ("_Float16", "__bf16") for shaped in range(3)])
    assert len(report) == 6
    for name, r in report.items():
        assert r["VGPRs"] <= 128 and r["Occupancy"] >= 4 and r["ScratchSize"] == 0, (name, r)
