"""The streaming decode kernels keep their state in registers: nvcc reports no
spills for them.  No GPU is needed."""
import os
import re
import subprocess

import pytest

from test_work_split_host import HERE, ROOT, _nvcc


def test_no_spills(tmp_path):
    nvcc = _nvcc()
    if nvcc is None:
        pytest.skip("nvcc not available")
    build = subprocess.run(
        [nvcc, "-std=c++17", "-O3", "-gencode", "arch=compute_103a,code=sm_103a", "-Xptxas", "-v",
         "-I", os.path.join(ROOT, "include"), "-I", os.path.join(ROOT, "paged_kv_cache_74_gb300", "csrc"),
         "-c", os.path.join(HERE, "host", "decode_registers.cu"), "-o", str(tmp_path / "out.o")],
        capture_output=True, text=True)
    assert build.returncode == 0, build.stderr
    spills = re.findall(r"Function properties for (\S+)\s+\d+ bytes stack frame, (\d+) bytes spill stores, "
                        r"(\d+) bytes spill loads", build.stderr)
    assert sum("paged_decode_kernel" in s[0] for s in spills) == 6
    assert [s for s in spills if int(s[1]) or int(s[2])] == []
