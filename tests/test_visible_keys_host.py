"""Host-side checks of which keys a masked query tile needs, compiled with nvcc
as a plain host program.  No GPU is needed."""
import os
import subprocess

import pytest

from test_work_split_host import HERE, ROOT, _nvcc


def test_visible_keys_host_checks(tmp_path):
    nvcc = _nvcc()
    if nvcc is None:
        pytest.skip("nvcc not available")
    exe = str(tmp_path / "visible_keys_check")
    src = os.path.join(HERE, "host", "visible_keys_check.cu")
    build = subprocess.run(
        [nvcc, "-std=c++17", "-O1", "-gencode", "arch=compute_103a,code=sm_103a",
         "-I", os.path.join(ROOT, "paged_kv_cache_74_gb300", "csrc"), src, "-o", exe],
        capture_output=True, text=True)
    assert build.returncode == 0, build.stderr
    run = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert run.returncode == 0 and run.stdout.strip() == "ok", run.stdout + run.stderr
