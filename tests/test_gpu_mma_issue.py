"""How the issue of tcgen05.mma bounds its rate on this GPU (measurement
support for the paged attention's issue code, not a check of the method): builds
and runs the probe `tests/probes/mma_issue.cu`.  Passes when the probe completes
on every SM; the rates are printed (-s)."""
import os
import shutil
import subprocess

import pytest

pytestmark = pytest.mark.gpu

HERE = os.path.dirname(os.path.abspath(__file__))


def test_mma_issue_probe_runs(tmp_path):
    nvcc, exe = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc", str(tmp_path / "mma_issue")
    subprocess.run([nvcc, "-gencode", "arch=compute_100a,code=sm_100a", "-O3", "-std=c++17", "-o", exe,
                    os.path.join(HERE, "probes", "mma_issue.cu")], check=True, timeout=300)
    out = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    print(out.stdout)
    assert out.returncode == 0, out.stdout + out.stderr
    lines = [ln for ln in out.stdout.splitlines() if "ok=" in ln]
    assert len(lines) == 12 and all("ok=148 " in ln for ln in lines), out.stdout
