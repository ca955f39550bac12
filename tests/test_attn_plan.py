"""Every launch that attn_paged plans within its documented limits is one that
can be made: the argument checks and the plan, swept on the host (CPU only)."""
import os
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)


@pytest.mark.skipif(shutil.which("g++") is None or not os.path.isdir("/opt/rocm/include"),
                    reason="g++ or the HIP headers not available")
def test_planned_launches_are_possible(tmp_path):
    exe = tmp_path / "attn_plan_driver"
    r = subprocess.run(["g++", "-std=c++17", "-O1", "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include",
                        "-I" + os.path.join(ROOT, "include"),
                        "-I" + os.path.join(ROOT, "quantized_dequant_matrix_amd", "csrc"),
                        os.path.join(HERE, "native", "attn_plan_driver.cpp"),
                        os.path.join(ROOT, "quantized_dequant_matrix_amd", "csrc", "step_api.cpp"), "-o", str(exe)],
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and "attention plan driver: ok" in r.stdout, r.stdout[-3000:]
