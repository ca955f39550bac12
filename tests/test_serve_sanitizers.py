"""The argument checking of include/qmv_serve.h under AddressSanitizer and
UndefinedBehaviorSanitizer (host code only), with the kernel launchers replaced
by stubs that check what reaches them."""
import os
import shutil

import pytest

from test_native_sanitizers import HERE, ROOT, SAN, _run


@pytest.mark.skipif(shutil.which("g++") is None or not os.path.isdir("/opt/rocm/include"),
                    reason="g++ or the HIP headers not available")
def test_serve_argument_checks_under_sanitizers(tmp_path):
    exe = tmp_path / "serve_host_driver"
    out = _run(["g++", "-std=c++17", *SAN, "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include",
                "-I" + os.path.join(ROOT, "include"), "-I" + os.path.join(ROOT, "quantized_dequant_matrix_amd", "csrc"),
                os.path.join(HERE, "native", "serve_host_driver.cpp"),
                os.path.join(ROOT, "quantized_dequant_matrix_amd", "csrc", "serve_api.cpp"), "-o", str(exe)], exe, tmp_path)
    assert "serve host driver: ok" in out
