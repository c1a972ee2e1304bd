"""csrc/gdr_api.hip (argument checks and kernel selection) under AddressSanitizer and
UndefinedBehaviorSanitizer on the CPU, driven by tests/sanitize/gdr_driver.cpp."""
import os
import shutil

import pytest

from test_sanitizers import FLAGS, ROCM, ROOT, SAN, _build_and_run


@pytest.mark.skipif(shutil.which("g++") is None, reason="g++ not available")
def test_gdr_abi_layer_under_sanitizers(tmp_path):
    exe = str(tmp_path / "gdr_driver")
    cmd = (["g++", "-std=c++17"] + FLAGS + ["-D__HIP_PLATFORM_AMD__", "-I", os.path.join(ROCM, "include"),
           "-x", "c++", os.path.join(ROOT, "rwkv_linear_attention_amd", "csrc", "gdr_api.hip"), "-x", "none",
           os.path.join(SAN, "gdr_driver.cpp"), "-o", exe])
    _build_and_run(cmd, exe, tmp_path)
