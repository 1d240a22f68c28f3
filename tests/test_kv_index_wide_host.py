"""The attention kernels' integer work for hundreds of sequences, contexts of many chunks and windows, on the host under
AddressSanitizer and UndefinedBehaviorSanitizer: tests/sanitize/kv_index_wide_driver.cpp."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.skipif(shutil.which("g++") is None, reason="g++ not available")
def test_wide_calls(tmp_path):
    exe = str(tmp_path / "kv_index_wide")
    subprocess.run(["g++", "-std=c++17", "-g", "-O1", "-fsanitize=address,undefined", "-fno-sanitize-recover=all",
                    "-D__HIP_PLATFORM_AMD__", "-I", "/opt/rocm/include",
                    "-I", os.path.join(ROOT, "block_scaled_fp4_fp4q_amd", "csrc"),
                    os.path.join(ROOT, "tests", "sanitize", "kv_index_wide_driver.cpp"), "-o", exe], check=True)
    p = subprocess.run([exe], capture_output=True, text=True, timeout=600)
    assert p.returncode == 0, p.stdout + p.stderr
    assert "indexed clean" in p.stdout
