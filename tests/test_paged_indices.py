"""The paged cache's index arithmetic (csrc/usp_paged.cuh) on the host, on x86 under the address sanitizer: tables,
lengths and boundaries of any content never lead outside the pool, and the decoding attention deals out every tile once."""
import os
import platform
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_indices_on_the_host(tmp_path):
    gxx = shutil.which("g++")
    cuda = next((d for d in ("/usr/local/cuda/include", os.path.join(os.environ.get("CUDA_HOME", ""), "include"))
                 if os.path.exists(os.path.join(d, "cuda_runtime.h"))), None)
    if gxx is None or cuda is None:
        pytest.skip("needs g++ and the CUDA headers")
    exe = str(tmp_path / "paged_indices")
    # (on 64-bit Arm the address sanitizer hangs at its start where the kernel spreads addresses over more bits than it knows)
    checks = "address,undefined" if platform.machine() == "x86_64" else "undefined"
    cmd = [gxx, "-std=c++17", "-O1", "-g", "-fsanitize=" + checks, "-fno-sanitize-recover=all", "-I", cuda, "-I",
           os.path.join(ROOT, "ulysses_sequence_long_gb300", "csrc"),
           os.path.join(ROOT, "tests", "paged_indices.cpp"), "-o", exe]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-3000:]
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout + r.stderr[-3000:]
