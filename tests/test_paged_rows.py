"""Rows of a page's heads beyond 32 bits (csrc/usp_paged.cuh), on the host: such a pool is larger than most cards."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def build_and_run(name, tmp_path, checks):
    gxx = shutil.which("g++")
    cuda = next((d for d in ("/usr/local/cuda/include", os.path.join(os.environ.get("CUDA_HOME", ""), "include"))
                 if os.path.exists(os.path.join(d, "cuda_runtime.h"))), None)
    if gxx is None or cuda is None:
        pytest.skip("needs g++ and the CUDA headers")
    exe = str(tmp_path / name)
    cmd = [gxx, "-std=c++17", "-O1", "-g", "-fsanitize=" + checks, "-fno-sanitize-recover=all", "-I", cuda, "-I",
           os.path.join(ROOT, "ulysses_sequence_long_gb300", "csrc"), os.path.join(ROOT, "tests", name + ".cpp"), "-o", exe]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-3000:]
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout + r.stderr[-3000:]


def test_rows_beyond_32_bits(tmp_path):
    build_and_run("paged_rows", tmp_path, "undefined")
