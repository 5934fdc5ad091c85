"""The launcher of the layer for a few tokens on a second device of the process, against a stand-in for the CUDA runtime
(tests/decode_devices_fake.cpp): no GPU needed."""
import os
import shutil
import subprocess

import pytest

from combine_fp32_softmax_gb300 import build as B

HERE = os.path.dirname(os.path.abspath(__file__))


def test_kernels_may_use_their_shared_memory_on_every_device(tmp_path):
    cxx, inc = shutil.which("g++"), "/usr/local/cuda/include"
    if not cxx or not os.path.isdir(inc):
        pytest.skip("needs g++ and the CUDA headers")
    obj = os.path.join(B.OUT_DIR, "decode.o")
    if not os.path.exists(obj):
        B.build()
    exe = str(tmp_path / "devices")
    subprocess.run([cxx, "-std=c++17", "-I", inc, "-I", B.CSRC, "-o", exe, os.path.join(HERE, "decode_devices_fake.cpp"),
                    obj], check=True, capture_output=True, text=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, r.stdout + r.stderr
