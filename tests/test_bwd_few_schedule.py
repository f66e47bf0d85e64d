"""CPU check of the few-row unit order of the distillation's backward, compiled from
the same header the kernel uses (no GPU needed)."""
import os
import subprocess

import pytest

from invariant_lm_head_gemm_b200 import build

HERE = os.path.dirname(os.path.abspath(__file__))
EXE = os.path.join(HERE, "..", "_build", "bwd_few_schedule_check")


@pytest.fixture(scope="module")
def exe():
    os.makedirs(os.path.dirname(EXE), exist_ok=True)
    subprocess.check_call([build.NVCC] + build.ARCH + ["-std=c++17", "-O1", "-I" + build.CSRC,
                           "-I" + build.INCLUDE,
                           os.path.join(HERE, "bwd_few_schedule_check.cu"), "-o", EXE])
    return EXE


@pytest.mark.parametrize("T,H,V", [
    (1, 64, 8193), (7, 64, 20000), (130, 4096, 151936), (257, 192, 16384), (513, 1024, 32768),
    (2000, 256, 8192 * 3 + 1), (600, 320, 40000),
])
def test_schedule(exe, T, H, V):
    out = subprocess.run([exe, str(T), str(H), str(V), "8192"], capture_output=True, text=True, timeout=600)
    assert out.returncode == 0 and out.stdout.startswith("OK"), out.stdout + out.stderr
