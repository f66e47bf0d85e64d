"""CPU check of the backward's unit schedule without dW, compiled from the same header
the kernel uses (no GPU needed)."""
import os
import subprocess

import pytest

from invariant_lm_head_gemm_b200 import build
from tests.test_bwd_schedule import _vchunk

HERE = os.path.dirname(os.path.abspath(__file__))
EXE = os.path.join(HERE, "..", "_build", "bwd_frozen_schedule_check")


@pytest.fixture(scope="module")
def exe():
    os.makedirs(os.path.dirname(EXE), exist_ok=True)
    subprocess.check_call([build.NVCC] + build.ARCH + ["-std=c++17", "-O1", "-I" + build.CSRC,
                           "-I" + build.INCLUDE, "-I" + HERE,
                           os.path.join(HERE, "bwd_frozen_schedule_check.cu"), "-o", EXE])
    return EXE


@pytest.mark.parametrize("T,H,V", [
    (1, 64, 1), (130, 128, 1000), (257, 192, 8193), (300, 256, 20000), (512, 1024, 32768),
    (600, 4096, 33000), (2047, 4096, 151936), (129, 4096, 3 * 8192), (200, 320, 4 * 8192 + 5),
])
def test_schedule(exe, T, H, V):
    out = subprocess.run([exe, str(T), str(H), str(V), str(_vchunk(V))], capture_output=True,
                         text=True, timeout=600)
    assert out.returncode == 0 and out.stdout.startswith("OK"), out.stdout + out.stderr
    # recompute and dHidden tiles alone
    tiles = -(-V // 256) * -(-T // 256)
    chunks = -(-V // _vchunk(V))
    assert int(out.stdout.split()[1]) == tiles + chunks * -(-T // 256) * -(-H // 256)
