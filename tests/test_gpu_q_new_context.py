"""The sampling calls in a device context made after another one was destroyed (what a
host that resets its device does), in a process of their own."""
import os
import subprocess
import sys

import pytest

from invariant_lm_head_gemm_b200 import binding

pytestmark = pytest.mark.gpu

CHILD = r"""
import ctypes as C, struct, sys
cu, L = C.CDLL("libcuda.so.1"), C.CDLL(sys.argv[1])
I64, P = C.c_int64, C.c_void_p
L.rlk_token_probs.argtypes = [P, C.c_int, I64, I64, I64, C.c_float, P, P, C.c_int, I64, P, C.c_size_t, P]
L.rlk_draft_verify.argtypes = [P, I64, I64, P, I64, I64, C.c_int, P, P, P, P, I64, I64, I64, P, P, P,
                               C.c_size_t, P]

def ok(r):
    assert r == 0, r

dev = C.c_int()
ok(cu.cuInit(0))
ok(cu.cuDeviceGet(C.byref(dev), 0))

def room(nbytes):
    p = C.c_uint64()
    ok(cu.cuMemAlloc_v2(C.byref(p), C.c_size_t(nbytes)))
    ok(cu.cuMemsetD32_v2(p, 0, C.c_size_t(nbytes // 4)))
    return p.value

def first(p, form, size):
    b = (C.c_char * size)()
    ok(cu.cuMemcpyDtoH_v2(b, C.c_uint64(p), C.c_size_t(size)))
    return struct.unpack(form, bytes(b))[0]

def once():
    ctx = P()
    ok(cu.cuDevicePrimaryCtxRetain(C.byref(ctx), dev))
    ok(cu.cuCtxSetCurrent(ctx))
    V = 262144
    x, p, w, small = room(4 * V), room(4 * V), room(256), room(256)
    for v in (1000, 50257, 151936, 262144):        # equal logits, every form of the kernel
        for src in (0, 1):
            for dst in (0, 1):
                ok(L.rlk_token_probs(x, src, 1, v, v, 1.0, None, p, dst, v, w, 256, None))
                ok(cu.cuCtxSynchronize())
                got = first(p, "<f", 4) if dst else struct.unpack("<f", b"\0\0" + struct.pack(
                    "<H", first(p, "<H", 2)))[0]
                assert abs(got * v - 1) < (1e-4 if dst else 2.0 ** -8), (v, src, dst, got)
    ok(L.rlk_token_probs(x, 1, 1, V, V, 1.0, None, p, 1, V, w, 256, None))
    # no drafts, u = 0: the first token
    ok(L.rlk_draft_verify(p, V, V, None, 0, 0, 1, None, None, small, None, 1, 0, V, small + 64, small + 128,
                          w, 256, None))
    ok(cu.cuCtxSynchronize())
    assert first(small + 64, "<q", 8) == 0 and first(w, "<I", 4) == 0

once()
ok(cu.cuDevicePrimaryCtxReset_v2(dev))
once()
print("done")
"""


def test_calls_after_the_context_is_made_again():
    r = subprocess.run([sys.executable, "-c", CHILD, os.path.abspath(binding.LIB_PATH)], capture_output=True,
                       text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "done", r.stdout + r.stderr
