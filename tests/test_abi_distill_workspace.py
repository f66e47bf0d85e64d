"""Which workspaces the distillation's backward takes, without a GPU: a call that is
accepted goes on to the device check, so on a machine without one it is refused for
that reason only."""
import random

import pytest
import torch

from tests.test_abi_distill import DEVICE, WS_SMALL, L, _bwd, _fwd  # noqa: F401 (L: a fixture)

pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="pointers are not real")


def _a(x):
    return (x + 255) // 256 * 256


def _least(T, H, V, K):
    """The chunk-by-chunk order's bytes: linear-logp's and the teacher's rows."""
    from invariant_lm_head_gemm_b200 import binding
    return binding.workspace_bytes(T, H, V, True) + 3 * _a(T * K * 4) + 2 * _a(T * 4) + \
        _a(T * (-(-V // 256)) * 8)


@pytest.mark.parametrize("H,V,K", [(4096, 151936, 64), (1024, 32768, 20), (64, 8193, 1), (8192, 524288, 8)])
def test_a_workspace_for_many_rows_serves_fewer(L, H, V, K):
    f = L.rlk_linear_distill_workspace_bytes
    for most in (5980, 1024, 513, 257):
        n = f(most, H, V, K, 1)
        for T in (1, 16, 100, 256, 257, 512, 513, 862, 1024, 2047):
            if T <= most:
                assert _bwd(L, T=T, H=H, V=V, K=K, wsb=n) == DEVICE, (most, T)
                assert _fwd(L, T=T, H=H, V=V, K=K, wsb=n) == DEVICE, (most, T)


def test_smaller_sizes_fit_in_a_workspace_for_larger_ones(L):
    rng = random.Random(5)
    f = L.rlk_linear_distill_workspace_bytes
    for _ in range(300):
        big = [int(2 ** rng.uniform(0, 12)), 64 * int(2 ** rng.uniform(0, 6)), int(2 ** rng.uniform(4, 18)),
               int(2 ** rng.uniform(0, 8))]
        small = [max(1, int(b * rng.choice([1, 1, rng.random()]))) for b in big]
        small[1] = max(64, small[1] // 64 * 64)
        T, H, V, K = small
        n = f(*big, 1)
        assert _bwd(L, T=T, H=H, V=V, K=K, wsb=n) == DEVICE, (big, small)
        assert _fwd(L, T=T, H=H, V=V, K=K, wsb=n) == DEVICE, (big, small)


@pytest.mark.parametrize("T,H,V,K", [(300, 256, 5000, 8), (600, 4096, 33000, 24), (5980, 4096, 151936, 64),
                                     (512, 4096, 151936, 64), (1, 64, 20000, 3), (513, 1024, 32768, 32)])
def test_the_least_workspace_of_the_backward(L, T, H, V, K):
    least = _least(T, H, V, K)
    assert _bwd(L, T=T, H=H, V=V, K=K, wsb=least) == DEVICE
    assert _bwd(L, T=T, H=H, V=V, K=K, wsb=least - 1) == WS_SMALL
    assert L.rlk_linear_distill_workspace_bytes(T, H, V, K, 1) >= least


def test_the_few_row_order_keeps_to_its_bounds(L):
    """All of dX and one dHidden product per chunk, at most 256 MB each, beside the
    teacher's rows: not the chunk buffers that the order does not use."""
    f = L.rlk_linear_distill_workspace_bytes
    T, H, V, K = 512, 4096, 151936, 64
    rows = 3 * _a(T * K * 4) + 2 * _a(T * 4) + _a(T * 594 * 8)
    nc = 19
    assert f(T, H, V, K, 1) <= T * nc * 8192 * 2 + T * nc * H * 4 + rows + (1 << 16)
    T, H, V, K = 256, 8192, 524288, 8              # the products alone would take 512 MB
    assert f(T, H, V, K, 1) == max(_least(T, H, V, K), f(T, H, V, K, 0))
