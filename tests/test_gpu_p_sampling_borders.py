"""The lengths at which rlk_token_probs and rlk_draft_verify change their form, from
both sides.  Rows go to a cluster of 1, 2, 4 or 8 CTAs that hold 102400 bytes each, and
past those to the kernel that reads its row again; a row of at most 2048 entries has
small CTAs; a verified row's segments are 256 entries up to 640 of them, then 512.
Tolerances: tests/test_gpu_m_sampling.py."""
import numpy as np
import pytest
import torch

from invariant_lm_head_gemm_b200 import binding
from oracle import sampling
from tests.test_gpu_m_sampling import BF16, F32, _check_probs, _check_verify, _logits, _verify_case

pytestmark = pytest.mark.gpu

PAIRS = [(F32, F32), (F32, BF16), (BF16, F32), (BF16, BF16)]
ENTRIES = {F32: 25600, BF16: 51200}               # of one CTA
LONG = {F32: 204800 + 77, BF16: 409600 + 77}      # rows of the kernel for long ones


def _host(x):
    return x.float().cpu().numpy()


@pytest.mark.parametrize("src,dst", PAIRS)
@pytest.mark.parametrize("ctas", [1, 2, 4, 8])
@pytest.mark.parametrize("past", [0, 1])
def test_probs_at_the_borders(src, dst, ctas, past):
    V = ENTRIES[src] * ctas + past
    x = _logits(3, V, src, V)
    x[2, V - 1] = 20.0                             # the last entry counts
    t = [1.0, 0.4, 1.3]
    got = binding.rlk_token_probs(x, torch.tensor(t, device="cuda"), dst)
    _check_probs(_host(x), t, got, dst)
    assert float(got[2, V - 1]) > 0.1


@pytest.mark.parametrize("src,dst", PAIRS)
@pytest.mark.parametrize("V", [2047, 2048, 2049])
def test_probs_at_the_border_of_short_rows(src, dst, V):
    x = _logits(4, V, src, V)
    t = [1.0, 0.4, 1.3, 0.0]
    _check_probs(_host(x), t, binding.rlk_token_probs(x, torch.tensor(t, device="cuda"), dst), dst)


@pytest.mark.parametrize("src,dst", PAIRS)
def test_long_rows_masks_and_rows_without_a_distribution(src, dst):
    V = LONG[src]
    x = _logits(10, V, src, 5)
    low = torch.finfo(src).min
    x[0, 1:] = float("-inf")
    x[1] = float("-inf")
    x[2, : V // 2] = float("-inf")                 # whole CTAs of nothing
    x[3] = low
    x[4, V // 3:] = low
    x[5, V - 1] = float("nan")
    x[6, 0] = float("inf")
    x[7] = float("-inf")
    x[7, V - 1] = low
    x[8, V // 5] = float("nan")
    t = [1.0, 1.0, 0.5, 1.0, 1.0, 1.0, 1.0, 2.0, 0.7, 1.0]
    ws = binding.sampling_workspace()
    got = binding.rlk_token_probs(x, torch.tensor(t, device="cuda"), dst, workspace=ws)
    _check_probs(_host(x), t, got, dst)
    assert binding.rlk_read_device_error(ws) == binding.RLK_DEVERR_PROBS
    greedy = binding.rlk_token_probs(x, 0.0, dst, workspace=ws)
    for r in range(10):
        ref = sampling.token_probs(_host(x[r]), 0.0)
        assert np.array_equal(_host(greedy[r]).astype(np.float64), ref, equal_nan=True), r
    assert binding.rlk_read_device_error(ws) == binding.RLK_DEVERR_PROBS
    for tau in (-1.0, float("nan"), float("inf"), 1e-45):
        bad = binding.rlk_token_probs(x[9:], torch.full((1,), tau, device="cuda"), dst, workspace=ws)
        assert torch.isnan(bad).all()
        assert binding.rlk_read_device_error(ws) == binding.RLK_DEVERR_PROBS
    assert torch.equal(binding.rlk_token_probs(x[9:], 1.0, dst, workspace=ws), got[9:])
    assert binding.rlk_read_device_error(ws) == 0


@pytest.mark.parametrize("src,dst", PAIRS)
@pytest.mark.parametrize("V", ["long", "cluster"])
def test_the_first_of_equal_maxima_in_every_slice(src, dst, V):
    V = LONG[src] if V == "long" else ENTRIES[src] * 8
    x = torch.zeros(6, V, device="cuda")
    at = [(0, V - 1), (V // 8 - 1, V // 8), (V // 2, V // 2 + 1), (V - 2, V - 1), (V // 3, V // 2), (V - 1,)]
    for r, places in enumerate(at):
        x[r, list(places)] = 1.5
    got = binding.rlk_token_probs(x.to(src), 0.0, dst).float()
    assert got.sum(1).tolist() == [1.0] * 6
    assert got.argmax(1).tolist() == [min(places) for places in at]


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_long_rows_in_place_at_an_offset_and_in_any_batch(dtype):
    V = LONG[dtype]
    x = _logits(4, V, dtype, 6)
    t = torch.tensor([1.0, 0.0, 0.3, 2.0], device="cuda")
    want = binding.rlk_token_probs(x, t)
    inplace = x.clone()
    assert binding.rlk_token_probs(inplace, t, out=inplace) is inplace
    assert torch.equal(inplace, want)
    for r in range(4):
        assert torch.equal(binding.rlk_token_probs(x[r:r + 1].clone(), t[r:r + 1].clone())[0], want[r])
    wide = torch.full((4, V + 9), float("nan"), dtype=dtype, device="cuda")
    wide[:, 3:3 + V] = x
    out = torch.full((4, V + 5), 7.0, dtype=dtype, device="cuda")
    binding.rlk_token_probs(wide[:, 3:3 + V], t, out=out[:, 2:2 + V])
    assert torch.equal(out[:, 2:2 + V], want)
    assert (out[:, :2] == 7).all() and (out[:, 2 + V:] == 7).all()


@pytest.mark.parametrize("V", [163840, 163841, 327680, 327681])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_verify_at_the_borders_of_the_segments(V, dtype):
    c = _verify_case(6, 2, V, dtype, V)
    _check_verify(*c, binding.rlk_draft_verify(*c))
    p, q, d, ua, us, _ = c
    _check_verify(p, None, d, ua, us, None, binding.rlk_draft_verify(p, None, d, ua, us))
    # all on one token: the last entry, and both sides of a segment
    for at in (0, 255, 256, 511, 512, V - 2, V - 1):
        one = torch.zeros(2, 1, V, dtype=dtype, device="cuda")
        one[:, 0, at] = 0.75
        tok, n = binding.rlk_draft_verify(one, None, d[:2, :0].contiguous(), ua[:2, :0].contiguous(),
                                          torch.tensor([0.0, 1 - 2.0 ** -24], device="cuda"))
        assert tok[:, 0].tolist() == [at, at] and n.tolist() == [0, 0]


@pytest.mark.parametrize("V", [163841, 300007])
def test_verify_long_bf16_rows_at_every_alignment(V):
    B, K = 3, 1
    p, q, d, ua, us, _ = _verify_case(B, K, V, BF16, V + 1)
    want = binding.rlk_draft_verify(p, q, d, ua, us)
    _check_verify(p, q, d, ua, us, None, want)
    for shift in range(1, 9):
        ps = torch.empty(p.numel() + shift, dtype=BF16, device="cuda")[shift:].view(p.shape)
        qs = torch.empty(q.numel() + 2 * shift + 1, dtype=BF16, device="cuda")[2 * shift + 1:].view(q.shape)
        ps.copy_(p)
        qs.copy_(q)
        got = binding.rlk_draft_verify(ps, qs, d, ua, us)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
