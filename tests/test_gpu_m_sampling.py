"""rlk_token_probs and rlk_draft_verify against the fp64 oracle.

Tolerance of a probability (relative).  The exponent (x - m) log2(e) / tau, D
powers of two, takes a rounded factor (two half steps of 2^-24) and one or two
rounded operations more, the shift between two slices' maxima as many again: at
most 4 D ln2 2^-24 <= 3 D 2^-24.  Two ex2.approx of 2^-22 each, one division and one
product: 10 half steps of 2^-24.  The sum S carries the same errors averaged over
its terms (3 E[D] + 10) and its additions: a thread's entries of a slice (at most
102400 bytes over 256 threads: 200 in bf16, 100 in fp32; a long row's V / 4096), two
butterflies of 5 and 8 slices.  Together (3 D + 3 E[D] + n_thread + 40) 2^-24, plus what
flushes to zero below the smallest normal number.  bf16 storage adds half a step,
2^-8."""
import numpy as np
import pytest
import torch

from invariant_lm_head_gemm_b200 import binding
from oracle import sampling

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
EPS = 2.0 ** -24


def _tol(x, p, tau, dtype):
    x = x.astype(np.float64)
    fin = np.isfinite(x)
    D = np.where(fin, (x[fin].max() - np.where(fin, x, 0.0)) / tau * 1.4427, 0.0)
    per_thread = max(200, x.size // 4096 + 1)
    rel = (3 * D + 3 * float((p * D).sum()) + per_thread + 40) * EPS
    if dtype == BF16:
        return p * (rel + 2.0 ** -8) + 2.0 ** -125
    return p * rel + 2.0 ** -125


def _check_probs(x, t, got, dtype):
    """x: host fp32 [R, V]; t: list of temperatures."""
    got = got.float().cpu().numpy().astype(np.float64)
    for r in range(x.shape[0]):
        ref = sampling.token_probs(x[r], float(np.float32(t[r])))
        if np.isnan(ref).any():
            assert np.isnan(got[r]).all(), r
        elif t[r] == 0 or ref.sum() == 0:
            assert np.array_equal(got[r], ref), r
        else:
            d = np.abs(got[r] - ref)
            tol = _tol(x[r], ref, float(t[r]), dtype)
            assert np.all(d <= tol), (r, float((d - tol).max()))


def _logits(R, V, dtype, seed, scale=3.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (scale * torch.randn(R, V, generator=g, device="cuda")).to(dtype)


EDGES = [1, 2, 31, 33, 257, 2048, 2049, 8191, 8193, 20480, 20481, 40961, 50257, 81921, 151936, 163840,
         163841, 300007]


@pytest.mark.parametrize("V", EDGES)
def test_probs_match_the_oracle(V):
    x = _logits(5, V, F32, V)
    t = [1.0, 0.3, 0.0, 2.5, 0.05]
    got = binding.rlk_token_probs(x, torch.tensor(t, device="cuda"))
    assert got.dtype == F32
    _check_probs(x.cpu().numpy(), t, got, F32)


@pytest.mark.parametrize("V", [1, 100, 5001, 50257, 151936, 200001])
@pytest.mark.parametrize("src,dst", [(F32, BF16), (BF16, F32), (BF16, BF16)])
def test_probs_types(V, src, dst):
    x = _logits(3, V, src, V + 1)
    got = binding.rlk_token_probs(x, 0.7, dst)
    assert got.dtype == dst
    _check_probs(x.float().cpu().numpy(), [float(np.float32(0.7))] * 3, got, dst)


@pytest.mark.parametrize("V", [37, 2500, 50257, 170001])
def test_probs_masks_and_values_without_a_distribution(V):
    x = _logits(9, V, F32, 7)
    low = torch.finfo(F32).min
    x[0, 1:] = float("-inf")                       # one entry left
    x[1] = float("-inf")                           # nothing left
    x[2, : V // 2] = float("-inf")
    x[3] = low                                     # all at the lowest value: uniform
    x[4, V // 3:] = low
    x[5, V - 1] = float("nan")
    x[6, 0] = float("inf")
    x[7] = float("-inf")
    x[7, V - 1] = low
    t = [1.0, 1.0, 0.5, 1.0, 1.0, 1.0, 1.0, 2.0, 1.0]
    ws = binding.sampling_workspace()
    got = binding.rlk_token_probs(x, torch.tensor(t, device="cuda"), workspace=ws)
    _check_probs(x.cpu().numpy(), t, got, F32)
    assert binding.rlk_read_device_error(ws) == binding.RLK_DEVERR_PROBS
    clean = binding.rlk_token_probs(x[:1], 1.0, workspace=ws)
    assert binding.rlk_read_device_error(ws) == 0
    assert torch.equal(clean, got[:1])
    greedy = binding.rlk_token_probs(x, 0.0, workspace=ws)
    for r in range(9):
        ref = sampling.token_probs(x[r].cpu().numpy(), 0.0)
        assert np.array_equal(greedy[r].cpu().numpy().astype(np.float64), ref, equal_nan=True), r
    assert binding.rlk_read_device_error(ws) == binding.RLK_DEVERR_PROBS


@pytest.mark.parametrize("V", [300, 60001, 151936, 230000])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_probs_of_far_off_logits(V, dtype):
    """Rows far from zero, whole or in part: only differences count, however large
    the logits (or a mask's -1e9) are beside them."""
    base = _logits(8, V, F32, 15)
    t = [1.0, 0.5, 1.0, 1.0, 1.0, 0.01, 1.0, 1.0]
    off = [1e3, -3e5, 693147.0, -693140.0, -1e9, 1e4, 1e20, -2e38]
    x = base + torch.tensor(off, device="cuda")[:, None]
    x[2, V // 2:] -= 200.0                         # slices on both sides of the switch of form
    x[3, : V // 2] += 64.0
    x = x.to(dtype)
    got = binding.rlk_token_probs(x, torch.tensor(t, device="cuda"), F32)
    _check_probs(x.float().cpu().numpy(), t, got, F32)
    masked = _logits(2, V, F32, 16)
    masked[0, 3:] = -1e9
    masked[1, : V - 2] = -1e38
    _check_probs(masked.cpu().numpy(), [1.0, 0.3], binding.rlk_token_probs(
        masked, torch.tensor([1.0, 0.3], device="cuda")), F32)


def test_probs_row_temperatures_that_are_none():
    x = _logits(6, 3001, F32, 8)
    t = [-1.0, float("nan"), float("inf"), 1e-45, 1.0, 0.0]
    ws = binding.sampling_workspace()
    got = binding.rlk_token_probs(x, torch.tensor(t, device="cuda"), workspace=ws)
    assert torch.isnan(got[:4]).all()
    _check_probs(x[4:].cpu().numpy(), t[4:], got[4:], F32)
    assert binding.rlk_read_device_error(ws) == binding.RLK_DEVERR_PROBS


@pytest.mark.parametrize("V", [64, 8193, 151936, 170000])
def test_greedy_takes_the_first_of_equal_maxima(V):
    x = torch.zeros(4, V, device="cuda")
    x[1, [V // 2, V - 1]] = 1.0
    x[2, V - 1] = 0.5
    x[3, [V // 3, V // 3 + 1]] = 2.0
    got = binding.rlk_token_probs(x, 0.0, BF16).float()
    assert got.sum(1).tolist() == [1.0] * 4
    assert got.argmax(1).tolist() == [0, V // 2, V - 1, V // 3]


@pytest.mark.parametrize("V", [1000, 50257, 151937])
def test_probs_do_not_depend_on_the_batch_or_the_place(V):
    x = _logits(11, V, F32, 9)
    t = torch.linspace(0.2, 2.0, 11, device="cuda")
    full = binding.rlk_token_probs(x, t)
    for r in (0, 4, 10):
        one = binding.rlk_token_probs(x[r:r + 1].clone(), t[r:r + 1].clone())
        assert torch.equal(one[0].view(torch.int32), full[r].view(torch.int32))
    perm = torch.randperm(11, device="cuda")
    again = binding.rlk_token_probs(x[perm].contiguous(), t[perm].contiguous())
    assert torch.equal(again.view(torch.int32), full[perm].view(torch.int32))


def test_probs_strides_in_place_and_leading_shapes():
    V = 4099
    wide = _logits(6, V + 13, F32, 10)
    ref = binding.rlk_token_probs(wide[:, 5:5 + V].contiguous(), 0.9)
    got = binding.rlk_token_probs(wide[:, 5:5 + V], 0.9)
    assert torch.equal(got, ref)
    pad = torch.full((6, V + 3), 7.0, device="cuda")
    binding.rlk_token_probs(wide[:, 5:5 + V], 0.9, out=pad[:, 1:1 + V])
    assert torch.equal(pad[:, 1:1 + V], ref)
    assert (pad[:, 0] == 7).all() and (pad[:, 1 + V:] == 7).all()
    for vocab in (V, 170003):
        x = _logits(3, vocab, BF16, 11)
        want = binding.rlk_token_probs(x, 0.9)
        inplace = x.clone()
        assert binding.rlk_token_probs(inplace, 0.9, out=inplace) is inplace
        assert torch.equal(inplace, want)
    y = wide[:, :V].contiguous().view(2, 3, V)
    t = torch.tensor([[0.5, 1.0, 0.0], [2.0, 1.0, 0.25]], device="cuda")
    z = binding.rlk_token_probs(y, t)
    assert z.shape == y.shape
    assert torch.equal(z.view(6, V), binding.rlk_token_probs(y.view(6, V), t.view(6)))
    assert binding.rlk_token_probs(x[:0], 1.0).shape == (0, 170003)


@pytest.mark.parametrize("src,dst", [(F32, F32), (BF16, BF16), (F32, BF16), (BF16, F32)])
@pytest.mark.parametrize("V", [1, 5, 77, 4097, 60001])
def test_probs_at_every_alignment(src, dst, V):
    """The same bits wherever rows and outputs sit, and nothing written beside them."""
    x = _logits(3, V, src, 13)
    want = binding.rlk_token_probs(x, 0.8, dst)
    for shift in range(9):
        xs = torch.full((x.numel() + 24,), float("nan"), dtype=src, device="cuda")
        xs[shift:shift + x.numel()] = x.view(-1)
        ps = torch.full((x.numel() + 24,), 7.0, dtype=dst, device="cuda")
        at = (shift * 5) % 9
        out = ps[at:at + x.numel()].view(3, V)
        binding.rlk_token_probs(xs[shift:shift + x.numel()].view(3, V), 0.8, out=out)
        assert torch.equal(out, want)
        assert (ps[:at] == 7).all() and (ps[at + x.numel():] == 7).all()


def test_probs_offsets_past_32_bits():
    V, ld = 1000, (1 << 31) - 8
    base = torch.empty(ld + V, dtype=BF16, device="cuda")
    x = base.as_strided((2, V), (ld, 1))
    x.copy_(_logits(2, V, BF16, 12))
    got = binding.rlk_token_probs(x, 1.0, F32)
    assert torch.equal(got, binding.rlk_token_probs(x.contiguous(), 1.0, F32))
    _check_probs(x.float().cpu().numpy(), [1.0, 1.0], got, F32)


# ------------------------------------------------------------------ verification

def _verify_case(B, K, V, dtype, seed, lens=False, sharp=3.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = sharp * torch.randn(B, K + 1, V, generator=g, device="cuda")
    y = x[:, :K] + 0.8 * torch.randn(B, K, V, generator=g, device="cuda")
    p, q = torch.softmax(x, -1).to(dtype), torch.softmax(y, -1).to(dtype)
    race = torch.empty(B, K, V, device="cuda").exponential_(generator=g)
    d = (q.float() / race).argmax(-1)
    ua = torch.rand(B, K, generator=g, device="cuda")
    us = torch.rand(B, generator=g, device="cuda")
    n = torch.randint(0, K + 1, (B,), generator=g, device="cuda") if lens else None
    return p, q, d, ua, us, n


def _np(t):
    return None if t is None else t.float().cpu().numpy().astype(np.float64) if t.is_floating_point() \
        else t.cpu().numpy()


def _check_verify(p, q, d, ua, us, n, got):
    tok, acc = sampling.draft_verify(_np(p), _np(q), _np(d), _np(ua), _np(us), _np(n))
    assert np.array_equal(got[1].cpu().numpy(), acc)
    assert np.array_equal(got[0].cpu().numpy(), tok)


@pytest.mark.parametrize("V", [1, 2, 33, 511, 4096, 4097, 16385, 50257, 65537, 151936])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_verify_matches_the_oracle(V, dtype):
    c = _verify_case(12, 4, V, dtype, V)
    _check_verify(*c, binding.rlk_draft_verify(*c))


@pytest.mark.parametrize("B,K,V,lens", [(1, 0, 1000, False), (1, 1, 151936, False), (300, 7, 777, True),
                                        (7, 33, 2000, True), (3, 70, 900, False), (64, 2, 300007, True)])
def test_verify_batches_and_lengths(B, K, V, lens):
    c = _verify_case(B, K, V, F32, B + K, lens)
    ws = binding.sampling_workspace()
    _check_verify(*c, binding.rlk_draft_verify(*c, workspace=ws))
    p, q, d, ua, us, n = c
    _check_verify(p, None, d, ua, us, n, binding.rlk_draft_verify(p, None, d, ua, us, n, workspace=ws))
    assert binding.rlk_read_device_error(ws) == 0


@pytest.mark.parametrize("V", [40, 5000, 151936])
def test_verify_extremes(V):
    """Everything accepted; everything refused; numbers at and past the ends of
    [0, 1); a draft equal to the target (nothing left of the residual)."""
    B, K = 6, 3
    p, q, d, ua, us, _ = _verify_case(B, K, V, F32, V + 5)
    us = torch.tensor([0.0, 1 - 2.0 ** -24, 1.0, 1.5, float("nan"), 0.5], device="cuda")
    all_in = (p, q, d, torch.zeros_like(ua), us, None)
    got = binding.rlk_draft_verify(*all_in)
    assert got[1].tolist() == [K] * B
    _check_verify(*all_in, got)
    one = torch.zeros_like(q).scatter_(2, d[..., None], 1.0)
    none_in = (p, one, d, torch.full_like(ua, 1 - 2.0 ** -24), us, None)
    got = binding.rlk_draft_verify(*none_in)
    assert got[1].tolist() == [0] * B
    _check_verify(*none_in, got)
    # q = p but for u = 1: refused with an empty residual, so the target's own row
    same = (p, p[:, :K].clone(), d, torch.ones_like(ua), us, None)
    got = binding.rlk_draft_verify(*same)
    assert got[1].tolist() == [0] * B
    _check_verify(*same, got)
    lens = torch.tensor([-5, 0, 1, 3, 99, 2], device="cuda")
    some = (p, q, d, ua, us, lens)
    _check_verify(*some, binding.rlk_draft_verify(*some))


def test_verify_single_survivors_at_every_place():
    """All the residual on one token, at segment and lane borders."""
    V = 20000
    at = torch.tensor([0, 1, 31, 32, 63, 319, 320, 321, 1023, 1024, 9999, 10239, 10240, 19998, 19999],
                      device="cuda")
    B = at.numel()
    p = torch.zeros(B, 1, V, device="cuda").scatter_(2, at[:, None, None], 1.0)
    z = torch.zeros(B, 0, dtype=torch.int64, device="cuda")
    for u in (0.0, 0.5, 1 - 2.0 ** -24):
        tok, n = binding.rlk_draft_verify(p, None, z, torch.zeros(B, 0, device="cuda"),
                                          torch.full((B,), u, device="cuda"))
        assert tok[:, 0].tolist() == at.tolist() and n.tolist() == [0] * B


def test_verify_borders_between_tokens():
    """Equal powers of two: u at k / V falls exactly on a border and belongs to
    token k."""
    V = 4096
    k = torch.tensor([0, 1, 2, 255, 256, 1000, 2048, 4095], device="cuda")
    p = torch.full((8, 1, V), 1.0 / V, device="cuda")
    z = torch.zeros(8, 0, dtype=torch.int64, device="cuda")
    none = torch.zeros(8, 0, device="cuda")
    tok, _ = binding.rlk_draft_verify(p, None, z, none, k.float() / V)
    assert tok[:, 0].tolist() == k.tolist()
    tok, _ = binding.rlk_draft_verify(p, None, z, none, (k.float() + 1 - 2.0 ** -11) / V)
    assert tok[:, 0].tolist() == k.tolist()


def test_verify_bad_tokens_and_rows_without_a_distribution():
    B, K, V = 6, 2, 3000
    p, q, d, ua, us, _ = _verify_case(B, K, V, F32, 77)
    good = binding.rlk_draft_verify(p, q, d, ua, us)
    ws = binding.sampling_workspace()
    bad = d.clone()
    bad[1, 0], bad[2, 0], bad[3, 1] = V, -1, 1 << 40
    got = binding.rlk_draft_verify(p, q, bad, ua, us, workspace=ws)
    _check_verify(p, q, bad, ua, us, None, got)
    assert got[1][1] == 0 and got[1][2] == 0 and got[1][3] <= 1
    assert binding.rlk_read_device_error(ws) == binding.RLK_DEVERR_TARGET
    for b in (0, 4, 5):
        assert torch.equal(got[0][b], good[0][b])
    # what lies behind a sequence's length is not looked at
    lens = torch.tensor([2, 0, 0, 1, 2, 2], device="cuda")
    got = binding.rlk_draft_verify(p, q, bad, ua, us, lens, workspace=ws)
    _check_verify(p, q, bad, ua, us, lens, got)
    assert binding.rlk_read_device_error(ws) == 0
    pn = p.clone()
    pn[0, :, 5] = float("nan")
    pn[1] = 0
    pn[2, :, 9] = float("inf")
    got = binding.rlk_draft_verify(pn, q, d, ua, us, workspace=ws)
    _check_verify(pn, q, d, ua, us, None, got)
    assert binding.rlk_read_device_error(ws) == binding.RLK_DEVERR_PROBS
    assert got[0][0, got[1][0]] == -1 and got[0][1, 0] == -1
    for b in (3, 4, 5):
        assert torch.equal(got[0][b], good[0][b])
    # in the draft's rows they matter where a draft is refused
    for value in (float("nan"), float("inf")):
        qn = q.clone()
        qn[:, :, V - 1] = value
        got = binding.rlk_draft_verify(p, qn, d, ua, us, workspace=ws)
        _check_verify(p, qn, d, ua, us, None, got)
        refused = got[1] < K
        assert refused.any() and (got[0][refused, got[1][refused]] == -1).all()
        assert binding.rlk_read_device_error(ws) == binding.RLK_DEVERR_PROBS


def test_verify_subnormal_and_unnormalised_rows():
    """Probabilities down to the smallest subnormals, and rows that sum to
    anything: only their proportions count."""
    B, V = 8, 1500
    g = torch.Generator(device="cuda").manual_seed(9)
    p = torch.rand(B, 2, V, generator=g, device="cuda")
    p[0] *= 1e-42
    p[1] = (p[1] * 4).floor() * 2.0 ** -149
    p[2] *= 1e30
    p[3, :, ::2] = 0
    p[4, :, : V - 1] *= 1e-30
    q = p[:, :1] * torch.rand(B, 1, V, generator=g, device="cuda") * 1.5
    d = torch.full((B, 1), 3, device="cuda")
    ua = torch.rand(B, 1, generator=g, device="cuda")
    us = torch.rand(B, generator=g, device="cuda")
    for ua_k in (ua, torch.ones_like(ua), torch.zeros_like(ua)):
        _check_verify(p, q, d, ua_k, us, None, binding.rlk_draft_verify(p, q, d, ua_k, us))


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_verify_writes_its_outputs_only_and_any_alignment(dtype):
    B, K, V = 6, 3, 1537
    p, q, d, ua, us, _ = _verify_case(B, K, V, dtype, 51)
    ref = binding.rlk_draft_verify(p, q, d, ua, us)
    room = torch.full((B * (K + 1) + 16,), 77, dtype=torch.int64, device="cuda")
    count = torch.full((B + 16,), 77, dtype=torch.int64, device="cuda")
    out = (room[8:8 + B * (K + 1)].view(B, K + 1), count[8:8 + B])
    for shift in range(1, 9):                      # every offset of the rows within 16 bytes
        ps = torch.empty(p.numel() + shift, dtype=dtype, device="cuda")[shift:].view(p.shape)
        qs = torch.empty(q.numel() + 2 * shift, dtype=dtype, device="cuda")[2 * shift:].view(q.shape)
        ps.copy_(p)
        qs.copy_(q)
        binding.rlk_draft_verify(ps, qs, d, ua, us, out=out)
        assert torch.equal(out[0], ref[0]) and torch.equal(out[1], ref[1])
        assert (room[:8] == 77).all() and (room[-8:] == 77).all()
        assert (count[:8] == 77).all() and (count[-8:] == 77).all()


def test_verify_strides():
    B, K, V = 5, 3, 2001
    p, q, d, ua, us, _ = _verify_case(B, K, V, BF16, 31)
    ref = binding.rlk_draft_verify(p, q, d, ua, us)
    wide = torch.full((K + 1, B, V + 9), float("nan"), dtype=BF16, device="cuda")
    wide[:, :, 3:3 + V] = p.transpose(0, 1)
    got = binding.rlk_draft_verify(wide[:, :, 3:3 + V].transpose(0, 1), q, d, ua, us)
    assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])
    shared = q[:1, :1].expand(B, K, V)
    got = binding.rlk_draft_verify(p, shared, d, ua, us)
    want = binding.rlk_draft_verify(p, shared.contiguous(), d, ua, us)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_verify_offsets_past_32_bits():
    B, K, V = 2, 1, 500
    p, q, d, ua, us, _ = _verify_case(B, K, V, BF16, 41)
    far = (1 << 31) + 16
    base = torch.empty(far + 2 * V, dtype=BF16, device="cuda")
    pp = base.as_strided((B, K + 1, V), (far, V, 1))
    pp.copy_(p)
    got = binding.rlk_draft_verify(pp, q, d, ua, us)
    want = binding.rlk_draft_verify(p, q, d, ua, us)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


# ------------------------------------------------------------------ calls

def test_many_short_rows():
    x = _logits(100003, 5, F32, 17)
    got = binding.rlk_token_probs(x, 0.9)
    want = torch.softmax(x.double() / float(np.float32(0.9)), 1)
    assert ((got.double() - want).abs() <= want * 300 * EPS).all()
    c = _verify_case(20011, 2, 9, BF16, 18, True)
    tok, n = binding.rlk_draft_verify(*c)
    sel = torch.randperm(20011, device="cuda")[:300]
    _check_verify(*[t[sel].contiguous() for t in c], (tok[sel], n[sel]))


def test_binding_refusals():
    x = torch.zeros(2, 8, device="cuda")
    for bad in (lambda: binding.rlk_token_probs(x.double()),
                lambda: binding.rlk_token_probs(x.t()),
                lambda: binding.rlk_token_probs(x[:1].expand(2, 8)),
                lambda: binding.rlk_token_probs(x[:, :0]),
                lambda: binding.rlk_token_probs(x, torch.ones(3, device="cuda")),
                lambda: binding.rlk_token_probs(x, torch.ones(2)),
                lambda: binding.rlk_token_probs(x, 1.0, torch.float16),
                lambda: binding.rlk_token_probs(x, out=torch.zeros(2, 9, device="cuda")),
                lambda: binding.rlk_token_probs(x, workspace=torch.zeros(256, dtype=torch.uint8))):
        with pytest.raises(ValueError):
            bad()
    for tau in (-1.0, float("nan"), float("inf")):
        with pytest.raises(binding.RlkError):
            binding.rlk_token_probs(x, tau)
    p, q, d, ua, us, _ = _verify_case(2, 2, 16, F32, 1)
    ok = dict(target_probs=p, draft_probs=q, draft_tokens=d, u_accept=ua, u_sample=us)
    binding.rlk_draft_verify(**ok)
    for k, v in (("target_probs", p[0]), ("target_probs", p.double()), ("draft_probs", q.to(BF16)),
                 ("draft_probs", q[:, :1]), ("draft_tokens", d.int()), ("draft_tokens", d[:, :1]),
                 ("u_accept", ua.double()), ("u_sample", us[:1]), ("u_sample", us.cpu()),
                 ("target_probs", p.transpose(1, 2).contiguous().transpose(1, 2))):
        with pytest.raises(ValueError):
            binding.rlk_draft_verify(**{**ok, k: v})
    with pytest.raises(ValueError):
        binding.rlk_draft_verify(**ok, draft_lens=torch.zeros(2, dtype=torch.int32, device="cuda"))


def test_graphs_and_streams():
    """One captured graph of draft probabilities, target probabilities and the
    verification, replayed on new logits; and the same calls on a side stream."""
    B, K, V = 4, 3, 10007
    ws = binding.sampling_workspace()
    g = torch.Generator(device="cuda").manual_seed(3)
    xt = torch.randn(B, K + 1, V, generator=g, device="cuda")
    xd = torch.randn(B, K, V, generator=g, device="cuda")
    d = torch.randint(0, V, (B, K), generator=g, device="cuda")
    ua = torch.rand(B, K, generator=g, device="cuda")
    us = torch.rand(B, generator=g, device="cuda")
    tau = torch.full((B, K + 1), 0.8, device="cuda")
    p, q = torch.empty_like(xt), torch.empty_like(xd)
    out = (torch.empty(B, K + 1, dtype=torch.int64, device="cuda"),
           torch.empty(B, dtype=torch.int64, device="cuda"))

    def step(stream=None):
        binding.rlk_token_probs(xt, tau, out=p, workspace=ws, stream=stream)
        binding.rlk_token_probs(xd, 1.0, out=q, workspace=ws, stream=stream)
        binding.rlk_draft_verify(p, q, d, ua, us, out=out, workspace=ws, stream=stream)

    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for k in range(3):
        xt.copy_(2 * torch.randn(B, K + 1, V, generator=g, device="cuda"))
        xd.copy_(xt[:, :K] + 0.5 * torch.randn(B, K, V, generator=g, device="cuda"))
        d.copy_(xd.argmax(-1))
        graph.replay()
        _check_verify(p, q, d, ua, us, None, out)
        kept = [t.clone() for t in out]
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        step(side)
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(out[0], kept[0]) and torch.equal(out[1], kept[1])
    assert binding.rlk_read_device_error(ws) == 0
