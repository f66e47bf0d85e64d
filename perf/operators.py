"""Measured cases of the distillation and draft-verification operators.

Three operators, named by a case's "op":

  distill   the distillation loss of a student's LM head on a teacher's top
            logits, alone ("score") or with its gradients ("train"; "frozen":
            the head is shared and frozen, so only the hidden states' gradient)
  probs     probabilities of rows of logits at each row's temperature
  verify    acceptance of drafted tokens and the one token sampled after them

run() computes them in elementary torch operations, or through this package
where `own` is set.
"""
import math

import torch

own = False
_binding = None  # this package's binding, imported when its operators are asked for

_BF16, _F32, _F64 = torch.bfloat16, torch.float32, torch.float64
_TYPES = {"bf16": _BF16, "fp32": _F32}


def _own():
    global _binding
    if _binding is None:
        from invariant_lm_head_gemm_b200 import binding
        _binding = binding
    return _binding


def listed():
    return [
        # scoring a few tokens against a teacher (the short-batch forward)
        dict(name="distill score T16", op="distill", kind="score", T=16, H=4096, V=151936, K=20,
             teacher="fp32", tau=1.0, tail=True),
        # a test-sized step, where latency counts
        dict(name="distill train tiny", op="distill", kind="train", T=64, H=256, V=1024, K=8,
             teacher="fp32", tau=1.0, tail=False),
        # a small student at a soft temperature
        dict(name="distill train small", op="distill", kind="train", T=513, H=1024, V=32768, K=32,
             teacher="bf16", tau=2.0, tail=False),
        # a draft model that shares the target's frozen head
        dict(name="distill frozen head", op="distill", kind="frozen", T=2047, H=4096, V=151936, K=64,
             teacher="bf16", tau=1.0, tail=True),
        # a whole step of packed sequences
        dict(name="distill train step", op="distill", kind="train", T=5980, H=4096, V=151936, K=64,
             teacher="fp32", tau=1.0, tail=False),
        # one request's next token
        dict(name="probs one row", op="probs", R=1, V=151936, src="fp32", dst="fp32", greedy=0.0,
             masked=0.0),
        # 64 requests with four drafts each and a temperature of their own, some greedy
        dict(name="probs 64 x 5", op="probs", R=320, V=151936, src="fp32", dst="fp32", greedy=0.1,
             masked=0.0),
        # rows under a grammar's mask, an odd vocabulary, halved storage
        dict(name="probs masked bf16", op="probs", R=1027, V=50257, src="bf16", dst="bf16", greedy=0.0,
             masked=0.9),
        # one request with four drafts
        dict(name="verify one", op="verify", B=1, K=4, V=151936, dtype="fp32", draft=True, ragged=False),
        # a batch of requests
        dict(name="verify 64", op="verify", B=64, K=4, V=151936, dtype="fp32", draft=True, ragged=False),
        # many short requests with drafts of several lengths, an odd vocabulary
        dict(name="verify 256 ragged", op="verify", B=256, K=7, V=50257, dtype="bf16", draft=True,
             ragged=True),
        # drafts looked up in the prompt: no draft probabilities
        dict(name="verify looked up", op="verify", B=48, K=10, V=32768, dtype="fp32", draft=False,
             ragged=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["distill", "distill", "probs", "verify"])
    V = min(151936, _log_int(rng, 1000, 170000))
    if op == "distill":
        H = 64 * _log_int(rng, 1, 64)
        T = min(_log_int(rng, 1, 5980), max(1, 5980 * 4096 * 151936 // (H * V)))
        return dict(op=op, kind=rng.choice(["score", "train", "train", "frozen"]), T=T, H=H, V=V,
                    K=_log_int(rng, 1, 128), teacher=rng.choice(["fp32", "bf16"]),
                    tau=rng.choice([0.7, 1.0, 2.0]), tail=rng.random() < 0.5)
    if op == "probs":
        R = min(_log_int(rng, 1, 4096), max(1, 320 * 151936 // V))
        return dict(op=op, R=R, V=V, src=rng.choice(["fp32", "bf16"]), dst=rng.choice(["fp32", "bf16"]),
                    greedy=rng.choice([0.0, 0.1]), masked=rng.choice([0.0, 0.5, 0.9]))
    K = rng.randint(0, 12)
    B = min(_log_int(rng, 1, 256), max(1, 64 * 9 * 151936 // ((2 * K + 1) * V)))
    return dict(op=op, B=B, K=K, V=V, dtype=rng.choice(["fp32", "bf16"]), draft=rng.random() < 0.7,
                ragged=rng.random() < 0.5)


# ------------------------------------------------------------------ inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed * 2654435761 % (1 << 62))


def _prepare_distill(c, g):
    T, H, V, K = c["T"], c["H"], c["V"], min(c["K"], c["V"])
    std = 1.28 / math.sqrt(H)  # logits of a spread of 1.28, as at H = 4096 with weights of 0.02
    W = torch.empty(V, H, dtype=_F32, device="cuda").normal_(0.0, std, generator=g).to(_BF16)
    # distinct ids, denser towards the frequent (low) ones, in no order
    u = torch.rand(T, K, generator=g, device="cuda", dtype=_F64)
    ids = ((V - K + 1) * u * u).long().clamp_(max=V - K).sort(1).values
    ids = ids + torch.arange(K, device="cuda")
    ids = ids.gather(1, torch.rand(T, K, generator=g, device="cuda").argsort(1))
    logits = (4.0 + 2.0 * torch.randn(T, K, generator=g, device="cuda")).sort(1, descending=True).values
    # the student leans towards the teacher's first choice
    lean = 0.6 * math.log(V) / (std * std * H)
    hidden = torch.randn(T, H, generator=g, device="cuda")
    hidden = (hidden + lean * W[ids[:, 0]].float()).to(_BF16)
    # a tenth of the rows carry no loss (prompts), a third have fewer slots; what lies there is not looked at
    count = torch.full((T,), K, device="cuda")
    some = torch.rand(T, generator=g, device="cuda")
    count = torch.where(some < 0.33, 1 + (torch.rand(T, generator=g, device="cuda") * K).long(), count)
    count = torch.where(some < 0.1, 0, count).clamp(max=K)
    count[0] = K
    unused = torch.arange(K, device="cuda") >= count[:, None]
    # the teacher's own lse lies above that of its top logits
    s = dict(lse=None)
    if c["tail"]:
        scaled = logits.to(_TYPES[c["teacher"]]).float() / c["tau"]
        s["lse"] = torch.logsumexp(scaled.masked_fill(unused, -1e30), 1) + \
            0.3 * torch.rand(T, generator=g, device="cuda")
        s["lse"] = torch.where(count == 0, 0.0, s["lse"])
    s["ids"] = ids.masked_fill(unused, -1)
    s["logits"] = logits.masked_fill(unused, float("nan")).to(_TYPES[c["teacher"]])
    s["dloss"] = (0.5 + torch.rand(T, generator=g, device="cuda")) / T
    s["hidden"], s["W"] = hidden, W
    return s


def _prepare_probs(c, g):
    R, V = c["R"], c["V"]
    x = 3.0 * torch.randn(R, V, generator=g, device="cuda")
    if c["masked"]:
        off = torch.rand(R, V, generator=g, device="cuda") < c["masked"]
        off[:, V // 2] = False
        x.masked_fill_(off, float("-inf"))
    t = 0.3 + torch.rand(R, generator=g, device="cuda")
    t[torch.rand(R, generator=g, device="cuda") < c["greedy"]] = 0.0
    s = dict(x=x.to(_TYPES[c["src"]]), t=t)
    return s


def _prepare_verify(c, g):
    B, K, V = c["B"], c["K"], c["V"]
    dt = _TYPES[c["dtype"]]
    x = 3.0 * torch.randn(B, K + 1, V, generator=g, device="cuda")
    s = dict(p=torch.softmax(x, -1).to(dt), q=None, lens=None)
    y = x[:, :K] + 0.7 * torch.randn(B, K, V, generator=g, device="cuda")
    q = torch.softmax(y, -1)
    if c["draft"]:
        s["q"] = q.to(dt)
    # drafts drawn from the draft's own distribution (the least exponential of a race)
    race = torch.empty(B, K, V, device="cuda").exponential_(generator=g)
    s["d"] = (q / race).argmax(-1) if c["draft"] else y.argmax(-1)
    s["ua"] = torch.rand(B, K, generator=g, device="cuda")
    s["us"] = torch.rand(B, generator=g, device="cuda")
    if c["ragged"]:
        s["lens"] = (torch.rand(B, generator=g, device="cuda") * (K + 1)).long().clamp_(max=K)
        s["d"] = s["d"].masked_fill(torch.arange(K, device="cuda") >= s["lens"][:, None], -1)
    return s


def prepare(case, seed):
    g = _gen(seed)
    s = {"distill": _prepare_distill, "probs": _prepare_probs, "verify": _prepare_verify}[case["op"]](case, g)
    s["case"] = case
    if own:  # the scratch that a program keeps for its calls
        if case["op"] == "distill":
            s["ws"] = _own().make_distill_workspace(case["T"], case["H"], case["V"], s["ids"].shape[1],
                                                    case["kind"] != "score")
        else:
            s["ws"] = _own().sampling_workspace()
    return s


# ------------------------------------------------------------------ the plain forms

def _plain_distill(s):
    c = s["case"]
    h, W, tau = s["hidden"].float(), s["W"].float(), c["tau"]
    used = s["ids"] >= 0
    ids = s["ids"].clamp(min=0)
    a = torch.where(used, s["logits"].float() / tau, float("-inf"))
    top = a.max(1, keepdim=True).values
    any_used = top > float("-inf")
    top = torch.where(any_used, top, 0.0)
    L = s["lse"][:, None] if s["lse"] is not None else \
        top + (a - top).exp().sum(1, keepdim=True).clamp(min=1e-38).log()
    logq = torch.where(used, a - L, 0.0)
    q = torch.where(used, logq.exp(), 0.0)
    z = h @ W.t() / tau
    m = z.max(1, keepdim=True).values
    lse = m + (z - m).exp().sum(1, keepdim=True).log()
    loss = torch.where(used, q * (logq - z.gather(1, ids) + lse), 0.0).sum(1)
    if c["kind"] == "score":
        return {"loss": loss, "lse": lse[:, 0]}
    z.sub_(lse).exp_().mul_(q.sum(1, keepdim=True))
    z.scatter_add_(1, ids, -q)
    z.mul_(s["dloss"][:, None] / tau)
    out = {"loss": loss, "dhidden": (z @ W).to(_BF16)}
    if c["kind"] == "train":
        out["dW"] = (z.t() @ h).to(_BF16)
    return out


def _plain_probs(s):
    x, t = s["x"].float(), s["t"][:, None]
    m = x.max(1, keepdim=True).values
    e = ((x - m) / torch.where(t > 0, t, 1.0)).exp()
    p = e / e.sum(1, keepdim=True)
    at = torch.arange(x.shape[1], device=x.device)
    first = torch.where(x == m, at, x.shape[1]).min(1, keepdim=True).values
    p = torch.where(t > 0, p, (at == first).float())
    return {"probs": p.to(_TYPES[s["case"]["dst"]])}


def _plain_verify(s):
    p, q, d = s["p"], s["q"], s["d"]
    B, K1, V = p.shape
    K = K1 - 1
    at = torch.arange(K1, device=p.device)
    lens = s["lens"] if s["lens"] is not None else torch.full((B,), K, device=p.device)
    tok = d.clamp(min=0)[..., None]
    pd = p[:, :K].gather(2, tok)[..., 0].double()
    qd = q.gather(2, tok)[..., 0].double() if q is not None else torch.ones_like(pd)
    ok = (s["ua"].double() * qd < pd) & (at[:K] < lens[:, None])
    n = ok.long().cumprod(1).sum(1)
    r = p[torch.arange(B, device=p.device), n].double()
    row = r
    if K:
        i = n.clamp(max=K - 1)
        if q is not None:
            qr = q[torch.arange(B, device=p.device), i].double()
        else:
            qr = (torch.arange(V, device=p.device) == tok[torch.arange(B, device=p.device), i]).double()
        r = torch.where((n < lens)[:, None], (r - qr).clamp(min=0), r)
    r = torch.where(r.sum(1, keepdim=True) > 0, r, row)
    cum = r.cumsum(1)
    over = cum > s["us"].double()[:, None] * r.sum(1, keepdim=True)
    v = torch.arange(V, device=p.device)
    first = torch.where(over, v, V).min(1).values
    last = torch.where(r > 0, v, -1).max(1).values
    pick = torch.where(first < V, first, last)
    drafted = torch.cat([d, d.new_full((B, 1), -1)], 1)
    tokens = torch.where(at < n[:, None], drafted, torch.where(at == n[:, None], pick[:, None], -1))
    return {"tokens": tokens, "accepted": n}


def run(state):
    s, c = state, state["case"]
    if not own:
        return {"distill": _plain_distill, "probs": _plain_probs, "verify": _plain_verify}[c["op"]](s)
    b = _own()
    if c["op"] == "probs":
        return {"probs": b.rlk_token_probs(s["x"], s["t"], _TYPES[c["dst"]], workspace=s["ws"])}
    if c["op"] == "verify":
        tokens, n = b.rlk_draft_verify(s["p"], s["q"], s["d"], s["ua"], s["us"], s["lens"], workspace=s["ws"])
        return {"tokens": tokens, "accepted": n}
    loss, lse = b.rlk_linear_distill_fwd(s["hidden"], s["W"], s["ids"], s["logits"], c["tau"],
                                         teacher_lse=s["lse"], workspace=s["ws"])
    if c["kind"] == "score":
        return {"loss": loss, "lse": lse}
    dh, dW = b.rlk_linear_distill_bwd(s["hidden"], s["W"], s["ids"], s["logits"], c["tau"], lse, s["dloss"],
                                      teacher_lse=s["lse"], workspace=s["ws"],
                                      dW_dtype=_BF16 if c["kind"] == "train" else None)
    out = {"loss": loss, "dhidden": dh}
    if c["kind"] == "train":
        out["dW"] = dW
    return out


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    c = case
    if c["op"] == "distill":
        T, H, V, K = c["T"], c["H"], c["V"], min(c["K"], c["V"])
        nbytes = 2 * H * (T + V) + T * K * (8 + (4 if c["teacher"] == "fp32" else 2)) + 8 * T
        products = 1
        if c["kind"] != "score":
            nbytes += 2 * T * H + 4 * T
            products += 1
        if c["kind"] == "train":
            nbytes += 2 * V * H
            products += 1
        return {"bytes": nbytes, "flops": 2.0 * products * T * H * V}
    if c["op"] == "probs":
        size = {"fp32": 4, "bf16": 2}
        return {"bytes": c["R"] * (c["V"] * (size[c["src"]] + size[c["dst"]]) + 4), "flops": 4.0 * c["R"] * c["V"]}
    B, K, V = c["B"], c["K"], c["V"]
    size = 4 if c["dtype"] == "fp32" else 2
    # one row of the target and, after a rejection, one of the draft; the drafts' own entries; the tokens
    rows = 2 if c["draft"] and K else 1
    return {"bytes": B * (rows * V * size + K * (8 + 4 + rows * size) + 4 + 8 * (K + 2)), "flops": 3.0 * B * V}


# ------------------------------------------------------------------ from the definition, in 64 bits

def _exact_distill(c, s):
    T, H, V, tau = c["T"], c["H"], c["V"], c["tau"]
    W = s["W"].double()
    loss = torch.zeros(T, dtype=_F64, device="cuda")
    lse = torch.zeros(T, dtype=_F64, device="cuda")
    dh = torch.zeros(T, H, dtype=_F64, device="cuda")
    dW = torch.zeros(V, H, dtype=_F64, device="cuda") if c["kind"] == "train" else None
    for t0 in range(0, T, 1024):
        rows = slice(t0, min(T, t0 + 1024))
        h = s["hidden"][rows].double()
        logp = torch.mm(h, W.t()).div_(tau)
        lse[rows] = torch.logsumexp(logp, 1)
        logp -= lse[rows, None]
        ids = s["ids"][rows]
        a = s["logits"][rows].double().div(tau).masked_fill(ids < 0, float("-inf"))
        if s["lse"] is not None:
            logq = a - s["lse"][rows].double()[:, None]
        else:
            logq = torch.log_softmax(a, 1)
        logq = logq.masked_fill(ids < 0, float("-inf"))  # rows without a slot too
        q = logq.exp()
        cross = q * (logq - logp.gather(1, ids.clamp(min=0)))
        loss[rows] = cross.masked_fill(q == 0, 0.0).sum(1)
        if c["kind"] == "score":
            continue
        dense = torch.zeros_like(logp).scatter_add_(1, ids.clamp(min=0), q)
        dx = (logp.exp_() * dense.sum(1, keepdim=True) - dense) * (s["dloss"][rows].double() / tau)[:, None]
        dh[rows] = torch.mm(dx, W)
        if dW is not None:
            dW.addmm_(dx.t(), h)
    if c["kind"] == "score":
        return {"loss": loss, "lse": lse}
    out = {"loss": loss, "dhidden": dh}
    if dW is not None:
        out["dW"] = dW
    return out


def _exact_probs(c, s):
    out = torch.zeros(c["R"], c["V"], dtype=_F64, device="cuda")
    hot = s["t"] > 0
    out[hot] = torch.softmax(s["x"][hot].double() / s["t"][hot].double()[:, None], 1)
    for r in (~hot).nonzero().flatten().tolist():
        out[r, int((s["x"][r] == s["x"][r].max()).nonzero()[0])] = 1.0
    return {"probs": out}


def _exact_verify(c, s):
    B, K, V = c["B"], c["K"], c["V"]
    tokens, accepted = [], []
    for b in range(B):
        length = K if s["lens"] is None else int(s["lens"][b])
        drafts = s["d"][b].tolist()
        n = 0
        while n < length:
            d = drafts[n]
            pd, ua = float(s["p"][b, n, d]), float(s["ua"][b, n])
            qd = 1.0 if s["q"] is None else float(s["q"][b, n, d])
            if not ua * qd < pd:
                break
            n += 1
        r = s["p"][b, n].double()
        if n < length:
            if s["q"] is not None:
                r = torch.relu(r - s["q"][b, n].double())
            else:
                r = r.clone()
                r[drafts[n]] = 0.0
            if float(r.sum()) <= 0.0:
                r = s["p"][b, n].double()
        cum = r.cumsum(0)
        v = int(torch.searchsorted(cum, float(s["us"][b]) * cum[-1:], right=True))
        if v >= V:
            v = int(r.nonzero()[-1])
        tokens.append(drafts[:n] + [v] + [-1] * (K - n))
        accepted.append(n)
    return {"tokens": torch.tensor(tokens, device="cuda"), "accepted": torch.tensor(accepted, device="cuda")}


def exact(case, seed):
    s = prepare(case, seed)
    return {"distill": _exact_distill, "probs": _exact_probs, "verify": _exact_verify}[case["op"]](case, s)
