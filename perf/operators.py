"""Cases for the attention operators that sit between the two collective matmuls.

In a tensor-parallel transformer block ``ag_gemm`` produces the fused Q/K/V
activations of P logical ranks and ``gemm_rs`` consumes the attention output.
Between them run

* ``qk_norm_rope`` -- RMS norm of every query and key head with the rotary
  position rotation in the same pass -- and its gradient, and
* ``attn_fwd`` / ``attn_bwd`` -- attention over packed sequences with grouped
  heads, over a whole prompt, a later piece of one, or one token against a
  cache -- and its gradient.

A case is a dict of plain values.  Head counts are per rank.  ``q_lens`` and
``k_lens`` are comma-separated sequence lengths; ``cap`` is 0 for packed keys
or the rows of each sequence in a key/value cache.
"""
import math

import torch

own = False

BF16 = torch.bfloat16
ROPE_BASE = 10000.0
EPS = 1e-6


def _ints(text):
    return list(map(int, text.split(",")))


def _text(lens):
    return ",".join(map(str, lens))


def _attn(op, name, P, Hq, Hkv, D, q, k=None, cap=0, causal=True):
    c = {"op": op, "P": P, "Hq": Hq, "Hkv": Hkv, "D": D, "causal": causal, "q_lens": _text(q),
         "k_lens": _text(q if k is None else k), "cap": cap}
    return dict(c, name=name) if name else c


def _norm(op, name, P, Hq, Hkv, D, T, pairs):
    c = {"op": op, "P": P, "Hq": Hq, "Hkv": Hkv, "D": D, "T": T, "pairs": pairs}
    return dict(c, name=name) if name else c


def listed():
    return [
        # A handful of short prompts, one of a single token: latency is what counts.
        _attn("attn_fwd", "prompt short d64", 1, 8, 8, 64, [1, 17, 130, 64, 200, 5]),
        # A serving batch of prompts of very different lengths packed without padding.
        _attn("attn_fwd", "prompt ragged", 1, 32, 8, 128, [4097, 2500, 1, 777, 3333, 319]),
        # One long prompt on the 8 ranks of a 4096-wide model (32 query heads, 8 key heads).
        _attn("attn_fwd", "prompt 16k", 8, 4, 1, 128, [16384]),
        # The next pieces of two prompts whose earlier tokens are in the key/value cache.
        _attn("attn_fwd", "prompt pieces", 1, 16, 4, 96, [512, 301], [8192, 5003], 8192),
        # One user generating after a long prompt.
        _attn("attn_fwd", "token 1x32k", 8, 4, 1, 128, [1], [32768], 32768),
        # A full generation batch, every sequence at another length.
        _attn("attn_fwd", "token 64 ragged", 1, 32, 8, 128, [1] * 64, [200 + (i * 2917) % 7900 for i in range(64)], 8192),
        # Fine-tuning on short ragged samples.
        _attn("attn_bwd", "train short d64", 1, 12, 12, 64, [1, 100, 33, 257, 512, 391]),
        # A training sequence on 8 ranks.
        _attn("attn_bwd", "train 8k", 8, 4, 1, 128, [8192]),
        # The tokens of one generation step.
        _norm("norm_rope", "norm 64 tokens", 8, 4, 1, 128, 64, False),
        # A packed prompt batch, an odd number of tokens.
        _norm("norm_rope", "norm 16k", 8, 4, 1, 128, 16383, False),
        # A small training batch with adjacent-pair rotation.
        _norm("norm_rope_bwd", "norm grad d64", 1, 12, 12, 64, 1294, True),
        # A training batch on 8 ranks.
        _norm("norm_rope_bwd", "norm grad 8k", 8, 4, 1, 128, 8192, False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _split(rng, total, most):
    """`total` tokens as one to 8 lengths of at most `most`, one of them often a single token."""
    n = rng.randint(1, 8)
    w = [rng.uniform(0.05, 1.0) for _ in range(n)]
    lens = [max(1, min(most, int(total * x / sum(w)))) for x in w]
    return lens + [1] if rng.random() < 0.4 else lens


def _heads(rng):
    Hkv = rng.choice([1, 2, 4, 8])
    G = rng.choice([1, 2, 3, 4, 6, 8])
    P = rng.choice([1, 2, 4, 8])
    while P * Hkv * G > 48:
        P, Hkv = (P // 2, Hkv) if P > 1 else (P, Hkv // 2)
    return P, Hkv * G, Hkv


def _fit(lens, heads, most):
    """Shortens the lengths until heads x sequences x longest^2 is at most `most`."""
    while heads * len(lens) * max(lens) ** 2 > most:
        lens = [max(1, (3 * x) // 4) for x in lens]
    return lens


def draw(rng):
    op = rng.choice(["prompt", "prompt", "piece", "token", "token", "train", "train", "norm_rope", "norm_rope_bwd"])
    P, Hq, Hkv = _heads(rng)
    D = rng.choice([64, 80, 96, 128, 128])
    if op in ("prompt", "train"):
        q = _split(rng, _log(rng, 100, 16384 if op == "prompt" else 8192), 16384)
        q = _fit(q, P * Hq, (8 if op == "prompt" else 2) << 30)
        return _attn("attn_fwd" if op == "prompt" else "attn_bwd", "", P, Hq, Hkv, D, q, causal=rng.random() < 0.8)
    if op == "piece":
        q = [_log(rng, 2, 700) for _ in range(rng.randint(1, 4))]
        k = [x + _log(rng, 10, 8000) for x in q]
        return _attn("attn_fwd", "", P, Hq, Hkv, D, q, k, max(k) + rng.randint(0, 100))
    if op == "token":
        k = [_log(rng, 16, 16384) for _ in range(_log(rng, 1, 96))]
        k = _fit([min(x, 8192) for x in k] if len(k) > 16 else k, 1, 4 << 30)
        return _attn("attn_fwd", "", P, Hq, Hkv, D, [1] * len(k), k, max(k) + rng.randint(0, 100))
    return _norm(op, "", P, Hq, Hkv, D, _log(rng, 8, 16384 if op == "norm_rope" else 8192), rng.random() < 0.4)


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, shape, scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(BF16)


def _fused(x, P, Hq, Hkv, D):
    """Per-rank query, key and value heads [P, T, H, D] inside the fused activations
    [T, P * (Hq + 2 Hkv) * D] that the projection writes."""
    T = x.shape[0]
    h = x.view(T, P, Hq + 2 * Hkv, D).transpose(0, 1)
    return h[:, :, :Hq], h[:, :, Hq:Hq + Hkv], h[:, :, Hq + Hkv:]


def _starts(lens):
    out = [0]
    for n in lens:
        out.append(out[-1] + n)
    return out


def prepare(case, seed):
    g = _gen(seed)
    P, Hq, Hkv, D = case["P"], case["Hq"], case["Hkv"], case["D"]
    s = {"case": case, "op": case["op"]}
    if case["op"].startswith("norm"):
        T = case["T"]
        q, k, _ = _fused(_randn(g, (T, P * (Hq + 2 * Hkv) * D), 1.5), P, Hq, Hkv, D)
        npos = 2 * T + 7
        angle = torch.arange(npos, device="cuda", dtype=torch.float64)[:, None] * ROPE_BASE ** (
            -torch.arange(0, D, 2, device="cuda", dtype=torch.float64) / D)
        s |= {"q": q, "k": k, "cos": angle.cos().float(), "sin": angle.sin().float(),
              "pos": torch.randint(0, npos, (T,), generator=g, device="cuda", dtype=torch.int32),
              "gq": 1 + 0.2 * torch.randn(D, generator=g, device="cuda"),
              "gk": 1 + 0.2 * torch.randn(D, generator=g, device="cuda")}
        if case["op"] == "norm_rope_bwd":
            s |= {"dqo": _randn(g, (P, T, Hq, D)), "dko": _randn(g, (P, T, Hkv, D))}
        return s
    ql, kl, cap = _ints(case["q_lens"]), _ints(case["k_lens"]), case["cap"]
    Tq = sum(ql)
    Tk = cap * len(kl) if cap else sum(kl)
    s |= {"ql": ql, "kl": kl, "q": _randn(g, (P, Tq, Hq, D))}
    if cap:  # a key/value cache: `cap` rows for each sequence, the first k_lens of them in use
        s |= {"k": _randn(g, (P, Tk, Hkv, D)), "v": _randn(g, (P, Tk, Hkv, D))}
        s["used_k"] = torch.tensor(kl, dtype=torch.int32, device="cuda")
        s["cu_k"] = torch.tensor([cap * i for i in range(len(kl) + 1)], dtype=torch.int32, device="cuda")
    else:  # keys as qk_norm_rope leaves them, values still inside the fused activations
        s |= {"k": _randn(g, (P, Tk, Hkv, D)), "v": _fused(_randn(g, (Tk, P * (Hq + 2 * Hkv) * D)), P, Hq, Hkv, D)[2]}
        s["used_k"] = None
        s["cu_k"] = torch.tensor(_starts(kl), dtype=torch.int32, device="cuda")
    s["cu_q"] = torch.tensor(_starts(ql), dtype=torch.int32, device="cuda")
    if case["op"] == "attn_bwd":
        out, lse = _plain_attn(s)
        s |= {"out": out, "lse": lse, "dout": _randn(g, (P, Tq, Hq, D))}
    return s


# ---------------------------------------------------------------- plain forms, in 32 bits
def _pad_index(cu, used, most):
    """Rows [B, most] of each sequence's tokens (clipped to it) and which of them exist."""
    start = cu[:-1].long()
    n = (cu[1:] - cu[:-1] if used is None else used).long()
    i = torch.arange(most, device="cuda")
    return start[:, None] + torch.minimum(i[None], (n[:, None] - 1).clamp(min=0)), i[None] < n[:, None], n


def _padded(x, idx, Hkv):
    """[P, T, H, D] -> float32 [P, B, Hkv, (H / Hkv) * L, D]."""
    P, _, H, D = x.shape
    B, L = idx.shape
    y = x[:, idx].float().view(P, B, L, Hkv, H // Hkv, D)
    return y.permute(0, 1, 3, 4, 2, 5).reshape(P, B, Hkv, (H // Hkv) * L, D)


def _packed(y, s, lens, L, cu):
    """The inverse of _padded for packed tokens: [P, B, Hkv, G * L, D] -> [P, T, Hkv * G, D]."""
    P, B, Hkv, GL, D = y.shape
    T = sum(lens)
    seq = torch.repeat_interleave(torch.arange(B, device="cuda"), (cu[1:] - cu[:-1]).long(), output_size=T)
    at = torch.arange(T, device="cuda") - cu[:-1].long()[seq]
    y = y.view(P, B, Hkv, GL // L, L, D).permute(0, 1, 4, 2, 3, 5)
    return y[:, seq, at].reshape(P, T, Hkv * (GL // L), D)


def _scores(s):
    c = s["case"]
    Lq, Lk = max(s["ql"]), max(s["kl"])
    qi, _, nq = _pad_index(s["cu_q"], None, Lq)
    ki, kok, nk = _pad_index(s["cu_k"], s["used_k"], Lk)
    q, k, v = _padded(s["q"], qi, c["Hkv"]), _padded(s["k"], ki, c["Hkv"]), _padded(s["v"], ki, c["Hkv"])
    see = kok[:, None, :]
    if c["causal"]:
        last = torch.arange(Lq, device="cuda")[None, :, None] + (nk - nq)[:, None, None]
        see = see & (torch.arange(Lk, device="cuda")[None, None, :] <= last)
    x = torch.matmul(q * c["D"] ** -0.5, k.transpose(-1, -2))
    B, G = len(s["ql"]), c["Hq"] // c["Hkv"]
    x.view(c["P"], B, c["Hkv"], G, Lq, Lk).masked_fill_(~see[None, :, None, None], -math.inf)
    return x, q, k, v, qi


def _plain_attn(s):
    x, _, _, v, _ = _scores(s)
    m = x.amax(-1, keepdim=True)
    p = x.sub_(m.masked_fill(m == -math.inf, 0.0)).exp_()
    n = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v) / n.masked_fill(n == 0, 1.0)
    lse = m + n.log()
    L = max(s["ql"])
    return (_packed(o, s, s["ql"], L, s["cu_q"]).to(BF16), _packed(lse, s, s["ql"], L, s["cu_q"])[..., 0].contiguous())


def _plain_attn_grad(s):
    c = s["case"]
    x, q, k, v, qi = _scores(s)
    Lq, Lk, G = max(s["ql"]), max(s["kl"]), c["Hq"] // c["Hkv"]
    ok = torch.arange(Lq, device="cuda")[None] < (s["cu_q"][1:] - s["cu_q"][:-1])[:, None]
    lse = _padded(s["lse"][..., None], qi, c["Hkv"])
    p = x.sub_(lse.masked_fill(lse == -math.inf, math.inf)).exp_()
    P, B = c["P"], len(s["ql"])
    p.view(P, B, c["Hkv"], G, Lq, Lk).mul_(ok[None, :, None, None, :, None])
    do, o = _padded(s["dout"], qi, c["Hkv"]), _padded(s["out"], qi, c["Hkv"])
    dv = torch.matmul(p.transpose(-1, -2), do)
    ds = torch.matmul(do, v.transpose(-1, -2)).sub_((do * o).sum(-1, keepdim=True)).mul_(p)
    dq = torch.matmul(ds, k) * c["D"] ** -0.5
    dk = torch.matmul(ds.transpose(-1, -2), q * c["D"] ** -0.5)
    return (_packed(dq, s, s["ql"], Lq, s["cu_q"]).to(BF16), _packed(dk, s, s["kl"], Lk, s["cu_k"]).to(BF16),
            _packed(dv, s, s["kl"], Lk, s["cu_k"]).to(BF16))


def _rotate(y, cos, sin, pairs):
    """The rotation by the angles of cos and sin, [T, 1, D/2] each; with -sin its inverse."""
    h = y.shape[-1] // 2
    a, b = (y[..., 0::2], y[..., 1::2]) if pairs else (y[..., :h], y[..., h:])
    u, w = a * cos - b * sin, a * sin + b * cos
    return torch.stack((u, w), -1).flatten(-2) if pairs else torch.cat((u, w), -1)


def _tables(s):
    at = s["pos"].long()
    return s["cos"][at][:, None], s["sin"][at][:, None]


def _plain_norm(x, gamma, s):
    cos, sin = _tables(s)
    x = x.float()
    y = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * gamma
    return _rotate(y, cos, sin, s["case"]["pairs"]).to(BF16)


def _plain_norm_grad(x, gamma, dz, s):
    cos, sin = _tables(s)
    dy = _rotate(dz.float(), cos, -sin, s["case"]["pairs"])
    x = x.float()
    r = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
    xh, t = x * r, dy * gamma
    return ((t - xh * (t * xh).mean(-1, keepdim=True)) * r).to(BF16), (dy * xh).sum((1, 2))


# ---------------------------------------------------------------- one pass
def _run_plain(s):
    if s["op"] == "attn_fwd":
        return _plain_attn(s)
    if s["op"] == "attn_bwd":
        return _plain_attn_grad(s)
    if s["op"] == "norm_rope":
        return _plain_norm(s["q"], s["gq"], s), _plain_norm(s["k"], s["gk"], s)
    dq, dgq = _plain_norm_grad(s["q"], s["gq"], s["dqo"], s)
    dk, dgk = _plain_norm_grad(s["k"], s["gk"], s["dko"], s)
    return dq, dk, dgq, dgk


def _run_own(s):
    import ring_collectives_gb300 as rc

    c = s["case"]
    q, k = s["q"], s["k"]
    new = torch.empty
    if s["op"] == "attn_fwd":
        out = torch.empty_like(q)
        lse = new(q.shape[:3], dtype=torch.float32, device="cuda")
        rc.attn_fwd(q, k, s["v"], out, lse, s["cu_q"], s["cu_k"], used_k=s["used_k"], causal=c["causal"])
        return out, lse
    if s["op"] == "attn_bwd":
        dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(k)
        rc.attn_bwd(q, k, s["v"], s["out"], s["lse"], s["dout"], dq, dk, dv, s["cu_q"], s["cu_k"],
                    used_k=s["used_k"], causal=c["causal"])
        return dq, dk, dv
    layout = rc.RC_ROPE_PAIRS if c["pairs"] else rc.RC_ROPE_HALF
    qo, ko = new(q.shape, dtype=BF16, device="cuda"), new(k.shape, dtype=BF16, device="cuda")
    if s["op"] == "norm_rope":
        rc.qk_norm_rope(q, k, s["gq"], s["gk"], s["cos"], s["sin"], s["pos"], qo, ko, layout=layout, eps=EPS)
        return qo, ko
    dgq = new((c["P"], c["D"]), dtype=torch.float32, device="cuda")
    dgk = torch.empty_like(dgq)
    rc.qk_norm_rope_bwd(q, k, s["gq"], s["gk"], s["cos"], s["sin"], s["pos"], s["dqo"], s["dko"], qo, ko, dgq, dgk,
                        layout=layout, eps=EPS)
    return qo, ko, dgq, dgk


def run(state):
    return _run_own(state) if own else _run_plain(state)


def _visible(case):
    """Query-key pairs that the mask leaves, for one head."""
    n = 0
    for a, b in zip(_ints(case["q_lens"]), _ints(case["k_lens"])):
        n += a * b if not case["causal"] else sum(max(0, min(b, i + 1 + b - a)) for i in range(a))
    return n


def work(case):
    P, Hq, Hkv, D = case["P"], case["Hq"], case["Hkv"], case["D"]
    if case["op"].startswith("norm"):
        T = case["T"]
        rows = P * T * (Hq + Hkv)
        grad = case["op"] == "norm_rope_bwd"
        small = T * 4 + T * D * 4 + 2 * D * 4  # positions, one row of cos and sin for each token, the weights
        return {"bytes": rows * D * 2 * (3 if grad else 2) + small + (P * 2 * D * 4 if grad else 0),
                "flops": rows * D * (14 if grad else 7)}
    Tq, Tk = sum(_ints(case["q_lens"])), sum(_ints(case["k_lens"]))
    qb, kb, pairs = P * Tq * Hq * D * 2, P * Tk * Hkv * D * 2, _visible(case) * P * Hq
    if case["op"] == "attn_fwd":
        return {"bytes": 2 * qb + 2 * kb + P * Tq * Hq * 4, "flops": 4 * D * pairs}
    return {"bytes": 4 * qb + 4 * kb + P * Tq * Hq * 4, "flops": 10 * D * pairs}


# ---------------------------------------------------------------- the definitions, in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    P, Hq, Hkv, D = case["P"], case["Hq"], case["Hkv"], case["D"]
    F = torch.float64
    if case["op"].startswith("norm"):
        h = D // 2
        first = torch.arange(h, device="cuda") * (2 if case["pairs"] else 1)
        second = first + (1 if case["pairs"] else h)
        c, w = (s[n].to(F)[s["pos"].long()].unsqueeze(1) for n in ("cos", "sin"))
        res, grads = [], []
        for x, gamma, dz in ((s["q"], s["gq"], s.get("dqo")), (s["k"], s["gk"], s.get("dko"))):
            x, gamma = x.to(F), gamma.to(F)
            norm = ((x ** 2).sum(-1, keepdim=True) / D + EPS).sqrt()
            unit = x / norm
            z = torch.empty(x.shape, dtype=F, device="cuda")
            if dz is None:
                y = unit * gamma
                z[..., first] = y[..., first] * c - y[..., second] * w
                z[..., second] = y[..., second] * c + y[..., first] * w
                res.append(z)
            else:
                dz = dz.to(F)
                z[..., first] = dz[..., first] * c + dz[..., second] * w
                z[..., second] = dz[..., second] * c - dz[..., first] * w
                grads.append((z * unit).sum(dim=(1, 2)))
                du = z * gamma
                res.append(du / norm - x * (du * x).sum(-1, keepdim=True) / (D * norm ** 3))
        return tuple(res + grads)
    ql, kl, cap = s["ql"], s["kl"], case["cap"]
    grad, G, scale = case["op"] == "attn_bwd", Hq // Hkv, 1.0 / math.sqrt(D)
    outs = [torch.zeros(s["q"].shape, dtype=F, device="cuda")]
    if grad:
        outs += [torch.zeros(s["k"].shape, dtype=F, device="cuda") for _ in range(2)]
    else:
        outs.append(torch.full(s["q"].shape[:3], -math.inf, dtype=F, device="cuda"))
    q0 = k0 = 0
    for a, b in zip(ql, kl):
        for r in range(P):
            for h in range(Hq):
                k, v = (s[n][r, k0:k0 + b, h // G].to(F) for n in ("k", "v"))
                for i in range(0, a, 2048):
                    n = min(2048, a - i)
                    here = slice(q0 + i, q0 + i + n)
                    seen = max(0, min(b, i + n + b - a)) if case["causal"] else b
                    if not seen:
                        continue
                    x = (s["q"][r, here, h].to(F) @ k[:seen].T) * scale
                    if case["causal"]:
                        far = torch.arange(seen, device="cuda")[None] > torch.arange(i, i + n, device="cuda")[:, None] + (b - a)
                        x[far] = -math.inf
                    lse = torch.logsumexp(x, 1)
                    p = torch.nan_to_num(torch.exp(x - lse[:, None]), nan=0.0)
                    if not grad:
                        outs[0][r, here, h], outs[1][r, here, h] = p @ v[:seen], lse
                        continue
                    do = s["dout"][r, here, h].to(F)
                    dp = do @ v[:seen].T
                    ds = p * (dp - (p * dp).sum(1, keepdim=True)) * scale
                    outs[0][r, here, h] = ds @ k[:seen]
                    outs[1][r, k0:k0 + seen, h // G] += ds.T @ s["q"][r, here, h].to(F)
                    outs[2][r, k0:k0 + seen, h // G] += p.T @ do
        q0, k0 = q0 + a, k0 + (cap or b)
    return tuple(outs)
