"""Cases for the operators that close a tensor-parallel block around the two collective matmuls and
train it from 8-bit activation checkpoints.

* ``act8_pack`` / ``act8_unpack`` -- an activation held in 8 bits: signed bytes with one power of two for
  every 32 channels of a row.
* ``block_norm`` -- between a block's last matmul and the next block's first: norm of the block's output,
  gate and residual scale, the residual sum, and the next block's norm, in one pass that can leave 8-bit
  checkpoints of its inputs; and its gradient, from bf16 operands or from the checkpoints.
* ``glu`` -- the gated activation between the two matmuls of an MLP, with checkpoints; and its gradient.
* ``gemm_wgrad`` -- the weight gradient of either matmul from an activation held in 8 bits.

A case is a dict of plain values.  P logical ranks hold T rows (tokens) of N channels each; with
``cols`` the block's output lies as ``gemm_rs`` leaves it, [P, P * T, N / P], else as [P, T, N].
"""
import math

import torch

own = False

BF16 = torch.bfloat16
EPS = 1e-6
GROUP = 32          # channels of a row that share a power of two


def _case(op, name, **values):
    return dict(values, op=op, **({"name": name} if name else {}))


def listed():
    return [
        # A short tail of a batch, a width that fills neither a vector of 16 nor a group of 32.
        _case("act8", "act8 tail", P=1, T=37, N=1000),
        # The gathered activations of a training batch, 1024 tokens on each of 8 ranks.
        _case("act8", "act8 8k", P=8, T=1024, N=4096),
        # One generation step of 8 sequences: latency is what counts.
        _case("block_norm", "norm 8 tokens", P=8, T=1, N=4096, cols=True, post=True, gate=False, pre=True, save=False),
        # A training batch of 8192 tokens, the checkpoints written along the way.
        _case("block_norm", "norm train 8k", P=8, T=1024, N=4096, cols=True, post=True, gate=True, pre=True, save=True),
        # A short fine-tuning batch of an odd width, everything kept in bf16, no norm after the block.
        _case("block_norm_bwd", "norm grad 777", P=1, T=777, N=1544, cols=False, post=False, gate=True, pre=True, save=False),
        # The gradient of the training batch, from the checkpoints.
        _case("block_norm_bwd", "norm grad 8k", P=8, T=1024, N=4096, cols=True, post=True, gate=True, pre=True, save=True),
        # A generation step of 16 sequences on 8 ranks' shares of an MLP of 14336.
        _case("glu", "glu 16 tokens", P=8, T=16, N=1792, act="silu", save=False),
        # A training batch on 8 ranks.
        _case("glu", "glu train 8k", P=8, T=8192, N=1792, act="silu", save=True),
        # A short batch of an odd length, kept in bf16.
        _case("glu_bwd", "glu grad 1031", P=1, T=1031, N=2752, act="gelu", save=False),
        # The gradient of the training batch, from the checkpoints.
        _case("glu_bwd", "glu grad 8k", P=8, T=8192, N=1792, act="silu", save=True),
        # A projection's weight gradient over a short ragged batch, sizes that fill no tile.
        _case("wgrad", "wgrad 1031", P=1, T=1031, N=520, K=1000, shared=False),
        # The fused Q/K/V weights (4 query, 1 key, 1 value head of 128) of 8 ranks over the gathered batch.
        _case("wgrad", "wgrad 8k", P=8, T=8192, N=768, K=4096, shared=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi, unit=8):
    return unit * max(1, round(_log(rng, lo, hi) / unit))


def draw(rng):
    op = rng.choice(["act8", "block_norm", "block_norm", "block_norm_bwd", "block_norm_bwd", "glu", "glu_bwd", "wgrad", "wgrad"])
    P = rng.choice([1, 2, 4, 8])
    if op == "wgrad":
        N, K = _width(rng, 64, 6000), _width(rng, 64, 6000)
        T = max(1, min(_log(rng, 1, 16384), (150 << 30) // (P * N * K), (100 << 20) // (P * (N + K))))
        return _case(op, "", P=P, T=T, N=N, K=K, shared=rng.random() < 0.5)
    cols = rng.random() < 0.6
    N = min(16384, _width(rng, 64, 16384, 8 * P if cols and op.startswith("block") else 8))
    T = max(1, min(_log(rng, 1, 16384), (30 << 20) // (P * N)))
    if op == "act8":
        return _case(op, "", P=P, T=T, N=N)
    save = rng.random() < 0.5
    if op.startswith("glu"):
        return _case(op, "", P=P, T=T, N=N, act=rng.choice(["silu", "silu", "gelu"]), save=save)
    post, gate = rng.random() < 0.7, rng.random() < 0.5
    return _case(op, "", P=P, T=T, N=N, cols=cols, post=post, gate=gate, pre=rng.random() < 0.85, save=save)


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, shape, scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(BF16)


def _activation(g, shape, scale=1.0):
    """Rows of different sizes, and a few channels far above the others, as in a trained network."""
    x = torch.randn(shape, generator=g, device="cuda")
    x *= scale * torch.exp(0.5 * torch.randn(shape[:-1] + (1,), generator=g, device="cuda"))
    loud = torch.rand(shape[-1], generator=g, device="cuda") < 0.01
    return (x * torch.where(loud, 12.0, 1.0)).to(BF16)


def _weight(g, n):
    return 1 + 0.2 * torch.randn(n, generator=g, device="cuda")


def prepare(case, seed):
    g = _gen(seed)
    op, P, T, N = case["op"], case["P"], case["T"], case["N"]
    s = {"case": case, "op": op}
    if op == "act8":
        s["x"] = _activation(g, (P, T, N))
    elif op.startswith("block_norm"):
        s["res"] = _activation(g, (P, T, N), 2.0)
        s["y"] = _activation(g, (P, P * T, N // P) if case["cols"] else (P, T, N))
        for name, on in (("gamma_post", case["post"]), ("gate", case["gate"]), ("gamma_pre", case["pre"])):
            s[name] = _weight(g, N) if on else None
        s["alpha"] = 0.5
        if op == "block_norm_bwd":
            s["dh"] = _randn(g, (P, T, N), 0.1)
            s["dz"] = _randn(g, (P, T, N), 0.1) if case["pre"] else None
            if case["save"]:
                s["y8"], s["res8"] = _pack(_rows(s["y"], case)), _pack(s["res"])
    elif op.startswith("glu"):
        s["ab"] = _activation(g, (P, T, 2 * N))           # the fused result of the first matmul
        if op == "glu_bwd":
            s["dh"] = _randn(g, (P, T, N), 0.1)
            if case["save"]:
                s["a8"], s["b8"] = _pack(s["ab"][..., :N]), _pack(s["ab"][..., N:])
    else:
        s["dy"] = _randn(g, (P, T, N), 0.1)
        x8 = _pack(_activation(g, (1 if case["shared"] else P, T, case["K"])))
        s["x8"] = tuple(t.expand(P, -1, -1) for t in x8)  # one gathered activation for all ranks, or each its own
    return s


# ---------------------------------------------------------------- plain forms, in 32 bits
def _pack(x):
    """Signed bytes q and biased exponents e of every 32 channels: x is close to q * 2^(e - 127).
    e is the least that keeps |q| <= 127; 255 marks a group with an infinity or a NaN."""
    P, T, N = x.shape
    pad = -N % GROUP
    v = torch.nn.functional.pad(x.float(), (0, pad)).view(P, T, -1, GROUP)
    top = v.abs().amax(-1)
    bad = ~(top < math.inf)
    e = (((top.view(torch.int32) + 0x10000) >> 23) - 6).clamp(1, 248)
    q = (v * ((254 - e) << 23).view(torch.float32)[..., None]).round().clamp(-127, 127)
    q = torch.where(bad[..., None], 0.0, q).view(P, T, N + pad)[..., :N]
    return q.to(torch.int8).contiguous(), torch.where(bad, 255, e).to(torch.uint8)


def _unpack(x8):
    q, e = x8
    scale = (e.int() << 23).view(torch.float32)           # 255: infinity, which makes 0 a NaN
    return q.float() * scale.repeat_interleave(GROUP, -1)[..., :q.shape[-1]]


def _rows(t, case):
    """A block's output or its gradient as [P, T, N]."""
    P, T, N = case["P"], case["T"], case["N"]
    return t.transpose(0, 1).reshape(P, T, N) if case["cols"] else t


def _place(t, case):
    """The inverse of _rows."""
    P, T, N = case["P"], case["T"], case["N"]
    return t.reshape(P * T, P, N // P).transpose(0, 1).contiguous() if case["cols"] else t


def _rms(x):
    return torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)


def _block(s, y, res):
    """The normed output before its weight, its factor, and h."""
    c = s["case"]
    yh = y * _rms(y) if c["post"] else y
    w = s["alpha"] * torch.ones(c["N"], device="cuda")
    for name in ("gamma_post", "gate"):
        if s[name] is not None:
            w = w * s[name]
    return yh, w, res + w * yh


def _plain_block(s):
    c = s["case"]
    h = _block(s, _rows(s["y"], c).float(), s["res"].float())[2]
    out = [h.to(BF16)]
    if c["pre"]:
        out.append((h * _rms(h) * s["gamma_pre"]).to(BF16))
    if c["save"]:
        out += [_unpack(_pack(_rows(s["y"], c))).to(BF16), _unpack(_pack(s["res"])).to(BF16)]
    return tuple(out)


def _plain_block_grad(s):
    c = s["case"]
    y = _unpack(s["y8"]) if c["save"] else _rows(s["y"], c).float()
    res = _unpack(s["res8"]) if c["save"] else s["res"].float()
    yh, w, h = _block(s, y, res)
    d = s["dh"].float()
    grads = {}
    if c["pre"]:
        r = _rms(h)
        hh, t = h * r, s["dz"].float() * s["gamma_pre"]
        grads["gamma_pre"] = (s["dz"].float() * hh).sum(1)
        d = d + r * (t - hh * (t * hh).mean(-1, keepdim=True))
    total = s["alpha"] * (d * yh).sum(1)
    gate, post = s["gate"], s["gamma_post"]
    if post is not None:
        grads["gamma_post"] = total if gate is None else total * gate
    if gate is not None:
        grads["gate"] = total if post is None else total * post
    dy = d * w
    if c["post"]:
        dy = _rms(y) * (dy - yh * (dy * yh).mean(-1, keepdim=True))
    return (_place(dy.to(BF16), c), d.to(BF16), *(grads[n] for n in ("gamma_post", "gate", "gamma_pre") if n in grads))


def _act(a, kind):
    """The activation a * g and its derivative; both kinds are a sigmoid g of their own argument."""
    if kind == "silu":
        x, slope = a, 1.0
    else:                                                 # 0.5 (1 + tanh(x / 2)) = sigmoid(x)
        root = 2 * math.sqrt(2 / math.pi)
        x, slope = root * (a + 0.044715 * a ** 3), root * (1 + 3 * 0.044715 * a * a)
    g = 1 / (1 + torch.exp(-x))
    return a * g, g * (1 + a * slope / (1 + torch.exp(x)))


def _plain_glu(s):
    N = s["case"]["N"]
    a, b = s["ab"][..., :N], s["ab"][..., N:]
    h = (_act(a.float(), s["case"]["act"])[0] * b.float()).to(BF16)
    if not s["case"]["save"]:
        return h
    return h, _unpack(_pack(a)).to(BF16), _unpack(_pack(b)).to(BF16)


def _plain_glu_grad(s):
    c, N = s["case"], s["case"]["N"]
    a, b = (_unpack(s["a8"]), _unpack(s["b8"])) if c["save"] else (s["ab"][..., :N].float(), s["ab"][..., N:].float())
    f, df = _act(a, c["act"])
    dh = s["dh"].float()
    return torch.cat(((dh * b * df).to(BF16), (dh * f).to(BF16)), -1), (f * b).to(BF16)


def _run_plain(s):
    op = s["op"]
    if op == "act8":
        return _unpack(_pack(s["x"])).to(BF16)
    if op == "block_norm":
        return _plain_block(s)
    if op == "block_norm_bwd":
        return _plain_block_grad(s)
    if op == "glu":
        return _plain_glu(s)
    if op == "glu_bwd":
        return _plain_glu_grad(s)
    x8 = tuple(t[:1] for t in s["x8"]) if s["case"]["shared"] else s["x8"]
    return torch.matmul(s["dy"].float().transpose(1, 2), _unpack(x8)).to(BF16)


# ---------------------------------------------------------------- the framework's calls
def _values(rc, x8):
    return rc.act8_unpack(x8, torch.empty(x8[0].shape, dtype=BF16, device="cuda"))


def _run_own(s):
    import ring_collectives_gb300 as rc

    c, op, P, N = s["case"], s["op"], s["case"]["P"], s["case"]["N"]
    if op == "act8":
        return _values(rc, rc.act8_pack(s["x"], rc.act8_empty(s["x"].shape, s["x"].device)))
    if op == "block_norm":
        res = s["res"]
        h, z = torch.empty_like(res), torch.empty_like(res) if c["pre"] else None
        y8, res8 = (rc.act8_empty(res.shape, res.device) if c["save"] else None for _ in range(2))
        rc.block_norm(s["y"], res, h, z, gamma_post=s["gamma_post"], gate=s["gate"], gamma_pre=s["gamma_pre"],
                      alpha=s["alpha"], eps=EPS, y8=y8, res8=res8)
        return (h,) + ((z,) if c["pre"] else ()) + ((_values(rc, y8), _values(rc, res8)) if c["save"] else ())
    if op == "block_norm_bwd":
        dy, dres = torch.empty_like(s["y"]), torch.empty_like(s["res"])
        dw = [None if s[n] is None else torch.empty((P, N), device="cuda") for n in ("gamma_post", "gate", "gamma_pre")]
        rc.block_norm_bwd(s["y8"] if c["save"] else s["y"], s["res8"] if c["save"] else s["res"], s["dh"], s["dz"], dy, dres,
                          *dw, gamma_post=s["gamma_post"], gate=s["gate"], gamma_pre=s["gamma_pre"], alpha=s["alpha"], eps=EPS)
        return (dy, dres, *(t for t in dw if t is not None))
    if op.startswith("glu"):
        ab = s["ab"]
        act = rc.RC_GLU_SILU if c["act"] == "silu" else rc.RC_GLU_GELU
        a, b = ab[..., :N], ab[..., N:]
        h = torch.empty(ab.shape[:2] + (N,), dtype=BF16, device="cuda")
        if op == "glu":
            a8, b8 = (rc.act8_empty(h.shape, h.device) if c["save"] else None for _ in range(2))
            rc.glu(a, b, h, act=act, a8=a8, b8=b8)
            return (h, _values(rc, a8), _values(rc, b8)) if c["save"] else h
        d = torch.empty_like(ab)
        rc.glu_bwd(s["a8"] if c["save"] else a, s["b8"] if c["save"] else b, s["dh"], d[..., :N], d[..., N:], h=h, act=act)
        return d, h
    return rc.gemm_wgrad(s["dy"], s["x8"], torch.empty((P, N, c["K"]), dtype=BF16, device="cuda"))


def run(state):
    return _run_own(state) if own else _run_plain(state)


def work(case):
    op, P, T, N = case["op"], case["P"], case["T"], case["N"]
    n, rows = P * T * N, P * T
    groups = rows * -(-N // GROUP)
    if op == "wgrad":
        K = case["K"]
        x = (1 if case["shared"] else P) * T
        return {"bytes": 2 * n + x * (K + -(-K // GROUP)) + 2 * P * N * K, "flops": 2 * n * K}
    if op == "act8":                                      # read, and the values written
        return {"bytes": 4 * n, "flops": 4 * n}
    if op == "block_norm":
        weights = 4 * N * (case["post"] + case["gate"] + case["pre"])
        return {"bytes": n * (6 + 2 * case["pre"] + 4 * case["save"]) + weights, "flops": 10 * n}
    if op == "block_norm_bwd":
        operands = 2 * (n + groups) if case["save"] else 4 * n
        weights = 4 * N * (1 + P) * (case["post"] + case["gate"] + case["pre"])
        return {"bytes": operands + n * (6 + 2 * case["pre"]) + weights, "flops": 25 * n}
    if op == "glu":
        return {"bytes": n * (6 + 4 * case["save"]), "flops": 12 * n}
    return {"bytes": (2 * (n + groups) if case["save"] else 4 * n) + 8 * n, "flops": 20 * n}


# ---------------------------------------------------------------- the definitions, in 64 bits
def _nearest(x):
    """What 8 bits make of a bf16 activation: multiples of the least 2^k, -126 <= k <= 121, with no
    element of the 32 above 127 of them."""
    v = x.double()
    out = torch.empty_like(v)
    for i in range(0, v.shape[-1], GROUP):
        part = v[..., i:i + GROUP]
        m, k = torch.frexp(part.abs().max(-1, keepdim=True).values / 127)
        k = torch.where(m == 0.5, k - 1, k).clamp(-126, 121).double()
        out[..., i:i + GROUP] = torch.round(part * 2.0 ** -k).clamp(-127, 127) * 2.0 ** k
    return out


def _held(x8):
    q, e = x8
    k = torch.arange(q.shape[-1], device="cuda") // GROUP
    return q.double() * 2.0 ** (e.double() - 127)[..., k]


def _full(t, case):
    return torch.cat(tuple(t), -1).unflatten(0, (case["P"], case["T"])) if case["cols"] else t


def exact(case, seed):
    s = prepare(case, seed)
    F, op, P, N = torch.float64, case["op"], case["P"], case["N"]
    if op == "act8":
        return _nearest(s["x"])
    if op == "wgrad":
        x = _held(tuple(t[:1] if case["shared"] else t for t in s["x8"]))
        return torch.stack([s["dy"][r].to(F).T @ x[0 if case["shared"] else r] for r in range(P)])
    if op.startswith("glu"):
        a, b = s["ab"][..., :N], s["ab"][..., N:]
        kept = case["save"] and op == "glu_bwd"
        u, v = (_held(s["a8"]), _held(s["b8"])) if kept else (a.to(F), b.to(F))
        if case["act"] == "silu":
            f = u * torch.sigmoid(u)
            df = torch.sigmoid(u) + f * torch.sigmoid(-u)
        else:                                             # (1 + tanh x) / 2 = sigmoid(2 x)
            x2 = math.sqrt(8 / math.pi) * (u + 0.044715 * u.pow(3))
            f = u * torch.sigmoid(x2)
            df = torch.sigmoid(x2) + f * torch.sigmoid(-x2) * math.sqrt(8 / math.pi) * (1 + 0.134145 * u.pow(2))
        if op == "glu":
            return (f * v, _nearest(a), _nearest(b)) if case["save"] else f * v
        dh = s["dh"].to(F)
        return torch.cat((dh * v * df, dh * f), -1), f * v
    grad = op == "block_norm_bwd"
    kept = case["save"] and grad
    y = _held(s["y8"]) if kept else _full(s["y"], case).to(F)
    res = _held(s["res8"]) if kept else s["res"].to(F)
    one = torch.ones(N, dtype=F, device="cuda")
    post, gate, pre = (one if s[n] is None else s[n].to(F) for n in ("gamma_post", "gate", "gamma_pre"))
    size_y = ((y ** 2).sum(-1, keepdim=True) / N + EPS).sqrt() if case["post"] else torch.ones_like(y[..., :1])
    h = res + s["alpha"] * gate * post * y / size_y
    size_h = ((h ** 2).sum(-1, keepdim=True) / N + EPS).sqrt()
    if not grad:
        out = (h,) + ((h / size_h * pre,) if case["pre"] else ())
        return out + ((_nearest(_full(s["y"], case)), _nearest(s["res"])) if case["save"] else ())
    d = s["dh"].to(F)
    sums = []
    if case["pre"]:
        dz = s["dz"].to(F)
        sums.append((dz * h / size_h).sum(1))
        d = d + dz * pre / size_h - h * (dz * pre * h).sum(-1, keepdim=True) / (N * size_h ** 3)
    du = s["alpha"] * d
    if case["gate"]:
        sums.insert(0, (du * post * y / size_y).sum(1))
    if case["post"]:
        sums.insert(0, (du * gate * y / size_y).sum(1))
    t = du * gate * post
    dy = t / size_y
    if case["post"]:
        dy = dy - y * (t * y).sum(-1, keepdim=True) / (N * size_y ** 3)
    if case["cols"]:
        dy = torch.stack(dy.flatten(0, 1).chunk(P, -1))
    return (dy, d, *sums)
