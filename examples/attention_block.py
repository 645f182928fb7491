"""A tensor-parallel attention block on P logical ranks of one GPU, end to end.

    python examples/attention_block.py

Sequence-sharded activations go through the two collective matmuls with
attention between them, everything on the library's kernels:

    ag_gemm          gathers the token shards and projects to fused Q/K/V
    qk_norm_rope     RMS norm of every query and key head + rotation
    attn_fwd         causal attention over packed sequences, grouped heads
    gemm_rs          output projection, reduce-scattered by columns

then one generated token a sequence against the key/value cache the prompt
left, and the gradients back to the fused activations and the norm weights
(summed over the ranks by ring_allreduce).  Each stage is compared with plain
float32 torch on the same inputs.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import ring_collectives_gb300 as rc  # noqa: E402

BF = torch.bfloat16
P, M_R, E, HQ, HKV, D = 4, 128, 1024, 2, 1, 64      # per rank: 2 query heads on 1 key head
LENS = [300, 1, 150, 61]                            # packed prompts: P * M_R tokens in all
CAP = 384                                           # cache rows of a sequence


def heads(fused):
    """[T, P * (Hq + 2 Hkv) * D] -> per-rank query, key and value heads [P, T, H, D], views."""
    h = fused.view(fused.shape[0], P, HQ + 2 * HKV, D).transpose(0, 1)
    return h[:, :, :HQ], h[:, :, HQ:HQ + HKV], h[:, :, HQ + HKV:]


def tables(n):
    angle = torch.arange(n, device="cuda")[:, None] * 10000.0 ** (-torch.arange(0, D, 2, device="cuda") / D)
    return angle.cos(), angle.sin()


def plain_norm(x, gamma, cos, sin, pos):
    x = x.float()
    y = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * gamma
    c, s = cos[pos.long()][:, None], sin[pos.long()][:, None]
    a, b = y.chunk(2, -1)
    return torch.cat((a * c - b * s, a * s + b * c), -1)


def plain_attention(q, k, v, lens_q, lens_k):
    """float32, one sequence after another: q [P, T, Hq, D], k, v [P, T, Hkv, D]."""
    outs, i, j = [], 0, 0
    for n, m in zip(lens_q, lens_k):
        kk, vv = (x[:, j:j + m].float().repeat_interleave(HQ // HKV, 2) for x in (k, v))
        s = torch.einsum("pthd,pshd->phts", q[:, i:i + n].float(), kk) * D ** -0.5
        hide = torch.arange(m, device="cuda")[None] > torch.arange(n, device="cuda")[:, None] + m - n
        outs.append(torch.einsum("phts,pshd->pthd", s.masked_fill(hide, float("-inf")).softmax(-1), vv))
        i, j = i + n, j + m
    return torch.cat(outs, 1)


def close(name, got, want, tol=2e-2):
    err = float((got.float() - want.float()).norm() / want.float().norm())
    print(f"{name:34s} relative difference {err:.1e}")
    if not err < tol:
        raise AssertionError(f"{name}: {err} against plain torch")


def project(x, w_qkv):
    fused = torch.empty((P * x.shape[1], w_qkv.shape[0]), dtype=BF, device="cuda")
    gathered = torch.empty((P * x.shape[1], E), dtype=BF, device="cuda")
    rc.ag_gemm(x, gathered, w_qkv, fused, rank=0)
    return fused


def main():
    import __graft_entry__
    __graft_entry__.build()
    g = torch.Generator(device="cuda").manual_seed(0)
    rand = lambda *s, std=1.0: torch.randn(*s, generator=g, device="cuda") * std  # noqa: E731
    T, B = P * M_R, len(LENS)
    assert sum(LENS) == T
    x = rand(P, M_R, E).to(BF)                                       # each rank's tokens
    w_qkv = rand(P * (HQ + 2 * HKV) * D, E, std=E ** -0.5).to(BF)
    w_out = rand(P, E, HQ * D, std=(P * HQ * D) ** -0.5).to(BF)      # each rank's rows of the output weight
    gamma_q, gamma_k = 1 + rand(D, std=0.1), 1 + rand(D, std=0.1)
    cos, sin = tables(CAP)
    starts = [sum(LENS[:b]) for b in range(B + 1)]
    cu = torch.tensor(starts, dtype=torch.int32, device="cuda")
    pos = torch.cat([torch.arange(n, dtype=torch.int32, device="cuda") for n in LENS])

    # the prompt
    fused = project(x, w_qkv)
    q, k, v = heads(fused)
    qn, kn = torch.empty((P, T, HQ, D), dtype=BF, device="cuda"), torch.empty((P, T, HKV, D), dtype=BF, device="cuda")
    rc.qk_norm_rope(q, k, gamma_q, gamma_k, cos, sin, pos, qn, kn)
    out, lse = torch.empty_like(qn), torch.empty((P, T, HQ), device="cuda")
    rc.attn_fwd(qn, kn, v, out, lse, cu, cu)
    y = torch.empty((P, T, E // P), dtype=BF, device="cuda")
    rc.gemm_rs(out.view(P, T, HQ * D), w_out, y)
    close("Q/K/V projection (ag_gemm)", fused, x.view(T, E).float() @ w_qkv.float().T)
    close("query norm + rotation", qn, plain_norm(q, gamma_q, cos, sin, pos))
    close("key norm + rotation", kn, plain_norm(k, gamma_k, cos, sin, pos))
    close("prompt attention", out, plain_attention(qn, kn, v, LENS, LENS))
    want = torch.einsum("ptk,pek->te", out.view(P, T, HQ * D).float(), w_out.float())
    close("output projection (gemm_rs)", y.transpose(0, 1).reshape(T, E), want)

    # one more token for every sequence, against a cache of CAP rows each
    ck, cv = (torch.zeros((P, B * CAP, HKV, D), dtype=BF, device="cuda") for _ in range(2))
    for b, n in enumerate(LENS):
        ck[:, b * CAP:b * CAP + n] = kn[:, starts[b]:starts[b] + n]
        cv[:, b * CAP:b * CAP + n] = v[:, starts[b]:starts[b] + n]
    token = torch.zeros((P, M_R, E), dtype=BF, device="cuda")        # the projection takes whole tiles of tokens
    token[0, :B] = rand(B, E).to(BF)
    q1, k1, v1 = (h[:, :B] for h in heads(project(token, w_qkv)))
    used = torch.tensor(LENS, dtype=torch.int32, device="cuda")
    rc.qk_norm_rope(q1, k1, gamma_q, gamma_k, cos, sin, used, q1, k1)   # in place: the new token's position is n
    rows = torch.arange(B, device="cuda") * CAP + used
    ck[:, rows], cv[:, rows] = k1, v1
    o1 = torch.empty((P, B, HQ, D), dtype=BF, device="cuda")
    cache = torch.arange(0, B * CAP + 1, CAP, dtype=torch.int32, device="cuda")
    rc.attn_fwd(q1, ck, cv, o1, None, torch.arange(B + 1, dtype=torch.int32, device="cuda"), cache, used_k=used + 1)
    full = [torch.cat([c[:, b * CAP:b * CAP + n + 1] for b, n in enumerate(LENS)], 1) for c in (ck, cv)]
    close("one token against the cache", o1, plain_attention(q1, *full, [1] * B, [n + 1 for n in LENS]))

    # gradients of sum(out * dout), into one fused buffer
    dout = rand(P, T, HQ, D).to(BF)
    dfused = torch.empty_like(fused)
    dq, dk, dv = heads(dfused)
    rc.attn_bwd(qn, kn, v, out, lse, dout, dq, dk, dv, cu, cu)
    dgq, dgk = torch.empty((P, D), device="cuda"), torch.empty((P, D), device="cuda")
    rc.qk_norm_rope_bwd(q, k, gamma_q, gamma_k, cos, sin, pos, dq, dk, dq, dk, dgq, dgk)
    rc.ring_allreduce(dgq)
    rc.ring_allreduce(dgk)
    leaf, lq, lk = fused.float().requires_grad_(), gamma_q.clone().requires_grad_(), gamma_k.clone().requires_grad_()
    a, b, c = heads(leaf)
    plain = plain_attention(plain_norm(a, lq, cos, sin, pos), plain_norm(b, lk, cos, sin, pos), c, LENS, LENS)
    (plain * dout.float()).sum().backward()
    close("gradient of the fused Q/K/V", dfused, leaf.grad)
    close("gradient of the query norm weight", dgq[P - 1], lq.grad)
    close("gradient of the key norm weight", dgk[0], lk.grad)
    if rc.ring_status() != 0:
        raise RuntimeError(rc.ring_last_error())


if __name__ == "__main__":
    main()
