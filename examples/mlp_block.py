"""A training step of a tensor-parallel MLP block on P logical ranks of one GPU, from 8-bit checkpoints.

    python examples/mlp_block.py

What comes out of the attention block's last matmul goes through

    block_norm       norm of that, residual sum, norm before the MLP, in one pass
    ag_gemm          gathers the token shards and projects to gate and up of every rank
    glu              silu(gate) * up
    gemm_rs          down projection, reduce-scattered by columns
    block_norm       norm of that and the residual sum

and the gradients back, where every operand that the forward pass leaves is kept in 8 bits:

    block_norm_bwd   from the checkpoints of its inputs
    gemm_wgrad       of the down projection, from the checkpoint of silu(gate) * up
    ag_gemm_kn       gradient of its input
    glu_bwd          from the checkpoints of gate and up
    gemm_wgrad       of the up projection, from the checkpoint of the normed shards
    gemm_rs          gradient of its input, which block_norm_bwd reads as it lies

Each result is compared with plain float32 torch: the forward pass as it is, the gradients at
the values that the checkpoints hold.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import ring_collectives_gb300 as rc  # noqa: E402

BF = torch.bfloat16
P, M_R, E, F = 4, 128, 1024, 512                    # ranks, tokens a rank, model width, MLP width a rank
T, EPS, ALPHA = P * M_R, 1e-6, 0.5


def new(*shape, dtype=BF):
    return torch.empty(shape, dtype=dtype, device="cuda")


def held(*shape):
    return rc.act8_empty(shape, "cuda")


def values(x8):
    return rc.act8_unpack(x8, new(*x8[0].shape)).float()


def norm(x, gamma):
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * gamma


def rows(y):
    """[P, T, E / P], column chunks of all tokens, as [P, M_R, E]."""
    return y.transpose(0, 1).reshape(P, M_R, E)


def close(name, got, want, tol=2e-2):
    err = float((got.float() - want.float()).norm() / want.float().norm())
    print(f"{name:44s} relative difference {err:.1e}")
    if not err < tol:
        raise AssertionError(f"{name}: {err} against plain torch")


def main():
    import __graft_entry__
    __graft_entry__.build()
    g = torch.Generator(device="cuda").manual_seed(0)
    rand = lambda *s, std=1.0: torch.randn(*s, generator=g, device="cuda") * std  # noqa: E731
    x, y = rand(P, M_R, E, std=2.0).to(BF), rand(P, T, E // P).to(BF)      # residual shards; a gemm_rs result
    w_up = rand(P * 2 * F, E, std=E ** -0.5).to(BF)                        # gate and up rows of every rank
    w_down = rand(P, E, F, std=(P * F) ** -0.5).to(BF)
    post, post2, pre = (1 + rand(E, std=0.1) for _ in range(3))
    gate = 1 + rand(E, std=0.3)

    # forward, keeping 8 bits of every operand
    h, z = new(P, M_R, E), new(P, M_R, E)
    y8, x8, z8 = (held(P, M_R, E) for _ in range(3))
    rc.block_norm(y, x, h, z, gamma_post=post, gate=gate, gamma_pre=pre, alpha=ALPHA, eps=EPS, y8=y8, res8=x8, z8=z8)
    fused, gathered = new(T, P * 2 * F), new(T, E)
    rc.ag_gemm(z, gathered, w_up, fused, rank=0)
    a, b = fused.view(T, P, 2, F).permute(2, 1, 0, 3)                      # gate and up of every rank, views
    act = new(P, T, F)
    a8, b8, act8 = (held(P, T, F) for _ in range(3))
    rc.glu(a, b, act, a8=a8, b8=b8, h8=act8)
    y2 = new(P, T, E // P)
    rc.gemm_rs(act, w_down, y2)
    out = new(P, M_R, E)
    y28, h8 = held(P, M_R, E), held(P, M_R, E)
    rc.block_norm(y2, h, out, gamma_post=post2, eps=EPS, y8=y28, res8=h8)
    want = x.float() + ALPHA * gate * norm(rows(y).float(), post)
    close("residual sum (block_norm)", h, want)
    close("norm before the MLP", z, norm(want, pre))
    close("gate and up (ag_gemm)", fused, z.view(T, E).float() @ w_up.float().T)
    close("silu(gate) * up (glu)", act, torch.nn.functional.silu(a.float()) * b.float())
    close("down projection (gemm_rs)", rows(y2).view(T, E), torch.einsum("ptf,pef->te", act.float(), w_down.float()))
    close("block's result (block_norm)", out, h.float() + norm(rows(y2).float(), post2))

    # gradients of <out, dout>
    dout = rand(P, M_R, E).to(BF)
    dy2, dh = new(P, M_R, E), new(P, M_R, E)
    dpost2 = new(P, E, dtype=torch.float32)
    rc.block_norm_bwd(y28, h8, dout, None, dy2, dh, dgamma_post=dpost2, gamma_post=post2, eps=EPS)
    dw_down = new(P, E, F, dtype=torch.float32)
    rc.gemm_wgrad(dy2.view(1, T, E).expand(P, -1, -1), act8, dw_down)
    dact_all = new(T, P * F)
    rc.ag_gemm_kn(dy2, gathered, w_down.transpose(0, 1).reshape(E, P * F), dact_all, rank=0)
    dact = dact_all.view(T, P, F).transpose(0, 1)
    dfused = new(P, T, 2 * F)                                              # each rank's gradients, for gemm_rs
    rc.glu_bwd(a8, b8, dact, dfused[..., :F], dfused[..., F:])
    dw_up = new(P, 2 * F, E, dtype=torch.float32)
    rc.gemm_wgrad(dfused, tuple(t.reshape(1, T, -1).expand(P, -1, -1) for t in z8), dw_up)
    dz = new(P, T, E // P)
    rc.gemm_rs(dfused, w_up.view(P, 2 * F, E).transpose(1, 2).contiguous(), dz)
    dy, dx = new(P, T, E // P), new(P, M_R, E)
    dpost, dgate, dpre = (new(P, E, dtype=torch.float32) for _ in range(3))
    rc.block_norm_bwd(y8, x8, dh, dz, dy, dx, dpost, dgate, dpre, gamma_post=post, gate=gate, gamma_pre=pre, alpha=ALPHA, eps=EPS)
    for t in (dpost2, dpost, dgate, dpre):
        rc.ring_allreduce(t)                                               # the ranks' sums of the shared weights

    def grad(name, f, leaves, dout, got):
        """f's gradients at the leaves against what the calls wrote."""
        leaves = [t.detach().requires_grad_() for t in leaves]
        (f(*leaves) * dout.float()).sum().backward()
        for n, leaf, t in zip(name, leaves, got):
            close("gradient of " + n, t, leaf.grad)

    grad(("the MLP's result", "the sum before it", "the norm after it"), lambda u, v, p: v + norm(u, p),
         (values(y28), values(h8), post2), dout, (dy2, dh, dpost2[0]))
    grad(("the down projection",), lambda w: torch.einsum("ptf,pef->te", values(act8), w), (w_down.float(),), dy2.view(T, E), (dw_down,))
    close("gradient of silu(gate) * up", dact, torch.einsum("te,pef->ptf", dy2.view(T, E).float(), w_down.float()))
    grad(("gate", "up"), lambda u, v: torch.nn.functional.silu(u) * v, (values(a8), values(b8)), dact, (dfused[..., :F], dfused[..., F:]))
    grad(("the up projection",), lambda w: torch.einsum("te,pfe->ptf", values(z8).view(T, E), w), (w_up.view(P, 2 * F, E).float(),), dfused, (dw_up,))
    close("gradient of the normed shards", rows(dz).view(T, E), torch.einsum("ptf,pfe->te", dfused.float(), w_up.view(P, 2 * F, E).float()))

    def both(u, v, p, q, r):
        s = v + ALPHA * q * norm(u, p)
        return torch.cat((s, norm(s, r)))

    grad(("the block's input", "the residual", "the norm after", "the gate", "the norm before"), both,
         (values(y8), values(x8), post, gate, pre), torch.cat((dh, rows(dz))), (rows(dy), dx, dpost[0], dgate[0], dpre[0]))
    if rc.ring_status() != 0:
        raise RuntimeError(rc.ring_last_error())


if __name__ == "__main__":
    main()
