"""How far a gradient of attention, computed from the forward pass's own results, may be from
the derivative of the definition (plain numpy, 64 bits; used by the CPU and the GPU test).

The bounds of oracle.attention.attn_bwd hold for the log-sums and outputs that are given.  Those
are themselves off, by lb and ob: an error of the log-sum moves every weight of its row by the
same share, one of the output moves delta_i = dO_i . O_i by at most sum_c ob_ic |dO_ic|.
"""
import numpy as np

from oracle import attention as oa


def spread(q, k, v, do, ob, lb, seqs, scale=None):
    """What the errors ob and lb of out and lse add to the bounds of (dq, dk, dv)."""
    _, _, Hq, D = q.shape
    G = Hq // k.shape[2]
    scale = D ** -0.5 if scale is None else scale
    extra = [np.zeros(x.shape) for x in (q, k, v)]
    o, lse = oa.attn_fwd(q, k, v, seqs, True, scale)[:2]
    for q0, n, k0, m in seqs:
        mask = np.arange(m)[None] < oa.seen(n, m, True)[:, None]
        for r in range(q.shape[0]):
            for h in range(Hq):
                rows, keys = (r, slice(q0, q0 + n), h), (r, slice(k0, k0 + m), h // G)
                Q, K, V, dO, L, e = q[rows], k[keys], v[keys], do[rows], lse[rows], lb[rows][:, None]
                L = np.where(np.isneginf(L), np.inf, L)[:, None]
                p = np.where(mask, np.exp(np.where(mask, Q @ K.T * scale, 0.0) - L), 0.0)
                ds = np.abs(dO @ V.T - (dO * o[rows]).sum(1)[:, None])
                dl = (ob[rows] * np.abs(dO)).sum(1)[:, None]
                x = p * ((1 + np.expm1(e)) * dl + np.expm1(e) * ds)
                extra[0][rows] += scale * x @ np.abs(K)
                extra[1][keys] += scale * x.T @ np.abs(Q)
                extra[2][keys] += (p * np.expm1(e)).T @ np.abs(dO)
    return extra


def blocks(shape, seqs, side, tokens):
    """Index tuples of what is moved at a time: each rank and head's part of a sequence, or of
    one of its tokens."""
    for s in seqs:
        first, n = (s[0], s[1]) if side == "q" else (s[2], s[3])
        for r in range(shape[0]):
            for h in range(shape[2]):
                if tokens:
                    yield from ((r, slice(i, i + 1), h) for i in range(first, first + n))
                elif n:
                    yield r, slice(first, first + n), h


def compare(name, got, along, bound, x, do, seqs, tokens=False, step=1e-5):
    """For every block, moved along the direction `along` (near its gradient, so that the
    derivative is far above the bound): (got . t, difference quotient of sum(out * do), error
    bound)."""
    f = lambda y: np.nansum(oa.attn_fwd(y["q"], y["k"], y["v"], seqs)[0] * do)  # noqa: E731
    for at in blocks(x[name].shape, seqs, name, tokens):
        t = np.zeros_like(x[name])
        t[at] = along[at] / max(np.abs(along[at]).max(), 1e-30)
        want = (f({**x, name: x[name] + step * t}) - f({**x, name: x[name] - step * t})) / (2 * step)
        # central differences: the third derivative's share is O(step^2), rounding 2^-52 |f| / step
        slack = 1e-6 * abs(want) + 1e-7
        yield (got * t).sum(), want, (bound * np.abs(t)).sum() + slack
