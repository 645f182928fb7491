"""Attention and query/key norm with rotation, from their definitions, in 64 bits.

TEST INFRASTRUCTURE, under the rules of the package: plain numpy, sharing
nothing with the CUDA library.  Arrays are float64 of the layouts the calls
take: q, o, do [P, Tq, Hq, D]; k, v [P, Tk, Hkv, D]; lse [P, Tq, Hq].  A sequence is
(first query, queries, first key, keys).  Token i of n queries sees the first
max(0, min(m, i + 1 + m - n)) of m keys under the causal mask, else all m.

Next to each result stands what its binary32 / bf16 evaluation can be off by,
from the error of each step:
  * u = 2^-8: rounding to bf16, which keeps 8 significant bits (the results,
    and the weights and score gradients that go into a product);
  * e = 2^-24 (n + 8): n-term binary32 sums, relative to the sum of magnitudes
    (doubled: the tensor cores do not promise the order or the rounding);
  * scores are off by ds = 2 e(D) scale sum |q k| plus 2^-22 (1 + |s|) for the
    exponential and its argument, which moves a weight by the same share.
"""
from __future__ import annotations

import numpy as np

U = 2.0 ** -8
E = 2.0 ** -24


def sequences(cu_q, cu_k, used_k=None):
    n = len(cu_q) - 1
    return [(cu_q[b], cu_q[b + 1] - cu_q[b], cu_k[b], cu_k[b + 1] - cu_k[b] if used_k is None else used_k[b])
            for b in range(n)]


def seen(n, m, causal):
    return np.clip(np.arange(1, n + 1) + m - n, 0, m) if causal else np.full(n, m)


def _weights(q, k, vis, scale):
    """Scores' weights [n, m] of the visible prefixes, log-sums and the scores' error."""
    with np.errstate(invalid="ignore", over="ignore"):
        mask = np.arange(k.shape[0])[None] < vis[:, None]
        s = np.where(mask, (q @ np.where(np.isfinite(k), k, 0.0).T) * scale, -np.inf)
        if not np.isfinite(k).all():
            bad = ~np.isfinite(k).all(1)
            s = np.where(mask & bad[None], np.nan, s)
        off = np.where(mask, 2 * (q.shape[1] + 8) * E * scale * (np.abs(q) @ np.abs(np.where(np.isfinite(k), k, 0.0)).T), 0.0)
        off = off + 2.0 ** -22 * (1 + np.abs(np.where(mask, np.nan_to_num(s), 0.0)))
        m = np.max(np.where(mask, s, -np.inf), axis=1, initial=-np.inf)
        m0 = np.where(np.isneginf(m), 0.0, m)
        w = np.where(mask, np.exp(s - m0[:, None]), 0.0)
        tot = w.sum(1)
        lse = np.where(tot == 0, -np.inf, m0 + np.log(np.where(tot == 0, 1.0, tot)))
        return w / np.where(tot == 0, 1.0, tot)[:, None], lse, off.max(axis=1, initial=0.0)


def _mix(w, v, vis):
    """w @ v over each row's visible prefix only (0 x inf never happens)."""
    with np.errstate(invalid="ignore"):
        return np.stack([w[i, :vis[i]] @ v[:vis[i]] for i in range(len(vis))]) if len(vis) else np.zeros((0, v.shape[1]))


def attn_fwd(q, k, v, seqs, causal=True, scale=None):
    """(out, lse, bound of out, bound of lse); rows outside every sequence are NaN."""
    P, Tq, Hq, D = q.shape
    G = Hq // k.shape[2]
    scale = D ** -0.5 if scale is None else scale
    out, lse = np.full(q.shape, np.nan), np.full(q.shape[:3], np.nan)
    ob, lb = np.zeros(q.shape), np.zeros(q.shape[:3])
    for q0, n, k0, m in seqs:
        vis = seen(n, m, causal)
        for r in range(P):
            for h in range(Hq):
                kk, vv = k[r, k0:k0 + m, h // G], v[r, k0:k0 + m, h // G]
                w, ls, off = _weights(q[r, q0:q0 + n, h], kk, vis, scale)
                o = _mix(w, vv, vis)
                mag = w @ np.abs(np.where(np.isfinite(vv), vv, 0.0))
                out[r, q0:q0 + n, h], lse[r, q0:q0 + n, h] = o, ls
                ob[r, q0:q0 + n, h] = (U + 2 * off[:, None] + 2 * (m + 8) * E) * mag + U * np.abs(np.nan_to_num(o)) + 1e-30
                lb[r, q0:q0 + n, h] = off + (m + 8) * E + 2.0 ** -22 * (1 + np.abs(np.where(np.isfinite(ls), ls, 0.0)))
    return out, lse, ob, lb


def attn_bwd(q, k, v, o, lse, do, seqs, causal=True, scale=None):
    """((dq, dk, dv), their bounds) from the forward results o and lse as given; NaN outside the sequences."""
    P, Tq, Hq, D = q.shape
    G = Hq // k.shape[2]
    scale = D ** -0.5 if scale is None else scale
    g = [np.full(x.shape, np.nan) for x in (q, k, v)]
    b = [np.zeros(x.shape) for x in (q, k, v)]
    for q0, n, k0, m in seqs:
        vis = seen(n, m, causal)
        for r in range(P):
            for x in (g[1], g[2]):
                x[r, k0:k0 + m] = 0.0
            for h in range(Hq):
                qs, ks, rows, keys = slice(q0, q0 + n), slice(k0, k0 + m), (r, slice(q0, q0 + n), h), (r, slice(k0, k0 + m), h // G)
                Q, K, V, O, dO, L = q[rows], k[keys], v[keys], o[rows], do[rows], lse[rows]
                mask = np.arange(m)[None] < vis[:, None]
                s = Q @ K.T * scale
                p = np.where(mask, np.exp(np.where(mask, s, 0.0) - np.where(np.isneginf(L), np.inf, L)[:, None]), 0.0)
                ep = 2 * (D + 8) * E * scale * (np.abs(Q) @ np.abs(K).T) + 2.0 ** -22 * (2 + np.abs(s) + np.abs(np.where(np.isneginf(L), 0, L))[:, None])
                dp, delta = dO @ V.T, (dO * O).sum(1)[:, None]
                edp = 2 * (D + 8) * E * (np.abs(dO) @ np.abs(V).T + (np.abs(dO) * np.abs(O)).sum(1)[:, None])
                ds = p * (dp - delta)
                eds = (U + ep) * np.abs(ds) + p * edp
                g[0][rows] = scale * ds @ K
                b[0][rows] = scale * (eds + 2 * (m + 8) * E * np.abs(ds)) @ np.abs(K) + 1e-30
                g[1][keys] += scale * ds.T @ Q
                b[1][keys] += scale * (eds + 2 * (n * G + 8) * E * np.abs(ds)).T @ np.abs(Q) + 1e-30
                g[2][keys] += p.T @ dO
                b[2][keys] += (p * (U + ep + 2 * (n * G + 8) * E)).T @ np.abs(dO) + 1e-30
    return g, [x + U * np.abs(np.nan_to_num(y)) for x, y in zip(b, g)]


def _pairs(D, pairs):
    a = np.arange(D // 2) * (2 if pairs else 1)
    return a, a + (1 if pairs else D // 2)


def qk_norm_rope(x, gamma, cos, sin, pos, pairs=False, eps=1e-6):
    """(z, bound) for heads x [P, T, H, D]."""
    a, b = _pairs(x.shape[-1], pairs)
    c, s = cos[pos][:, None], sin[pos][:, None]
    y = x / np.sqrt((x ** 2).mean(-1, keepdims=True) + eps) * gamma
    z, mag = np.empty_like(y), np.empty_like(y)
    z[..., a], z[..., b] = y[..., a] * c - y[..., b] * s, y[..., a] * s + y[..., b] * c
    mag[..., a] = np.abs(y[..., a] * c) + np.abs(y[..., b] * s)
    mag[..., b] = np.abs(y[..., a] * s) + np.abs(y[..., b] * c)
    return z, U * np.abs(z) + (x.shape[-1] + 16) * E * mag + 1e-30


def qk_norm_rope_bwd(x, gamma, cos, sin, pos, dz, pairs=False, eps=1e-6):
    """(dx, dgamma [P, D], bound of dx, bound of dgamma)."""
    D = x.shape[-1]
    a, b = _pairs(D, pairs)
    c, s = cos[pos][:, None], sin[pos][:, None]
    dy, mag = np.empty_like(dz), np.empty_like(dz)
    dy[..., a], dy[..., b] = dz[..., a] * c + dz[..., b] * s, dz[..., b] * c - dz[..., a] * s
    mag[..., a] = np.abs(dz[..., a] * c) + np.abs(dz[..., b] * s)
    mag[..., b] = np.abs(dz[..., b] * c) + np.abs(dz[..., a] * s)
    r = 1.0 / np.sqrt((x ** 2).mean(-1, keepdims=True) + eps)
    xh, t = x * r, dy * gamma
    dx = r * (t - xh * (t * xh).mean(-1, keepdims=True))
    tm = mag * np.abs(gamma)
    e = (2 * D + 32) * E
    bx = U * np.abs(dx) + e * r * (tm + np.abs(xh) * (tm * np.abs(xh)).mean(-1, keepdims=True)) + 1e-30
    n = x.shape[1] * x.shape[2]
    return dx, (dy * xh).sum((1, 2)), bx, (e + 2 * (n + 8) * E) * (mag * np.abs(xh)).sum((1, 2)) + 1e-30
