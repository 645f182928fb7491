"""8-bit activations, norms around the residual sum, gated activations and weight gradients, from
their definitions, in 64 bits.

TEST INFRASTRUCTURE, under the rules of the package: plain numpy, sharing nothing with the CUDA
library.  Arrays are float64 (8-bit forms int8 and uint8) of shape [P, T, N].

Next to each result stands what its binary32 / bf16 evaluation can be off by, to first order in the
unit roundings, step by step as the formulas are written:
  * U = 2^-8: rounding a result to bf16;  E = 2^-24: one binary32 operation, relative to its result;
  * ROW = 64 E: a sum over a row, relative to its sum of magnitudes (no element passes through more
    than 16 products added up in a thread, 1 + 5 additions in its warp, and 32 over warps);
  * 4 E: a reciprocal square root (two units in the last place), 2 E: a reciprocal (one);
  * (4 + 2.4 |c|) E: exp(c) (2 + 1.173 |c| units in the last place), of an argument that is itself off.
"""
from __future__ import annotations

import numpy as np

U = 2.0 ** -8
E = 2.0 ** -24
ROW = 64 * E
GROUP = 32


# ---------------------------------------------------------------- 8 bits
def act8_pack(x):
    """(q, e) of bf16 values given in float64."""
    P, T, N = x.shape
    G = -(-N // GROUP)
    v = np.zeros((P, T, G * GROUP))
    v[..., :N] = x
    v = v.reshape(P, T, G, GROUP)
    bad = ~np.isfinite(v).all(-1)
    v = np.where(bad[..., None], 0.0, v)
    top = np.abs(v).max(-1)
    k = np.full(top.shape, -126)
    for i in range(-126, 121):                        # the least k with top <= 127 * 2^k, at most 121
        k = np.where(top > 127 * 2.0 ** i, i + 1, k)
    q = np.clip(np.rint(v * 2.0 ** -k[..., None].astype(float)), -127, 127)
    return (q.reshape(P, T, G * GROUP)[..., :N].astype(np.int8), np.where(bad, 255, k + 127).astype(np.uint8))


def act8_values(q, e):
    g = np.arange(q.shape[-1]) // GROUP
    with np.errstate(invalid="ignore"):
        return np.where(e[..., g] == 255, np.nan, q * 2.0 ** (e.astype(float) - 127)[..., g])


# ---------------------------------------------------------------- norms around the residual sum
def from_cols(y, T):
    """[P, P * T, N / P] as [P, T, N]."""
    P, _, c = y.shape
    return y.transpose(1, 0, 2).reshape(P, T, P * c)


def to_cols(y):
    P, T, N = y.shape
    return y.reshape(P * T, P, N // P).transpose(1, 0, 2)


def _mean(x):
    return x.mean(-1, keepdims=True)


def _forward(y, res, post, gate, alpha, eps):
    """yh, w, h with their errors, and 1 / rms(y) with its relative error."""
    p, pe = np.ones_like(y[..., :1]), np.zeros_like(y[..., :1])
    if post is not None:
        p, pe = 1 / np.sqrt(_mean(y ** 2) + eps), pe + ROW / 2 + 5 * E
    w = alpha * (1.0 if gate is None else gate) * (1.0 if post is None else post) * np.ones(y.shape[-1])
    yh = y * p
    eyh = np.abs(yh) * (pe + E)
    x = w * yh
    h = res + x
    eh = np.abs(w) * eyh + 3 * E * np.abs(x) + E * np.abs(h)
    return yh, eyh, w, h, eh, p, pe


def _rms(h, eh, eps):
    """1 / rms(h) and its relative error."""
    q = 1 / np.sqrt(_mean(h ** 2) + eps)
    return q, _mean(np.abs(h) * eh) * q ** 2 + ROW / 2 + 5 * E


def block_norm(y, res, post=None, gate=None, pre=None, alpha=1.0, eps=1e-6):
    """((h, z or None), their bounds)."""
    _, _, _, h, eh, _, _ = _forward(y, res, post, gate, alpha, eps)
    hb = eh + U * np.abs(h) + 1e-37
    if pre is None:
        return (h, None), (hb, None)
    q, qe = _rms(h, eh, eps)
    z = h * q * pre
    return (h, z), (hb, np.abs(q * pre) * eh + np.abs(z) * (qe + 3 * E + U) + 1e-37)


def block_norm_bwd(y, res, dh, dz, post=None, gate=None, pre=None, alpha=1.0, eps=1e-6):
    """(results, bounds) as dicts: dy, dres [P, T, N]; dgamma_post, dgate, dgamma_pre [P, N] where given."""
    P, T, N = y.shape
    a = np.abs
    yh, eyh, w, h, eh, p, pe = _forward(y, res, post, gate, alpha, eps)
    d, ed = dh.copy(), np.zeros_like(dh)
    out, off = {}, {}
    x = w * yh
    ex = a(w) * eyh + 3 * E * a(x)
    rows = lambda e: e.sum(1) + 0.0                                  # noqa: E731

    def total(u, v, eu, ev):
        """mean(u v) over the row and its error."""
        return _mean(u * v), _mean(a(u) * ev + a(v) * eu) + ROW * _mean(a(u * v))

    q = c = ec = qe = 0.0
    t = et = np.zeros_like(dh)
    if pre is not None:
        q, qe = _rms(h, eh, eps)
        t = dz * pre
        et = E * a(t)
        th, eth = total(t, h, et, eh)
        c = q ** 3 * th
        ec = a(c) * (3 * qe + 5 * E) + q ** 3 * eth
        d = dh + q * t - c * h
        ed = q * et + a(q * t) * (qe + E) + a(c) * eh + a(h) * ec + 3 * E * (a(dh) + a(q * t) + a(c * h))
        out["dgamma_pre"] = (dz * h * q).sum(1)
        off["dgamma_pre"] = rows(a(dz) * (q * eh + a(h * q) * (qe + 2 * E))) + (T + 64) * E * rows(a(dz * h * q))
    out["dres"], off["dres"] = d, ed + U * a(d) + 1e-37
    s = d * yh
    es = rows(a(d) * eyh + a(yh) * ed) + (T + 64) * E * rows(a(s))
    s = s.sum(1)
    for name, own, other in (("dgamma_post", post, gate), ("dgate", gate, post)):
        if own is not None:
            f = alpha * (1.0 if other is None else other)
            out[name], off[name] = f * s, a(f) * es + 3 * E * a(f * s)
    u = d * w
    eu = a(w) * ed + 3 * E * a(u)
    dy, ey = u, eu
    if post is not None:
        (vd, evd), (vt, evt), (vh, evh) = total(x, dh, ex, np.zeros_like(dh)), total(x, t, ex, et), total(x, h, ex, eh)
        m = vd + q * vt - c * vh
        em = evd + q * evt + a(q * vt) * qe + a(c) * evh + a(vh) * ec + 5 * E * (a(vd) + a(q * vt) + a(c * vh))
        dy = p * (u - yh * m)
        ey = p * (eu + a(yh) * em + a(m) * eyh + 2 * E * (a(u) + a(yh * m))) + a(dy) * (pe + 2 * E)
    out["dy"], off["dy"] = dy, ey + U * a(dy) + 1e-37
    return out, {k: v + 1e-37 for k, v in off.items()}


# ---------------------------------------------------------------- gated activations
def _act(x, kind):
    """act(x), act'(x) and their errors."""
    a = np.abs
    if kind == "silu":
        c, slope, ec = x, x, 0.0 * x
    else:
        root = 2 * np.sqrt(2 / np.pi)
        c, slope = root * x * (1 + 0.044715 * x * x), root * x * (1 + 3 * 0.044715 * x * x)
        ec = 6 * E * a(c)                             # both terms have one sign
    with np.errstate(over="ignore"):
        s, t = 1 / (1 + np.exp(-c)), 1 / (1 + np.exp(c))
    exp = (4 + 2.4 * a(c)) * E + ec
    es, et = s * (t * exp + 4 * E), t * (s * exp + 4 * E)
    d = s * (1 + slope * t)
    ed = es * (1 + a(slope) * t) + s * a(slope) * (et + 6 * E * t) + 3 * E * s * (1 + a(slope) * t)
    tiny = 1e-37 * (1 + a(slope))                     # results below the normal numbers
    return x * s, a(x) * (es + E * s) + tiny, d, ed + tiny


def glu(a, b, kind):
    """(h, bound)."""
    f, ef, _, _ = _act(a, kind)
    return f * b, np.abs(b) * ef + (U + E) * np.abs(f * b) + 1e-37


def glu_bwd(a, b, dh, kind):
    """((da, db, h), bounds)."""
    f, ef, d, ed = _act(a, kind)
    g = (dh * b * d, dh * f, f * b)
    e = (np.abs(dh * b) * ed, np.abs(dh) * ef, np.abs(b) * ef)
    return g, tuple(x + (U + 3 * E) * np.abs(y) + 1e-37 for x, y in zip(e, g))


# ---------------------------------------------------------------- weight gradient
def gemm_wgrad(dy, x, rounding=U):
    """(dw, bound): a T-term binary32 sum in any order and rounding, then one rounding to the result's type."""
    dw, mag = dy.transpose(0, 2, 1) @ x, np.abs(dy).transpose(0, 2, 1) @ np.abs(x)
    return dw, rounding * np.abs(dw) + 2 * (dy.shape[1] + 8) * E * mag + 1e-37
