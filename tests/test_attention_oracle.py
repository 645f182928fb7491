"""The 64-bit statements of attention and query/key norm (CPU): gradients
against differences, closed forms, masks, and planted mistakes that the same
checks must catch."""
import numpy as np
import pytest

from oracle import attention as oa


def _case(seed=0, P=1, ql=(3, 1, 4), kl=(3, 5, 2), Hq=4, Hkv=2, D=8):
    g = np.random.default_rng(seed)
    cu_q, cu_k = np.cumsum((0,) + ql), np.cumsum((0,) + kl)
    q, do = (g.standard_normal((P, cu_q[-1], Hq, D)) for _ in range(2))
    k, v = (g.standard_normal((P, cu_k[-1], Hkv, D)) for _ in range(2))
    return q, k, v, do, oa.sequences(cu_q, cu_k)


def _difference(f, x, step=1e-5):
    d = np.zeros_like(x)
    for i in np.ndindex(*x.shape):
        y = x.copy()
        y[i] += step
        up = f(y)
        y[i] -= 2 * step
        d[i] = (up - f(y)) / (2 * step)
    return d


def _attn_gradient_error(module, causal):
    q, k, v, do, seqs = _case()
    fwd = lambda *a: (module.attn_fwd(*a, seqs, causal)[0] * do).sum()  # noqa: E731
    o, lse = module.attn_fwd(q, k, v, seqs, causal)[:2]
    got, _ = module.attn_bwd(q, k, v, o, lse, do, seqs, causal)
    want = (_difference(lambda x: fwd(x, k, v), q), _difference(lambda x: fwd(q, x, v), k),
            _difference(lambda x: fwd(q, k, x), v))
    return max(np.abs(a - b).max() for a, b in zip(got, want))


@pytest.mark.parametrize("causal", [True, False])
def test_attention_gradient_against_differences(causal):
    assert _attn_gradient_error(oa, causal) < 1e-7      # central differences: O(1e-10) + rounding 1e-16 / 1e-5


@pytest.mark.parametrize("pairs", [False, True])
def test_norm_gradient_against_differences(pairs):
    g = np.random.default_rng(3)
    x, dz = g.standard_normal((2, 3, 2, 8)), g.standard_normal((2, 3, 2, 8))
    gamma, ang, pos = g.standard_normal(8), g.standard_normal((5, 4)), np.array([4, 0, 2])
    f = lambda x, gamma: (oa.qk_norm_rope(x, gamma, np.cos(ang), np.sin(ang), pos, pairs)[0] * dz).sum()  # noqa: E731
    dx, dg, _, _ = oa.qk_norm_rope_bwd(x, gamma, np.cos(ang), np.sin(ang), pos, dz, pairs)
    assert np.abs(dx - _difference(lambda y: f(y, gamma), x)).max() < 1e-7
    assert np.abs(dg.sum(0) - _difference(lambda y: f(x, y), gamma)).max() < 1e-7


def test_attention_closed_forms():
    q, k, v, _, seqs = _case()
    out, lse, _, _ = oa.attn_fwd(np.zeros_like(q), k, v, seqs, True)
    for q0, n, k0, m in seqs:                           # equal scores: the mean of what is seen
        for i in range(n):
            c = max(0, min(m, i + 1 + m - n))
            want = v[0, k0:k0 + c].mean(0) if c else np.zeros_like(v[0, 0])
            assert np.allclose(out[0, q0 + i], np.repeat(want, 2, axis=0))
            assert np.allclose(lse[0, q0 + i], np.log(c) if c else -np.inf)


def test_a_hidden_value_never_counts():
    q, k, v, _, seqs = _case(ql=(4,), kl=(4,))
    clean = oa.attn_fwd(q, k, v, seqs, True)[0]
    k2, v2 = k.copy(), v.copy()
    k2[0, 3], v2[0, 3] = np.nan, np.inf
    out = oa.attn_fwd(q, k2, v2, seqs, True)[0]
    assert np.array_equal(out[0, :3], clean[0, :3]) and not np.isfinite(out[0, 3]).any()


def test_rotation_keeps_lengths_and_undoes_itself():
    g = np.random.default_rng(4)
    x = g.standard_normal((1, 2, 3, 16))
    ang, pos, one = g.standard_normal((7, 8)), np.array([6, 1]), np.ones(16)
    for pairs in (False, True):
        z, _ = oa.qk_norm_rope(x, one, np.cos(ang), np.sin(ang), pos, pairs, eps=0.0)
        assert np.allclose((z ** 2).mean(-1), 1.0)
        back, _ = oa.qk_norm_rope(z, one, np.cos(ang), -np.sin(ang), pos, pairs, eps=0.0)
        assert np.allclose(back, x / np.sqrt((x ** 2).mean(-1, keepdims=True)))


@pytest.mark.parametrize("old,new", [("scale * ds @ K", "ds @ K"), ("(dp - delta)", "(dp + delta)"),
                                     ("ds.T @ Q", "p.T @ Q"), ("h // G]", "h % k.shape[2]]"),
                                     ("+ m - n, 0, m)", ", 0, m)")])
def test_planted_mistakes_are_caught(old, new, tmp_path):
    """The same checks fail for copies of the oracle with one wrong term (the grouping and
    the mask are pinned by the closed forms)."""
    import importlib.util
    text = open(oa.__file__, encoding="utf-8").read()
    assert old in text
    path = tmp_path / "mutant.py"
    path.write_text(text.replace(old, new), encoding="utf-8")
    spec = importlib.util.spec_from_file_location("mutant", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    q, k, v, do, seqs = _case()
    same = np.allclose(m.attn_fwd(q, k, v, seqs, True)[0], oa.attn_fwd(q, k, v, seqs, True)[0])
    o, lse = oa.attn_fwd(q, k, v, seqs, True)[:2]
    got, want = m.attn_bwd(q, k, v, o, lse, do, seqs, True)[0], oa.attn_bwd(q, k, v, o, lse, do, seqs, True)[0]
    assert not (same and all(np.allclose(a, b) for a, b in zip(got, want)))
