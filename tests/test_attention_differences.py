"""The comparison of gradients with differences: a gradient that is right to the steps of a bf16
evaluation passes, and every planted mistake fails by far (CPU)."""
import numpy as np
import pytest

from oracle import attention as oa
from tests.attention_differences import compare, spread


def bf16(x):
    """Rounded to 8 significant bits."""
    m, e = np.frexp(x)
    return np.ldexp(np.round(m * 256) / 256, e)


@pytest.fixture(scope="module")
def case():
    g = np.random.default_rng(0)
    ql, kl, Hq, Hkv, D = (33, 7), (33, 40), 4, 2, 32
    cq, ck = np.cumsum((0,) + ql), np.cumsum((0,) + kl)
    q, do = (bf16(g.standard_normal((1, cq[-1], Hq, D))) for _ in range(2))
    k, v = (bf16(g.standard_normal((1, ck[-1], Hkv, D))) for _ in range(2))
    seqs = oa.sequences(cq, ck)
    o, lse, ob, lb = oa.attn_fwd(q, k, v, seqs)
    grads, bounds = oa.attn_bwd(q, k, v, bf16(o), lse, do, seqs)
    bounds = [b + e for b, e in zip(bounds, spread(q, k, v, do, ob, lb, seqs))]
    return dict(q=q, k=k, v=v), do, seqs, o, lse, grads, bounds


def outcome(case, which, got, tokens):
    x, do, seqs, _, _, grads, bounds = case
    n = "qkv"[which]
    return list(compare(n, got, grads[which], bounds[which], x, do, seqs, tokens))


@pytest.mark.parametrize("which", range(3))
def test_a_rounded_gradient_passes_and_the_bound_is_far_below_it(case, which):
    for got, want, bound in outcome(case, which, bf16(case[5][which]), False):
        assert abs(got - want) <= bound < abs(want) / 4
    assert all(abs(got - want) <= bound for got, want, bound in outcome(case, which, bf16(case[5][which]), True))


def _without_delta(case):
    x, do, seqs, o, lse, _, _ = case
    return oa.attn_bwd(x["q"], x["k"], x["v"], 0 * o, lse, do, seqs)[0]


def _without_scale(case):
    return [case[5][0] * 32 ** 0.5, case[5][1] * 32 ** 0.5, None]


def _no_mask(case):
    x, do, seqs, o, lse, _, _ = case
    return oa.attn_bwd(x["q"], x["k"], x["v"], o, lse, do, seqs, causal=False)[0]


@pytest.mark.parametrize("which,mistake", [
    (w, m) for w in range(3) for m in (lambda c: [0 * g for g in c[5]], lambda c: [-g for g in c[5]], _no_mask)]
    + [(w, m) for w in (0, 1) for m in (_without_delta, _without_scale)])
def test_mistakes_fail(case, which, mistake):
    wrong = mistake(case)[which]
    res = outcome(case, which, wrong, False) + outcome(case, which, wrong, True)
    assert max(abs(got - want) / bound for got, want, bound in res) > 2
