"""GPU gradients of attention against differences of the definition, with a bound far below the
derivative (needs a GB300)."""
import pytest
import torch

import ring_collectives_gb300 as rc
from oracle import attention as oa
from tests.attention_differences import compare, spread
from tests.test_gpu_attention import DEV, f64, forward, ints, problem, rand, seqs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(DEV)
    rc.ring_set_timeout_ms(2000)


@pytest.mark.parametrize("ql,kl,Hq,Hkv,D", [((65, 20), (65, 150), 4, 2, 64), ((33, 7), (33, 40), 4, 1, 32), ((130,), (131,), 2, 2, 128)])
def test_gradients_are_the_derivatives(ql, kl, Hq, Hkv, D):
    p = problem(ql, kl, Hq=Hq, Hkv=Hkv, D=D, seed=21)
    out, lse = forward(p)
    do = rand(p["g"], *p["q"].shape)
    grads = [torch.empty_like(p[n]) for n in "qkv"]
    rc.attn_bwd(p["q"], p["k"], p["v"], out, lse, do, *grads, ints(p["cu_q"]), ints(p["cu_k"]))
    assert rc.ring_status() == 0, rc.ring_last_error()
    x, d, s = {n: f64(p[n]) for n in "qkv"}, f64(do), seqs(p)
    _, _, ob, lb = oa.attn_fwd(x["q"], x["k"], x["v"], s)
    along, bounds = oa.attn_bwd(x["q"], x["k"], x["v"], f64(out), f64(lse), d, s)
    for n, g, a, b, e in zip("qkv", grads, along, bounds, spread(x["q"], x["k"], x["v"], d, ob, lb, s)):
        for got, want, bound in compare(n, f64(g), a, b + e, x, d, s):
            assert abs(got - want) <= bound < abs(want) / 2, (n, got, want, bound)   # or nothing would be said
        for got, want, bound in compare(n, f64(g), a, b + e, x, d, s, tokens=True):
            assert abs(got - want) <= bound, (n, got, want, bound)
