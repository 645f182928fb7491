"""Attention at the sizes that its times are quoted for, against 64 bits (needs a GB300).

Rows of the forward pass and of dQ depend on their own query only, given the other results, and
the mask is aligned to the end: a run of queries [a, b) of a prompt is a later piece with keys
[0, b).  The last keys' gradients come from the last queries alone, the first keys' from all.
"""
import pytest
import torch

import ring_collectives_gb300 as rc
from oracle import attention as oa
from tests.test_gpu_attention import DEV, check_backward, check_forward, f64, inside, ints, problem, rand

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(DEV)
    rc.ring_set_timeout_ms(2000)


@pytest.mark.parametrize("ql,kl,Hq,Hkv,D", [((2500, 1, 777), (2500, 1, 777), 4, 1, 128), ((1333,), (1333,), 3, 3, 64),
                                            ((600, 301), (2600, 1003), 4, 2, 96)])
def test_prompts_and_pieces(ql, kl, Hq, Hkv, D):
    p = problem(ql, kl, Hq=Hq, Hkv=Hkv, D=D, seed=31)
    check_forward(p)
    check_backward(p)


def test_tokens_of_a_full_batch():
    kl = [200 + (i * 2917) % 7900 for i in range(64)]
    check_forward(problem([1] * 64, kl, Hq=32, Hkv=8, D=128, cap=8192, seed=32))


def test_one_token_on_a_long_cache():
    check_forward(problem([1], [32768], P=8, Hq=4, Hkv=1, D=128, cap=32768, seed=33))


def test_a_long_prompt_on_eight_ranks():
    """Four heads on one key head of 128 on each rank, 16384 tokens: 150 rows at the start, around the middle
    and at the end, on the first and the last rank."""
    T, G, D = 16384, 4, 128
    p = problem([T], [T], P=8, Hq=G, Hkv=1, D=D, seed=34)
    out, lse = torch.empty_like(p["q"]), torch.empty(p["q"].shape[:3], device=DEV)
    rc.attn_fwd(p["q"], p["k"], p["v"], out, lse, ints([0, T]), ints([0, T]))
    assert rc.ring_status() == 0, rc.ring_last_error()
    for r in (0, 7):
        k, v = (f64(p[n][r:r + 1]) for n in "kv")
        for a in (0, 8101, T - 150):
            rows = slice(a, a + 150)
            o, ls, ob, lb = oa.attn_fwd(f64(p["q"][r:r + 1, rows]), k, v, [(0, 150, 0, a + 150)])
            inside(out[r:r + 1, rows], o, ob, "out")
            inside(lse[r:r + 1, rows], ls, lb, "lse")


def test_a_long_gradient_on_eight_ranks():
    """The same heads, 8192 tokens: dQ in three places, dK and dV of the first and of the last keys."""
    T, G, D, n = 8192, 4, 128, 130
    p = problem([T], [T], P=8, Hq=G, Hkv=1, D=D, seed=35)
    cu = ints([0, T])
    out, lse = torch.empty_like(p["q"]), torch.empty(p["q"].shape[:3], device=DEV)
    rc.attn_fwd(p["q"], p["k"], p["v"], out, lse, cu, cu)
    do = rand(p["g"], *p["q"].shape)
    dq, dk, dv = (torch.full_like(p[x], float("nan")) for x in "qkv")
    rc.attn_bwd(p["q"], p["k"], p["v"], out, lse, do, dq, dk, dv, cu, cu)
    assert rc.ring_status() == 0, rc.ring_last_error()
    for r in (0, 7):
        q, k, v, o, ls, d = (f64(x[r:r + 1]) for x in (p["q"], p["k"], p["v"], out, lse, do))

        def part(a, b, c, e, causal=True):
            """Gradients from queries [a, b) on keys [c, e)."""
            return oa.attn_bwd(q[:, a:b], k[:, c:e], v[:, c:e], o[:, a:b], ls[:, a:b], d[:, a:b],
                               [(0, b - a, 0, e - c)], causal)

        for a in (0, 4003, T - n):
            want, bound = part(a, a + n, 0, a + n)
            inside(dq[r:r + 1, a:a + n], want[0], bound[0], "dq")
        want, bound = part(T - n, T, T - n, T)
        for x, i in ((dk, 1), (dv, 2)):
            inside(x[r:r + 1, T - n:], want[i], bound[i], "the last keys")
        (w0, b0), (w1, b1) = part(0, n, 0, n), part(n, T, 0, n, causal=False)
        for x, i in ((dk, 1), (dv, 2)):
            inside(x[r:r + 1, :n], w0[i] + w1[i], b0[i] + b1[i], "the first keys")
