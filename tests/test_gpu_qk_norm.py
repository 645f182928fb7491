"""GPU query/key norm with rotation, and its gradient, against 64 bits (needs a GB300)."""
import numpy as np
import pytest
import torch

import ring_collectives_gb300 as rc
from oracle import attention as oa

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(DEV)


def f64(t):
    return t.detach().double().cpu().numpy()


def problem(P, T, Hq, Hkv, D, seed=0, npos=50):
    g = torch.Generator(device=DEV).manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    ang = r(npos, D // 2) * 3
    return dict(q=r(P, T, Hq, D).to(BF), k=r(P, T, Hkv, D).to(BF), gq=r(D), gk=r(D), cos=ang.cos(), sin=ang.sin(),
                pos=torch.randint(0, npos, (T,), generator=g, device=DEV, dtype=torch.int32),
                dq=r(P, T, Hq, D).to(BF), dk=r(P, T, Hkv, D).to(BF))


def common(p):
    return p["q"], p["k"], p["gq"], p["gk"], p["cos"], p["sin"], p["pos"]


def inside(got, want, bound):
    err = np.abs(f64(got) - want)
    assert (err <= bound).all(), float((err / bound).max())


def check(p, layout, eps=1e-6):
    pairs = layout == rc.RC_ROPE_PAIRS
    qo, ko = torch.full_like(p["q"], float("nan")), torch.full_like(p["k"], float("nan"))
    rc.qk_norm_rope(*common(p), qo, ko, layout=layout, eps=eps)
    P, _, _, D = p["q"].shape
    dq, dk, dgq, dgk = qo.clone(), ko.clone(), torch.empty(P, D, device=DEV), torch.empty(P, D, device=DEV)
    rc.qk_norm_rope_bwd(*common(p), p["dq"], p["dk"], dq, dk, dgq, dgk, layout=layout, eps=eps)
    c, s, pos = f64(p["cos"]), f64(p["sin"]), p["pos"].cpu().numpy()
    for x, g, z, dz, dx, dg in ((p["q"], p["gq"], qo, p["dq"], dq, dgq), (p["k"], p["gk"], ko, p["dk"], dk, dgk)):
        inside(z, *oa.qk_norm_rope(f64(x), f64(g), c, s, pos, pairs, eps))
        wx, wg, bx, bg = oa.qk_norm_rope_bwd(f64(x), f64(g), c, s, pos, f64(dz), pairs, eps)
        inside(dx, wx, bx)
        inside(dg, wg, bg)
    return qo, ko, dq, dk, dgq, dgk


@pytest.mark.parametrize("layout", [0, 1])
@pytest.mark.parametrize("D", [8, 16, 24, 40, 64, 80, 96, 120, 128, 176, 200, 248, 256])
def test_head_sizes(D, layout):
    check(problem(2, 37, 3, 2, D, seed=D), layout)


@pytest.mark.parametrize("P,T,Hq,Hkv", [(1, 1, 1, 1), (8, 64, 4, 1), (1, 1000, 12, 12), (3, 333, 9, 5), (64, 2, 1, 1), (1, 5, 70, 3)])
def test_shapes(P, T, Hq, Hkv):
    check(problem(P, T, Hq, Hkv, 128, seed=1), 0)


def test_small_and_zero_heads():
    """A head of zeros has r = eps^-1/2: finite, with gradient r dy; a tiny one is carried by eps."""
    p = problem(1, 6, 2, 1, 64, seed=2)
    p["q"][0, 0] = 0
    p["q"][0, 1] *= 2.0 ** -20
    check(p, 0)
    check(p, 1, eps=1e-2)


def test_views_in_place_and_gaps():
    P, T, Hq, Hkv, D = 2, 45, 4, 2, 64
    p = problem(P, T, Hq, Hkv, D, seed=3)
    qo, ko, dq, dk, dgq, dgk = check(p, 0)
    fused = torch.full((T, P, Hq + 2 * Hkv, D), 5.0, dtype=BF, device=DEV)
    q, k = (x.transpose(0, 1) for x in (fused[:, :, :Hq], fused[:, :, Hq:Hq + Hkv]))
    q.copy_(p["q"]), k.copy_(p["k"])
    rc.qk_norm_rope(q, k, *common(p)[2:], q, k)                     # in place, strided
    assert torch.equal(q, qo) and torch.equal(k, ko) and (fused[:, :, Hq + Hkv:] == 5).all()
    a, b, ga, gb = p["dq"].clone(), p["dk"].clone(), torch.empty_like(dgq), torch.empty_like(dgk)
    rc.qk_norm_rope_bwd(*common(p), a, b, a, b, ga, gb)             # gradients in place
    assert all(torch.equal(x, y) for x, y in ((a, dq), (b, dk), (ga, dgq), (gb, dgk)))


def test_positions_outside_the_table_are_nan():
    p = problem(1, 4, 2, 1, 64, seed=4)
    qo, ko = torch.empty_like(p["q"]), torch.empty_like(p["k"])
    rc.qk_norm_rope(*common(p), qo, ko)
    p["pos"][1], p["pos"][2] = -1, 50
    q2, k2 = torch.empty_like(p["q"]), torch.empty_like(p["k"])
    rc.qk_norm_rope(*common(p), q2, k2)
    assert torch.isnan(q2[0, 1:3]).all() and torch.isnan(k2[0, 1:3]).all()
    assert torch.equal(q2[0, ::3], qo[0, ::3]) and torch.equal(k2[0, ::3], ko[0, ::3])


def test_a_non_finite_head_stays_alone():
    p = problem(1, 8, 4, 2, 128, seed=5)
    qo, ko = torch.empty_like(p["q"]), torch.empty_like(p["k"])
    rc.qk_norm_rope(*common(p), qo, ko)
    p["q"][0, 3, 1, 7] = float("nan")
    q2, k2 = torch.empty_like(p["q"]), torch.empty_like(p["k"])
    rc.qk_norm_rope(*common(p), q2, k2)
    assert torch.isnan(q2[0, 3, 1]).all()
    q2[0, 3, 1] = qo[0, 3, 1]
    assert torch.equal(q2, qo) and torch.equal(k2, ko)


def test_same_bits_streams_and_workspace():
    p = problem(4, 700, 4, 2, 128, seed=6)
    P, T, Hq, D = p["q"].shape
    want = check(p, 0)
    s = torch.cuda.Stream()
    ws = torch.full((rc.qk_norm_rope_bwd_workspace_bytes(P, T, Hq, 2, D),), 255, dtype=torch.uint8, device=DEV)
    torch.cuda.synchronize()
    for _ in range(5):
        dq, dk, a, b = torch.empty_like(p["q"]), torch.empty_like(p["k"]), torch.empty(P, D, device=DEV), torch.empty(P, D, device=DEV)
        s.wait_stream(torch.cuda.current_stream())
        rc.qk_norm_rope_bwd(*common(p), p["dq"], p["dk"], dq, dk, a, b, workspace=ws, stream=s)
        s.synchronize()
        assert all(torch.equal(x, y) for x, y in zip((dq, dk, a, b), want[2:]))
    with pytest.raises(rc.RingError):
        rc.qk_norm_rope_bwd(*common(p), p["dq"], p["dk"], dq, dk, a, b, workspace=ws[:256])


def test_no_tokens_give_no_gradient():
    p = problem(2, 0, 2, 1, 64)
    a, b = torch.full((2, 64), 9.0, device=DEV), torch.full((2, 64), 9.0, device=DEV)
    rc.qk_norm_rope_bwd(*common(p), p["dq"], p["dk"], p["dq"].clone(), p["dk"].clone(), a, b)
    assert (a == 0).all() and (b == 0).all()


def test_rank_gradients_reduce_round_the_ring():
    """dgamma slots are what ring_allreduce takes: the gradient of the shared weight on every rank."""
    p = problem(4, 50, 2, 1, 64, seed=7)
    a, b = torch.empty(4, 64, device=DEV), torch.empty(4, 64, device=DEV)
    rc.qk_norm_rope_bwd(*common(p), p["dq"], p["dk"], torch.empty_like(p["q"]), torch.empty_like(p["k"]), a, b)
    total = a.double().sum(0)
    rc.ring_allreduce(a)
    assert rc.ring_status() == 0
    assert (a.double() - total).abs().max() <= 4 * 2.0 ** -24 * a.abs().max() * 4
    assert torch.equal(a[0], a[3])
