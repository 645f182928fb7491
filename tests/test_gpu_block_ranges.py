"""GPU block operators at few rows and at the ends of the number range, against 64 bits (needs a GB300)."""
import numpy as np
import pytest
import torch

import ring_collectives_gb300 as rc
from oracle import block as ob

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


def inside(got, want, bound):
    err = np.abs(f64(got) - want)
    assert (err <= bound).all(), float((err / bound).max())


def rand(seed, *shape):
    return torch.randn(shape, generator=torch.Generator(device=DEV).manual_seed(seed), device=DEV).to(BF)


def norm_problem(P, T, N, seed=0):
    y, res, dh, dz = (rand(seed + i, P, T, N) for i in range(4))
    w = [1 + 0.3 * torch.randn(N, generator=torch.Generator(device=DEV).manual_seed(seed + 4 + i), device=DEV) for i in range(3)]
    return y, res, dh, dz, w


def norm_gradient(y, res, dh, dz, w, held, alpha=0.7, eps=1e-6, workspace=None):
    """{name: result} of block_norm_bwd with the weights that are given."""
    P, T, N = dz.shape if dz is not None else dh.shape
    out = {k: torch.full((P, T, N), float("nan"), dtype=BF, device=DEV) for k in ("dy", "dres")}
    dw = [None if t is None else torch.full((P, N), float("nan"), device=DEV) for t in w]
    if held:
        y, res = (rc.act8_pack(t, rc.act8_empty(t.shape, DEV)) for t in (y, res))
    names = ("gamma_post", "gate", "gamma_pre")
    rc.block_norm_bwd(y, res, dh, dz, out["dy"], out["dres"], *dw, **dict(zip(names, w)), alpha=alpha, eps=eps, workspace=workspace)
    return out | {"d" + n: t for n, t in zip(names, dw) if t is not None}


def held_values(t):
    return ob.act8_values(*ob.act8_pack(f64(t)))


@pytest.mark.parametrize("held", [False, True], ids=["bf16", "8bit"])
@pytest.mark.parametrize("N", [8, 64, 72, 128, 136, 256, 264, 512])
def test_sums_of_few_narrow_rows(N, held):
    """Rows within a warp, fewer of them than a block takes at once: some warps have none, and each block's sums follow
    its last row at once.  The same bits every time."""
    for T in (1, 2, 3, 4, 5, 7, 8, 15, 16, 17):
        y, res, dh, dz, w = norm_problem(2, T, N, seed=T)
        first = norm_gradient(y, res, dh, dz, w, held)
        at = [held_values(t) if held else f64(t) for t in (y, res)]
        want, bound = ob.block_norm_bwd(*at, f64(dh), f64(dz), *(f64(t) for t in w), alpha=0.7)
        for name, t in first.items():
            inside(t, want[name], bound[name])
        for _ in range(20):
            again = norm_gradient(y, res, dh, dz, w, held)
            assert all(torch.equal(t, again[name]) for name, t in first.items())


# ---------------------------------------------------------------- gated activations
KINDS = {"silu": rc.RC_GLU_SILU, "gelu": rc.RC_GLU_GELU}


@pytest.mark.parametrize("held", [False, True], ids=["bf16", "8bit"])
@pytest.mark.parametrize("kind", ["silu", "gelu"])
def test_glu_gradient_of_every_finite_gate(kind, held):
    """With factors 3 and -1/2.  Beyond 100 the derivative is 1 or 0: the logistic function's distance from 1 or 0 is at
    most 100 e^-100 < 4e-42 there, times 1.5, so da is -1.5 without an error, or nearly nothing."""
    bits = torch.arange(65536, dtype=torch.int32, device=DEV).to(torch.int16).view(BF)
    a = torch.zeros((1, 65280, 32), dtype=BF, device=DEV)                # a group for every gate, with zeros
    a[0, :, 0] = bits[torch.isfinite(bits)]
    dh, b = torch.full_like(a, 3.0), torch.full_like(a, -0.5)
    da, db, h = (torch.full_like(a, float("nan")) for _ in range(3))
    operands = [rc.act8_pack(t, rc.act8_empty(t.shape, DEV)) for t in (a, b)] if held else [a, b]
    rc.glu_bwd(*operands, dh, da, db, h=h, act=KINDS[kind])
    x = held_values(a) if held else f64(a)
    (wa, wb, wh), (oa, obb, oh) = ob.glu_bwd(x, f64(b), f64(dh), kind)
    near = np.abs(x) <= 1e9                                              # the bound for tiny results grows beyond
    assert (np.abs(f64(da) - wa) <= oa)[near].all()
    assert (np.abs(f64(da) - np.where(x > 0, -1.5, 0.0)) <= 1e-37)[np.abs(x) >= 100].all()
    # db = 3 act(a) and h = -act(a) / 2: past the limit an infinity
    for got, want, off in ((db, wb, obb), (h, wh, oh)):
        fits = np.abs(want) <= 3.38e38
        assert (np.abs(f64(got) - want) <= off)[fits].all() and np.isinf(f64(got)[np.abs(want) > 3.4e38]).all()


# ---------------------------------------------------------------- norm's gradient: loud and quiet rows
def check_gradient(y, res, dh, dz, w, held, alpha, eps):
    got = norm_gradient(y, res, dh, dz, w, held, alpha, eps)
    at = [held_values(t) if held else f64(t) for t in (y, res)]
    at += [np.zeros(at[0].shape) if dh is None else f64(dh), f64(dz)]
    want, bound = ob.block_norm_bwd(*at, *(None if t is None else f64(t) for t in w), alpha=alpha, eps=eps)
    assert set(want) == set(got)
    for name, t in got.items():
        # the definition's bound counts 1e-37 for results below the normal numbers; those here are far above
        assert (np.abs(want[name]) > 1e-34).mean() > 0.9
        inside(t, want[name], bound[name])


@pytest.mark.parametrize("held", [False, True], ids=["bf16", "8bit"])
@pytest.mark.parametrize("N", [64, 1024, 1544, 12288])
@pytest.mark.parametrize("power", [40, 44, 50, 55])
def test_gradient_of_loud_rows(N, held, power):
    """Rows of 2^power, whose squares' sum is a number: the part along the row counts as much as the rest, with the gradient
    of the sum itself left out so that nothing hides it."""
    y, res, _, dz, w = norm_problem(2, 3, N, seed=power)
    loud = (res.float() * 2.0 ** power).to(BF)
    dz = (dz.float() + res.float()).to(BF)                               # along the row too
    check_gradient(y, loud, None, dz, w, held, 0.7, 1e-6)
    check_gradient((y.float() * 2.0 ** power).to(BF), loud, None, dz, (None, w[1], w[2]), held, 0.7, 1e-6)


@pytest.mark.parametrize("held", [False, True], ids=["bf16", "8bit"])
@pytest.mark.parametrize("N", [64, 1024, 1544, 12288])
@pytest.mark.parametrize("power", [20, 45, 50])
def test_gradient_of_quiet_rows(N, held, power):
    """Rows of 2^-power, without eps: only a row of zeros has no gradient."""
    y, res, dh, dz, w = norm_problem(2, 3, N, seed=power)
    quiet = (res.float() * 2.0 ** -power).to(BF)
    dz = (dz.float() + res.float()).to(BF)
    check_gradient(y, quiet, dh, dz, w, held, 0.7 * 2.0 ** -power, 0.0)
    check_gradient((y.float() * 2.0 ** -power).to(BF), quiet, dh, dz, (None, w[1], w[2]), held, 0.7, 0.0)


# ---------------------------------------------------------------- weight gradient: every power of two
@pytest.mark.parametrize("K", [64, 72])
def test_weight_gradient_of_every_exponent(K):
    """A token for every exponent, with every byte, alone in its column of dy: products with 1 are the held values
    themselves, among them those at the limit from which on they are widened in two steps (231 and 232)."""
    T = 248
    q = (torch.arange(T * K, device=DEV) % 255 - 127).to(torch.int8).view(1, T, K)
    e = torch.arange(1, T + 1, device=DEV).to(torch.uint8).view(1, T, 1).expand(1, T, -(-K // 32)).contiguous()
    dy = torch.eye(T, device=DEV).to(BF)[None]
    for first in (0, 230, 231):                                          # with all others, and in launches of their own
        some = slice(first, first + (T if first == 0 else 1))
        dw = torch.full((1, T, K), float("nan"), device=DEV)
        rc.gemm_wgrad(dy[:, some], (q[:, some].contiguous(), e[:, some].contiguous()), dw)
        want = ob.act8_values(q.cpu().numpy(), e.cpu().numpy())
        want[0, [t for t in range(T) if not some.start <= t < some.stop]] = 0
        assert np.array_equal(f64(dw), want)
