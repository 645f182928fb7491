"""GPU 8-bit activations, norms around the residual sum and gated activations against 64 bits (needs a GB300)."""
import numpy as np
import pytest
import torch

import ring_collectives_gb300 as rc
from oracle import block as ob

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
BF = torch.bfloat16
NAN = float("nan")


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


def rows(g, *shape, scale=1.0):
    """Rows of different sizes with a few loud channels."""
    x = torch.randn(shape, generator=g, device=DEV) * scale * torch.exp(torch.randn(shape[:-1] + (1,), generator=g, device=DEV))
    return (x * torch.where(torch.rand(shape[-1], generator=g, device=DEV) < 0.02, 16.0, 1.0)).to(BF)


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def same(pair, q, e):
    return np.array_equal(pair[0].cpu().numpy(), q) and np.array_equal(pair[1].cpu().numpy(), e)


def empty8(shape):
    q, e = rc.act8_empty(shape, DEV)
    return q.fill_(77), e.fill_(77)


# ---------------------------------------------------------------- 8 bits
@pytest.mark.parametrize("P,T,N", [(1, 1, 8), (1, 1, 32), (3, 5, 40), (2, 37, 1000), (1, 129, 248), (8, 64, 4096), (64, 3, 72), (1, 2, 65536)])
def test_act8_is_exact(P, T, N):
    x = rows(gen(N), P, T, N, scale=2.0 ** -3)
    x[..., ::7] *= 2.0 ** -9
    x8 = rc.act8_pack(x, empty8(x.shape))
    q, e = ob.act8_pack(f64(x))
    assert same(x8, q, e)
    assert np.array_equal(f64(rc.act8_unpack(x8, torch.empty_like(x))), ob.act8_values(q, e))


def test_act8_every_bf16_value():
    """All 65536 patterns, each a group of its own with zeros, and in one group with its neighbours."""
    bits = torch.arange(65536, dtype=torch.int32, device=DEV).to(torch.int16).view(BF)
    x = torch.zeros((1, 65536, 32), dtype=BF, device=DEV)
    x[0, torch.arange(65536), torch.arange(65536, device=DEV) % 32] = bits
    for x in (x, bits.view(1, 64, 1024)):
        x8 = rc.act8_pack(x, empty8(x.shape))
        q, e = ob.act8_pack(f64(x))
        assert same(x8, q, e)
        got, want = f64(rc.act8_unpack(x8, torch.empty_like(x))), ob.act8_values(q, e)
        assert np.array_equal(np.nan_to_num(got, nan=7e37), np.nan_to_num(want, nan=7e37))


def test_act8_every_byte_and_exponent():
    q = torch.arange(-127, 128, device=DEV).to(torch.int8).repeat(255)[None, None].expand(1, 1, -1)
    n = q.shape[-1] // 32 * 32
    q = q[..., :n].contiguous()
    e = (torch.arange(n // 32, device=DEV) * 113 % 248 + 1).to(torch.uint8)[None, None].contiguous()
    x = rc.act8_unpack((q, e), torch.empty((1, 1, n), dtype=BF, device=DEV))
    assert np.array_equal(f64(x), ob.act8_values(q.cpu().numpy(), e.cpu().numpy()))


def test_act8_views_leave_the_rest():
    P, T, N = 2, 19, 72
    x = rows(gen(1), P, T, 3 * N)
    q, e = torch.full((T, P, 4 * N), 5, dtype=torch.int8, device=DEV), torch.full((P, T, 11), 6, dtype=torch.uint8, device=DEV)
    part = x[..., N:2 * N]
    x8 = (q.transpose(0, 1)[..., N:2 * N], e[..., 3:6])
    rc.act8_pack(part, x8)
    assert same(x8, *ob.act8_pack(f64(part)))
    assert (q[..., :N] == 5).all() and (q[..., 2 * N:] == 5).all() and (e[..., :3] == 6).all() and (e[..., 6:] == 6).all()
    back = torch.full_like(x, 3.0)
    rc.act8_unpack(x8, back[..., :N])
    assert np.array_equal(f64(back[..., :N]), ob.act8_values(*ob.act8_pack(f64(part)))) and (back[..., N:] == 3).all()


# ---------------------------------------------------------------- norms around the residual sum
def problem(P, T, N, seed=0, post=True, gate=True, pre=True):
    g = gen(seed)
    w = [1 + 0.3 * torch.randn(N, generator=g, device=DEV) if on else None for on in (post, gate, pre)]
    dz = (torch.randn((P, T, N), generator=g, device=DEV) * 0.3).to(BF)
    return dict(y=rows(g, P, T, N), res=rows(g, P, T, N, scale=2.0), w=w, dh=(torch.randn((P, T, N), generator=g, device=DEV)).to(BF),
                dz=dz if pre else None)


def named(w, d=""):
    return dict(zip((d + "gamma_post", d + "gate", d + "gamma_pre"), w))


def cols(t, on):
    P, T, N = t.shape
    return t.view(P * T, P, N // P).transpose(0, 1).contiguous() if on else t


def w64(w):
    return [None if t is None else f64(t) for t in w]


def check_forward(p, in_cols=False, save=True, alpha=0.7, eps=1e-6):
    y, res = p["y"], p["res"]
    h = torch.full_like(res, NAN)
    z = h.clone() if p["w"][2] is not None else None
    y8, res8, z8 = (empty8(res.shape) if save else None for _ in range(3))
    rc.block_norm(cols(y, in_cols), res, h, z, **named(p["w"]), alpha=alpha, eps=eps, y8=y8, res8=res8, z8=z8 if z is not None else None)
    want, bound = ob.block_norm(f64(y), f64(res), *w64(p["w"]), alpha=alpha, eps=eps)
    inside(h, want[0], bound[0])
    if z is not None:
        inside(z, want[1], bound[1])
    if save:
        assert same(y8, *ob.act8_pack(f64(y))) and same(res8, *ob.act8_pack(f64(res)))
        assert z is None or same(z8, *ob.act8_pack(f64(z)))
    return h, z, y8, res8


def grads(p, in_cols=False):
    P, T, N = p["res"].shape
    dy = torch.full_like(cols(p["y"], in_cols), NAN)
    return dy, torch.full_like(p["res"], NAN), [None if t is None else torch.full((P, N), NAN, device=DEV) for t in p["w"]]


def check_gradient(p, in_cols=False, held=False, dh=True, alpha=0.7, eps=1e-6, workspace=None):
    y, res = p["y"], p["res"]
    P, T, N = res.shape
    dy, dres, dw = grads(p, in_cols)
    y8, res8 = (rc.act8_pack(t, rc.act8_empty(t.shape, DEV)) for t in (y, res)) if held else (cols(y, in_cols), res)
    dz = p["dz"] if p["dz"] is None else cols(p["dz"], in_cols)
    rc.block_norm_bwd(y8, res8, p["dh"] if dh else None, dz, dy, dres, **named(dw, "d"), **named(p["w"]), alpha=alpha, eps=eps,
                      workspace=workspace)
    at = [ob.act8_values(*ob.act8_pack(f64(t))) if held else f64(t) for t in (y, res)]
    dz = np.zeros(res.shape) if p["dz"] is None else f64(p["dz"])
    want, bound = ob.block_norm_bwd(*at, f64(p["dh"]) * dh, dz, *w64(p["w"]), alpha=alpha, eps=eps)
    got = {k: v for k, v in named(dw, "d").items() if v is not None} | {"dres": dres}
    assert set(want) == set(got) | {"dy"}
    inside(dy, ob.to_cols(want["dy"]) if in_cols else want["dy"], ob.to_cols(bound["dy"]) if in_cols else bound["dy"])
    for k, v in got.items():
        inside(v, want[k], bound[k])
    return dy, dres, dw


WIDTHS = [8, 16, 40, 64, 72, 128, 136, 248, 256, 264, 512, 520, 1000, 1032, 2048, 4096, 4104, 8192, 8200, 12288, 16384]


@pytest.mark.parametrize("N", WIDTHS)
def test_block_norm_widths(N):
    p = problem(2, 5, N, seed=N)
    check_forward(p)
    check_gradient(p)
    check_gradient(p, held=True)


@pytest.mark.parametrize("post,gate,pre", [(1, 0, 1), (0, 1, 1), (0, 0, 1), (1, 1, 0), (1, 0, 0), (0, 1, 0), (0, 0, 0)])
@pytest.mark.parametrize("N", [264, 9000])
def test_block_norm_parts(post, gate, pre, N):
    p = problem(3, 4, N, seed=3, post=post, gate=gate, pre=pre)
    check_forward(p)
    check_gradient(p)
    check_gradient(p, held=True)
    check_gradient(p, dh=False)


@pytest.mark.parametrize("P,T,N", [(1, 1, 64), (8, 1, 4096), (1, 1000, 512), (4, 777, 1024), (64, 7, 512), (2, 2500, 96), (8, 40, 8192)])
def test_block_norm_rows_and_column_chunks(P, T, N):
    p = problem(P, T, N, seed=T)
    a = check_forward(p, in_cols=True, save=False)
    b = check_forward(p, in_cols=False)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    x, u, du = check_gradient(p, in_cols=True)
    y, v, dv = check_gradient(p, in_cols=False)
    assert torch.equal(x, cols(y, True)) and torch.equal(u, v) and all(torch.equal(s, t) for s, t in zip(du, dv))
    check_gradient(p, in_cols=True, held=True)


def test_block_norm_small_and_zero_rows():
    p = problem(1, 6, 256, seed=2)
    p["y"][0, 0], p["res"][0, 0] = 0, 0
    p["y"][0, 1], p["res"][0, 2] = 0, 0
    p["y"][0, 3] *= 2.0 ** -30
    p["res"][0, 3] *= 2.0 ** -30
    check_forward(p, eps=1e-2)
    check_gradient(p, eps=1e-2)
    check_gradient(p, eps=1e-2, held=True)


@pytest.mark.parametrize("N", [24, 136, 328])
@pytest.mark.parametrize("T", [1, 3, 13])
def test_block_norm_few_rows_without_eps(N, T):
    """Warps that hold several rows, some of them past the last: with eps = 0 nothing of those may reach a sum."""
    p = problem(1, T, N, seed=T)
    check_forward(p, eps=0.0)
    check_gradient(p, eps=0.0)
    check_gradient(p, eps=0.0, held=True)


@pytest.mark.parametrize("N", [24, 136, 328, 1000])
def test_block_norm_rows_behind_a_marked_one(N):
    """A last row whose groups are marked as holding no numbers reaches its own results only, not the sums of
    rows that come after it in the same lanes and do not exist."""
    p = problem(1, 700, N, seed=N)
    clean = check_gradient(p, held=True)
    y8, res8 = (rc.act8_pack(p[k], rc.act8_empty(p[k].shape, DEV)) for k in ("y", "res"))
    dy, dres, dw = grads(p)
    for q, e in (y8, res8):
        q[0, 650:], e[0, 650:] = 0, 255
    p["dh"][0, 650:], p["dz"][0, 650:] = 0, 0
    rc.block_norm_bwd(y8, res8, p["dh"], p["dz"], dy, dres, **named(dw, "d"), **named(p["w"]), alpha=0.7)
    assert torch.equal(dy[0, :650], clean[0][0, :650]) and torch.isnan(dy[0, 650:]).all() and all(torch.isnan(t).all() for t in dw)


@pytest.mark.parametrize("N", [40, 264, 1000, 4104, 9000])
def test_block_norm_many_rows(N):
    """More rows than the GPU holds at once, so that blocks go round."""
    p = problem(2, 2600 if N < 4000 else 700, N, seed=N)
    check_forward(p)
    check_gradient(p, held=True)


@pytest.mark.parametrize("N", [1024, 12288])
def test_block_norm_rows_that_fill_their_threads(N):
    """Many rows of a width that needs no bounds, some of them zeros, tiny, or marked in one group."""
    p = problem(1, 400, N, seed=N)
    p["y"][0, 7], p["y"][0, 211] = 0, 0
    p["y"][0, 30] *= 2.0 ** -30
    p["y"][0, 31, 32:64] *= 2.0 ** -60
    clean = check_gradient(p, held=True, eps=1e-2)
    check_gradient(p, eps=1e-2)
    (q, e), res8 = (rc.act8_pack(p[k], rc.act8_empty(p[k].shape, DEV)) for k in ("y", "res"))
    q[0, 390, 64:96], e[0, 390, 2] = 0, 255
    dy, dres, dw = grads(p)
    rc.block_norm_bwd((q, e), res8, p["dh"], p["dz"], dy, dres, **named(dw, "d"), **named(p["w"]), alpha=0.7, eps=1e-2)
    keep = [i for i in range(400) if i != 390]
    assert torch.equal(dy[0, keep], clean[0][0, keep]) and torch.equal(dres[0, keep], clean[1][0, keep])
    assert torch.isnan(dy[0, 390]).all() and torch.isnan(dres[0, 390]).all() and all(torch.isnan(t).all() for t in dw)


def test_block_norm_without_rows():
    p = problem(3, 0, 64)
    _, _, dw = grads(p)
    e = torch.empty((3, 0, 64), dtype=BF, device=DEV)
    rc.block_norm(e, e, e.clone(), e.clone(), **named(p["w"]))
    rc.block_norm_bwd(e, e, None, e, e.clone(), e.clone(), **named(dw, "d"), **named(p["w"]))
    assert all((t == 0).all() for t in dw)


def test_block_norm_strided_views_in_place_and_gaps():
    P, T, N = 2, 33, 272
    p = problem(P, T, N, seed=6)
    h, z, _, _ = check_forward(p, alpha=1.0)
    dy, dres, dw = check_gradient(p, alpha=1.0)
    room = torch.full((T, P, 2 * N + 16), 9.0, dtype=BF, device=DEV)
    a, b = room.transpose(0, 1)[..., :N], room.transpose(0, 1)[..., N:2 * N]
    a.copy_(p["res"])
    rc.block_norm(p["y"], a, a, b, **named(p["w"]))                                    # h over res
    assert torch.equal(a, h) and torch.equal(b, z) and (room[..., 2 * N:] == 9).all()
    a.copy_(p["dh"]), b.copy_(p["dz"])
    dw2 = [torch.empty_like(t) for t in dw]
    rc.block_norm_bwd(p["y"], p["res"], a, b, b, a, **named(dw2, "d"), **named(p["w"]))  # dres over dh, dy over dz
    assert torch.equal(a, dres) and torch.equal(b, dy) and (room[..., 2 * N:] == 9).all()
    assert all(torch.equal(s, t) for s, t in zip(dw, dw2))
    both = cols(p["dz"], True)
    rc.block_norm_bwd(p["y"], p["res"], p["dh"], both, both, dres, **named(dw2, "d"), **named(p["w"]))   # dy over dz, in chunks
    assert torch.equal(both, cols(dy, True)) and torch.equal(a, dres)


def test_a_non_finite_row_stays_alone():
    p = problem(1, 9, 128, seed=7, gate=False)
    h, z, y8, res8 = check_forward(p)
    dy, dres, _ = check_gradient(p)
    p["y"][0, 4, 3], p["res"][0, 6, 5] = NAN, float("inf")
    h2, z2, dy2, dres2 = (torch.empty_like(h) for _ in range(4))
    dw = [None if t is None else torch.empty((1, 128), device=DEV) for t in p["w"]]
    q, e = empty8(h.shape)
    rc.block_norm(p["y"], p["res"], h2, z2, **named(p["w"]), alpha=0.7, y8=(q, e))
    rc.block_norm_bwd(p["y"], p["res"], p["dh"], p["dz"], dy2, dres2, **named(dw, "d"), **named(p["w"]), alpha=0.7)
    keep = [i for i in range(9) if i not in (4, 6)]
    assert torch.isnan(h2[0, 4]).all() and torch.isnan(z2[0, 4]).all() and torch.isnan(dy2[0, 4]).all() and torch.isnan(dres2[0, 6, 5])
    assert all(torch.equal(a[:, keep], b[:, keep]) for a, b in ((h, h2), (z, z2), (dy, dy2), (dres, dres2)))
    assert e[0, 4, 0] == 255 and (q[0, 4, :32] == 0).all() and torch.equal(q[0, 4, 32:], y8[0][0, 4, 32:])


def test_block_norm_same_bits_streams_workspace_and_graph():
    p = problem(4, 700, 1024, seed=8)
    P, T, N = p["res"].shape
    want = check_gradient(p, in_cols=True)
    ws = torch.zeros(rc.block_norm_bwd_workspace_bytes(P, T, N), dtype=torch.uint8, device=DEV)
    ws[:256] = 3
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = check_gradient(p, in_cols=True, workspace=ws)
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1]) and all(torch.equal(a, b) for a, b in zip(want[2], got[2]))
    assert (ws[:256] == 3).all() and (ws[256:] == 0).all()
    with pytest.raises(rc.RingError):
        check_gradient(p, in_cols=True, workspace=ws[:-256])
    # forward and gradient in one captured graph, replayed on other values
    y, h, z = cols(p["y"], True), torch.empty_like(p["res"]), torch.empty_like(p["res"])
    dy, dres, dw = grads(p, True)
    y8, res8 = (rc.act8_empty(h.shape, DEV) for _ in range(2))

    def step():
        rc.block_norm(y, p["res"], h, z, **named(p["w"]), alpha=0.7, y8=y8, res8=res8)
        rc.block_norm_bwd(y8, res8, p["dh"], p["dz"], dy, dres, **named(dw, "d"), **named(p["w"]), alpha=0.7)

    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    other = problem(4, 700, 1024, seed=9)
    y.copy_(cols(other["y"], True)), p["res"].copy_(other["res"]), p["dh"].copy_(other["dh"]), p["dz"].copy_(other["dz"])
    p["y"] = other["y"]
    graph.replay()
    want = check_gradient(p, in_cols=True, held=True)
    assert torch.equal(want[0], dy) and torch.equal(want[1], dres) and all(torch.equal(a, b) for a, b in zip(want[2], dw))


def test_block_norm_gradient_against_differences():
    """<gradient, v> against central differences of the 64-bit forward along v, for every argument."""
    p = problem(2, 3, 96, seed=10)
    dy, dres, dw = check_gradient(p, alpha=0.7, eps=1e-3)
    dh, dz, rng = f64(p["dh"]), f64(p["dz"]), np.random.default_rng(1)
    at = [f64(p["y"]), f64(p["res"]), *w64(p["w"])]
    _, off = ob.block_norm_bwd(*at[:2], dh, dz, *at[2:], alpha=0.7, eps=1e-3)
    names = ("dy", "dres", "dgamma_post", "dgate", "dgamma_pre")
    for i, g in enumerate((dy, dres, *dw)):
        v = rng.standard_normal(at[i].shape)
        ends = []
        for s in (1e-5, -1e-5):
            moved = list(at)
            moved[i] = at[i] + s * v
            (h, z), _ = ob.block_norm(*moved, alpha=0.7, eps=1e-3)
            ends.append((h * dh).sum() + (z * dz).sum())
        slope, room = (f64(g) * v).sum(), (off[names[i]] * np.abs(v)).sum()
        assert abs((ends[0] - ends[1]) / 2e-5 - slope) <= room + 1e-6 * np.abs(f64(g) * v).sum()


# ---------------------------------------------------------------- gated activations
KINDS = {"silu": rc.RC_GLU_SILU, "gelu": rc.RC_GLU_GELU}


def check_glu(a, b, dh, kind):
    h = torch.full(a.shape, NAN, dtype=BF, device=DEV)
    a8, b8, h8, g8 = (empty8(a.shape) for _ in range(4))
    rc.glu(a, b, h, act=KINDS[kind], a8=a8, b8=b8, h8=h8)
    inside(h, *ob.glu(f64(a), f64(b), kind))
    assert all(same(x8, *ob.act8_pack(f64(x))) for x8, x in ((a8, a), (b8, b), (h8, h)))
    for held in (False, True):
        da, db, h2 = (torch.full(a.shape, NAN, dtype=BF, device=DEV) for _ in range(3))
        rc.glu_bwd(a8 if held else a, b8 if held else b, dh, da, db, h=h2, act=KINDS[kind], h8=g8)
        at = [ob.act8_values(*ob.act8_pack(f64(x))) if held else f64(x) for x in (a, b)]
        want, bound = ob.glu_bwd(*at, f64(dh), kind)
        for x, w, o in zip((da, db, h2), want, bound):
            inside(x, w, o)
        assert same(g8, *ob.act8_pack(f64(h2)))
    return h, da, db


@pytest.mark.parametrize("kind", ["silu", "gelu"])
@pytest.mark.parametrize("P,T,N", [(1, 1, 8), (3, 7, 40), (1, 1031, 264), (8, 16, 1792), (64, 1, 72), (2, 300, 2752)])
def test_glu_shapes(P, T, N, kind):
    g = gen(N)
    check_glu(rows(g, P, T, N), rows(g, P, T, N), torch.randn((P, T, N), generator=g, device=DEV).to(BF), kind)


@pytest.mark.parametrize("kind", ["silu", "gelu"])
def test_glu_over_the_whole_range(kind):
    """Every finite bf16 gate whose square is finite, with factors of 1: tails, the far ends and zeros."""
    bits = torch.arange(65536, dtype=torch.int32, device=DEV).to(torch.int16).view(BF)
    a = bits[bits.abs() < 1e9]
    a = a[:a.numel() // 8 * 8][None, None]
    one = torch.ones_like(a)
    h, da, db = (torch.empty_like(a) for _ in range(3))
    rc.glu(a, one, h, act=KINDS[kind])
    inside(h, *ob.glu(f64(a), f64(one), kind))
    rc.glu_bwd(a, one, one, da, db, act=KINDS[kind])
    (wa, wb, _), (oa, obb, _) = ob.glu_bwd(f64(a), f64(one), f64(one), kind)
    inside(da, wa, oa)
    inside(db, wb, obb)


def test_glu_fused_halves_in_place_and_streams():
    P, T, N = 2, 45, 136
    g = gen(5)
    ab = rows(g, P, T, 2 * N + 8)
    dh = torch.randn((P, T, N), generator=g, device=DEV).to(BF)
    a, b = ab[..., :N], ab[..., N:2 * N]
    h, _, _ = check_glu(a.contiguous(), b.contiguous(), dh, "silu")
    da, db = torch.empty_like(dh), torch.empty_like(dh)
    rc.glu_bwd(a, b, dh, da, db)
    tail, keep = ab[..., 2 * N:].clone(), ab.clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        rc.glu(a, b, b)                                    # h over b
        out = b.clone()
        ab.copy_(keep)
        rc.glu_bwd(a, b, dh, a, b)                         # the gradient over the fused activations
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(out, h) and torch.equal(a, da) and torch.equal(b, db) and torch.equal(ab[..., 2 * N:], tail)


def test_glu_non_finite_values_stay_alone():
    g = gen(6)
    a, b = rows(g, 1, 3, 64), rows(g, 1, 3, 64)
    dh = torch.randn((1, 3, 64), generator=g, device=DEV).to(BF)
    h, da, db = (torch.empty_like(a) for _ in range(3))
    rc.glu(a, b, h)
    rc.glu_bwd(a, b, dh, da, db)
    a[0, 1, 5], a[0, 1, 6], b[0, 2, 7] = NAN, float("inf"), -float("inf")
    h2, da2, db2 = (torch.empty_like(a) for _ in range(3))
    rc.glu(a, b, h2)
    rc.glu_bwd(a, b, dh, da2, db2)
    spot = torch.zeros_like(a, dtype=torch.bool)
    spot[0, 1, 5] = spot[0, 1, 6] = spot[0, 2, 7] = True
    assert all(torch.equal(x[~spot], y[~spot]) for x, y in ((h, h2), (da, da2), (db, db2)))
    assert torch.isnan(h2[0, 1, 5]) and torch.isinf(h2[0, 1, 6]) and torch.isinf(h2[0, 2, 7]) and torch.isnan(da2[0, 1, 5])
