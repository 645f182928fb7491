"""GPU block operators as programs call them: captured graphs, several streams, a training step replayed, slots far
apart, wide rows under a time bound (needs a GB300)."""
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


class Step:
    """glu, its weight gradient and its own gradient between two norms, on buffers of its own."""

    def __init__(self, seed, P=2, T=300, N=384, ws=False):
        self.P, self.T, self.N = P, T, N
        self.y, self.res, self.dz = rand(seed, P, P * T, N // P), rand(seed + 1, P, T, N), rand(seed + 2, P, T, N)
        self.h, self.z, self.a, self.da, self.db, self.dy, self.dres = (torch.empty_like(self.res) for _ in range(7))
        self.y8, self.res8, self.a8, self.b8, self.g8 = (rc.act8_empty(self.res.shape, DEV) for _ in range(5))
        self.w = [torch.rand(N, generator=torch.Generator(device=DEV).manual_seed(seed + 3), device=DEV) + 0.5 for _ in range(3)]
        self.dw = [torch.empty((P, N), device=DEV) for _ in range(3)]
        self.wg = torch.empty((P, N, N), device=DEV)
        self.ws = torch.zeros(max(rc.block_norm_bwd_workspace_bytes(P, T, N, held=True), rc.gemm_wgrad_workspace_bytes(P, T, N, N)),
                              dtype=torch.uint8, device=DEV) if ws else None

    def run(self):
        w = dict(zip(("gamma_post", "gate", "gamma_pre"), self.w))
        rc.block_norm(self.y, self.res, self.h, self.z, **w, y8=self.y8, res8=self.res8)
        rc.glu(self.h, self.z, self.a, a8=self.a8, b8=self.b8, h8=self.g8)
        rc.gemm_wgrad(self.dz, self.g8, self.wg, workspace=self.ws)
        rc.glu_bwd(self.a8, self.b8, self.dz, self.da, self.db)
        rc.block_norm_bwd(self.y8, self.res8, self.da, self.db, self.dy, self.dres, *self.dw, **w, workspace=self.ws)
        return [t.clone() for t in (self.h, self.z, self.a, self.wg, self.da, self.db, self.dy, self.dres, *self.dw)]


def test_a_step_is_what_its_definitions_say():
    s = Step(1)
    h, z, a, wg, da, db, dy, dres, *dw = s.run()
    w = [f64(t) for t in s.w]
    want, bound = ob.block_norm(ob.from_cols(f64(s.y), s.T), f64(s.res), *w)
    inside(h, want[0], bound[0])
    inside(z, want[1], bound[1])
    inside(a, *ob.glu(f64(h), f64(z), "silu"))
    inside(wg, *ob.gemm_wgrad(f64(s.dz), ob.act8_values(*ob.act8_pack(f64(a))), 2.0 ** -24))
    held = [ob.act8_values(*ob.act8_pack(f64(t))) for t in (h, z)]
    (wa, wb, _), (ba, bb, _) = ob.glu_bwd(*held, f64(s.dz), "silu")
    inside(da, wa, ba)
    inside(db, wb, bb)
    held = [ob.act8_values(*ob.act8_pack(t)) for t in (ob.from_cols(f64(s.y), s.T), f64(s.res))]
    want, bound = ob.block_norm_bwd(*held, f64(da), f64(db), *w)
    for name, t in zip(("dy", "dres", "dgamma_post", "dgate", "dgamma_pre"), (dy, dres, *dw)):
        inside(t, want[name], bound[name])


def test_a_step_captured_and_replayed_on_other_values():
    s, other = Step(5), Step(9)
    want = [s.run(), other.run()]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.run()
    for name in ("y", "res", "dz"):
        getattr(s, name).copy_(getattr(other, name))
    for a, b in zip(s.w, other.w):
        a.copy_(b)
    Step(3, P=4, T=900, N=1024).run()                     # a larger call in between
    graph.replay()
    got = [s.h, s.z, s.a, s.wg, s.da, s.db, s.dy, s.dres, *s.dw]
    assert all(torch.equal(a, b) for a, b in zip(want[1], got)) and not torch.equal(want[0][0], want[1][0])


def test_two_steps_at_once_on_two_streams():
    steps = [Step(11, ws=True), Step(17, ws=True)]
    want = [s.run() for s in steps]
    streams = [torch.cuda.Stream() for _ in steps]
    got = [None, None]
    for k, (s, st) in enumerate(zip(steps, streams)):
        st.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(st):
            for _ in range(4):
                got[k] = s.run()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for x, y in zip(want, got) for a, b in zip(x, y))
    assert all((s.ws[256:] == 0).all() and rc.ring_status_ex(s.ws) == 0 for s in steps)


def test_slots_far_apart():
    """Slots 5 GB apart: no offset is kept in 32 bits."""
    P, T, N, far = 2, 40, 264, (5 << 30) // 2
    room = torch.empty(far + T * N * 4, dtype=BF, device=DEV)
    near = rand(1, P, T, N), rand(2, P, T, N)
    a, b = (room[k * T * N:].as_strided((P, T, N), (far, N, 1)) for k in (0, 1))
    a.copy_(near[0]), b.copy_(near[1])
    out, want = (room[2 * T * N:].as_strided((P, T, N), (far, N, 1)) for _ in range(2))
    bytes_ = torch.empty((5 << 30) + T * N, dtype=torch.int8, device=DEV)
    q, e = bytes_.as_strided((P, T, N), (5 << 30, N, 1)), torch.empty((P, T, 9), dtype=torch.uint8, device=DEV)
    rc.act8_pack(a, (q, e))
    assert np.array_equal(q.cpu().numpy(), ob.act8_pack(f64(near[0]))[0])
    rc.glu(a, b, out)
    inside(out, *ob.glu(f64(near[0]), f64(near[1]), "silu"))
    rc.block_norm(a, b, out, None)
    inside(out, *(x[0] for x in ob.block_norm(f64(near[0]), f64(near[1]))))
    dw = torch.empty((P, N, N), dtype=BF, device=DEV)
    rc.gemm_wgrad(b, (q, e), dw)
    inside(dw, *ob.gemm_wgrad(f64(near[1]), ob.act8_values(q.cpu().numpy(), e.cpu().numpy())))
    dy = room[3 * T * N:].as_strided((P, T, N), (far, N, 1))
    rc.block_norm_bwd(a, b, b, None, dy, out)
    assert torch.equal(dy.cpu(), near[1].cpu()) and torch.equal(out.cpu(), near[1].cpu())


def test_many_elements():
    """More than 2^31 elements: the last rows are packed and unpacked like the first."""
    T, N = 40000, 57344
    x = torch.zeros((1, T, N), dtype=BF, device=DEV)
    some = rand(3, 64, N)
    x[0, :64], x[0, -64:] = some, some
    x8 = rc.act8_pack(x, rc.act8_empty(x.shape, DEV))
    q, e = ob.act8_pack(f64(some)[None])
    for rows in (slice(0, 64), slice(T - 64, T)):
        assert np.array_equal(x8[0][0, rows].cpu().numpy(), q[0]) and np.array_equal(x8[1][0, rows].cpu().numpy(), e[0])
    rc.act8_unpack(x8, x)
    assert np.array_equal(f64(x[0, -64:]), ob.act8_values(q, e)[0])


def test_wide_rows_leave_no_status():
    p = rand(1, 2, 300, 16384), rand(2, 2, 300, 16384)
    g = torch.ones(16384, device=DEV)
    h, z, dy, dres = (torch.empty_like(p[0]) for _ in range(4))
    dg = torch.empty((2, 16384), device=DEV)
    for _ in range(5):
        rc.block_norm(*p, h, z, gamma_post=g, gamma_pre=g)
        rc.block_norm_bwd(*p, h, z, dy, dres, dg, None, dg.clone(), gamma_post=g, gamma_pre=g)
    assert rc.ring_status() == 0


def test_devices_and_types_are_checked():
    x, x8 = rand(1, 1, 4, 64), rc.act8_empty((1, 4, 64), DEV)
    for bad in (lambda: rc.act8_pack(x.cpu(), x8), lambda: rc.act8_pack(x.float(), x8), lambda: rc.act8_pack(x, (x8[0].cpu(), x8[1])),
                lambda: rc.act8_pack(x, x8[::-1]), lambda: rc.glu(x, x.cpu(), x.clone()), lambda: rc.block_norm(x, x, x.float()),
                lambda: rc.block_norm_bwd(x8, x, x, None, x.clone(), x.clone()), lambda: rc.gemm_wgrad(x, x8, torch.empty((1, 64, 64), device=DEV).half()),
                lambda: rc.block_norm(x, x, x.clone(), gate=torch.ones(64)), lambda: rc.act8_pack(x, None)):
        with pytest.raises((TypeError, KeyError)):
            bad()
    for bad in (lambda: rc.act8_pack(x, rc.act8_empty((1, 4, 72), DEV)), lambda: rc.glu(x, x[:, :3], x.clone()),
                lambda: rc.gemm_wgrad(x[:, :3], x8, torch.empty((1, 64, 64), device=DEV)), lambda: rc.block_norm(x, x.transpose(1, 2), x.clone())):
        with pytest.raises((ValueError, TypeError)):
            bad()
