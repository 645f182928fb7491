"""GPU attention against its definition in 64 bits (needs a GB300).

Every element is held to the bound that oracle/attention.py derives for it
from the steps of a binary32 / bf16 evaluation; rows that see nothing,
lengths of zero and one, hidden non-finite values, cache tails, strided
operands, splits and group sizes that leave tile rows over are covered at
the sizes where a tile, a part or a sequence ends.
"""
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
    rc.ring_set_timeout_ms(2000)


def f64(t):
    return t.detach().double().cpu().numpy()


def rand(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV).to(BF)


def ints(x):
    return torch.tensor([int(v) for v in x], dtype=torch.int32, device=DEV)


def problem(ql, kl, P=1, Hq=4, Hkv=2, D=64, cap=0, seed=0, lead=0):
    """Packed operands (or a cache with `cap` rows a sequence), `lead` tokens before the first sequence."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    cu_q = np.cumsum([lead] + list(ql))
    cu_k = lead + cap * np.arange(len(kl) + 1) if cap else np.cumsum([lead] + list(kl))
    q = rand(g, P, int(cu_q[-1]), Hq, D)
    k, v = (rand(g, P, int(cu_k[-1]), Hkv, D) for _ in range(2))
    return dict(q=q, k=k, v=v, cu_q=cu_q, cu_k=cu_k, used=list(kl) if cap else None, g=g)


def forward(p, causal=True, scale=None, out=None, **kw):
    out = torch.full_like(p["q"], float("nan")) if out is None else out
    lse = torch.full(p["q"].shape[:3], float("nan"), device=DEV)
    rc.attn_fwd(p["q"], p["k"], p["v"], out, lse, ints(p["cu_q"]), ints(p["cu_k"]),
                used_k=None if p["used"] is None else ints(p["used"]), causal=causal, scale=scale, **kw)
    assert rc.ring_status() == 0, rc.ring_last_error()
    return out, lse


def seqs(p):
    return oa.sequences(p["cu_q"], p["cu_k"], p["used"])


def inside(got, want, bound, name):
    got = f64(got)
    assert np.array_equal(np.isnan(got), np.isnan(want)), name
    assert np.array_equal(np.isinf(got), np.isinf(want)), name
    fin = np.isfinite(want)
    assert np.array_equal(got[~fin & ~np.isnan(want)], want[~fin & ~np.isnan(want)]), name
    err = np.abs(got[fin] - want[fin])
    over = err > bound[fin]
    assert not over.any(), (name, int(over.sum()), float((err / bound[fin]).max()))


def check_forward(p, causal=True, scale=None):
    out, lse = forward(p, causal, scale)
    want = oa.attn_fwd(f64(p["q"]), f64(p["k"]), f64(p["v"]), seqs(p), causal, scale)
    inside(out, want[0], want[2], "out")
    inside(lse, want[1], want[3], "lse")
    return out, lse


def check_backward(p, causal=True, scale=None):
    out, lse = forward(p, causal, scale)
    do = rand(p["g"], *p["q"].shape)
    grads = [torch.full_like(x, float("nan")) for x in (p["q"], p["k"], p["v"])]
    rc.attn_bwd(p["q"], p["k"], p["v"], out, lse, do, *grads, ints(p["cu_q"]), ints(p["cu_k"]),
                used_k=None if p["used"] is None else ints(p["used"]), causal=causal, scale=scale)
    assert rc.ring_status() == 0, rc.ring_last_error()
    want, bound = oa.attn_bwd(*(f64(p[n]) for n in "qkv"), f64(out), f64(lse), f64(do), seqs(p), causal, scale)
    for n, a, b, c in zip(("dq", "dk", "dv"), grads, want, bound):
        inside(a, b, c, n)
    return grads


LENGTHS = [([1], [1]), ([128], [128]), ([129, 127], [129, 127]), ([0, 5, 0, 260], [0, 5, 0, 260]), ([300], [300]),
           ([64, 3], [400, 130]), ([40, 200], [17, 0]), ([0, 0], [3, 0]), ([1, 1, 1], [1, 128, 129])]
HEADS = [(1, 1, 64), (4, 2, 128), (6, 2, 80), (5, 1, 8), (7, 1, 120), (8, 8, 40), (16, 1, 96)]


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("lengths", LENGTHS, ids=str)
def test_lengths(lengths, causal):
    p = problem(*lengths, Hq=4, Hkv=2, D=64)
    check_forward(p, causal)
    check_backward(p, causal)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("Hq,Hkv,D", HEADS)
def test_heads(Hq, Hkv, D, causal):
    p = problem([70, 1, 133], [70, 140, 133], P=2, Hq=Hq, Hkv=Hkv, D=D, seed=2)
    check_forward(p, causal)
    check_backward(p, causal)


@pytest.mark.parametrize("Hq,Hkv,D", [(128, 1, 64), (100, 1, 16), (64, 1, 128)])
def test_large_groups(Hq, Hkv, D):
    p = problem([3, 1], [130, 70], Hq=Hq, Hkv=Hkv, D=D, seed=3)
    check_forward(p)
    check_backward(p)


@pytest.mark.parametrize("scale", [0.02, 1.0, 3.0])
def test_scales(scale):
    """Large scales move the running maximum often; small ones make weights nearly equal."""
    p = problem([200, 30], [200, 333], D=128, seed=4)
    check_forward(p, scale=scale)
    check_backward(p, scale=scale)


def test_growing_scores_move_the_maximum():
    """Every key tile has larger scores than all before it, so the accumulator is rescaled each time."""
    p = problem([4], [1030], Hq=2, Hkv=1, D=64, seed=5)
    p["k"] *= torch.linspace(0.1, 6.0, 1030, device=DEV)[None, :, None, None].to(BF)
    p["q"] = p["q"].abs()
    p["k"] = p["k"].abs()
    check_forward(p, scale=0.2)
    p2 = problem([700], [700], Hq=1, Hkv=1, D=128, seed=6)
    p2["q"], p2["k"] = p2["q"].abs(), p2["k"].abs() * torch.linspace(0.1, 4.0, 700, device=DEV)[None, :, None, None].to(BF)
    check_forward(p2, scale=0.1)


@pytest.mark.parametrize("P,kl,Hq,Hkv,D", [(2, [1, 5000, 129, 2000], 4, 1, 128), (1, [3001] * 3, 8, 8, 64), (8, [9000], 4, 1, 128),
                                           (1, [255, 256, 257], 6, 2, 72), (1, [700] * 160, 4, 4, 64)])
def test_single_tokens_against_a_cache(P, kl, Hq, Hkv, D):
    """One token a sequence; rows of the cache past the used ones hold NaN."""
    p = problem([1] * len(kl), kl, P=P, Hq=Hq, Hkv=Hkv, D=D, cap=max(kl) + 37, seed=7)
    for b, n in enumerate(kl):
        end = int(p["cu_k"][b + 1])
        p["k"][:, end - (max(kl) + 37 - n):end] = float("nan")
        p["v"][:, end - (max(kl) + 37 - n):end] = float("inf")
    check_forward(p)


@pytest.mark.parametrize("ql,kl,D", [([100, 3], [1500, 2900], 96), ([33], [4000], 128), ([65, 1, 64], [1025, 2048, 640], 64)])
def test_later_pieces_split_over_blocks(ql, kl, D):
    p = problem(ql, kl, P=1, Hq=8, Hkv=2, D=D, cap=max(kl), seed=8)
    check_forward(p)
    check_backward(p)


def test_mixed_prompt_and_tokens():
    p = problem([1, 500, 1, 1, 20], [900, 500, 1, 77, 20], Hq=4, Hkv=2, D=128, seed=9)
    check_forward(p)
    check_backward(p)


def test_hidden_values_do_not_reach_a_row():
    """Keys and values that the causal mask hides hold NaN and infinities: rows that do not
    see them are what they are without, rows that do are not finite (column by column)."""
    p = problem([300, 200], [300, 200], Hq=4, Hkv=2, D=64, seed=10)
    clean, _ = check_forward(p)
    p["v"][0, 140, 0, 3] = float("inf")
    p["v"][0, 141, 1, 5] = float("nan")
    p["v"][0, 299, 0, 7] = float("-inf")
    p["v"][0, 400, 1, 9] = float("nan")
    out, _ = check_forward(p)
    assert torch.equal(out[0, :140], clean[0, :140]) and torch.isinf(out[0, 140, 0, 3])
    p["k"][0, 250] = float("nan")
    out, _ = check_forward(p)
    assert torch.equal(out[0, :140], clean[0, :140]) and torch.isnan(out[0, 250:300]).all()


def test_neighbours_do_not_reach_a_sequence():
    """Everything outside the second sequence is not finite, forward and backward."""
    for D in (64, 128):
        p = problem([90, 77, 60], [90, 203, 60], Hq=6, Hkv=2, D=D, seed=11, lead=5)
        keep = {n: p[n].clone() for n in "qkv"}
        for causal in (True, False):
            for n, cu in (("q", p["cu_q"]), ("k", p["cu_k"]), ("v", p["cu_k"])):
                p[n] = torch.full_like(keep[n], float("nan"))
                p[n][:, cu[1]:cu[2]] = keep[n][:, cu[1]:cu[2]]
            only = dict(p, cu_q=p["cu_q"][1:3], cu_k=p["cu_k"][1:3])
            check_forward(only, causal)
            out, lse = forward(only, causal)
            do = torch.full_like(p["q"], float("nan"))
            do[:, p["cu_q"][1]:p["cu_q"][2]] = 1.0
            grads = [torch.zeros_like(p[n]) for n in "qkv"]
            rc.attn_bwd(p["q"], p["k"], p["v"], out, lse, do, *grads, ints(only["cu_q"]), ints(only["cu_k"]), causal=causal)
            assert rc.ring_status() == 0
            assert all(torch.isfinite(x).all() for x in grads)
            for x, cu in zip(grads, (p["cu_q"], p["cu_k"], p["cu_k"])):   # untouched outside
                assert (x[:, :cu[1]] == 0).all() and (x[:, cu[2]:] == 0).all() and (x[:, cu[1]:cu[2]] != 0).any()


def test_fused_layouts_and_untouched_gaps():
    """Operands inside a fused projection output, the result in a layout of its own, gradients
    into one fused buffer: nothing between the heads is written."""
    P, T, Hq, Hkv, D = 2, 150, 4, 2, 64
    g = torch.Generator(device=DEV).manual_seed(12)
    fused = rand(g, T, P, Hq + 2 * Hkv, D)

    def views(x):
        y = x.transpose(0, 1)
        return y[:, :, :Hq], y[:, :, Hq:Hq + Hkv], y[:, :, Hq + Hkv:]

    q, k, v = views(fused)
    p = dict(q=q, k=k, v=v, cu_q=np.array([0, 37, 150]), cu_k=np.array([0, 37, 150]), used=None, g=g)
    room = torch.full((P, T, Hq + 1, D + 16), 7.0, dtype=BF, device=DEV)
    out, lse = forward(p, out=room[:, :, :Hq, :D])
    want = oa.attn_fwd(f64(q), f64(k), f64(v), seqs(p))
    inside(out, want[0], want[2], "out")
    assert (room[:, :, Hq] == 7).all() and (room[..., D:] == 7).all()
    do = rand(g, P, T, Hq, D)
    grad = torch.full_like(fused, 3.0)
    rc.attn_bwd(q, k, v, out, lse, do, *views(grad), ints(p["cu_q"]), ints(p["cu_k"]))
    plain = [torch.empty_like(x, memory_format=torch.contiguous_format) for x in (q, k, v)]
    rc.attn_bwd(q.contiguous(), k.contiguous(), v.contiguous(), out.contiguous(), lse, do, *plain, ints(p["cu_q"]), ints(p["cu_k"]))
    assert rc.ring_status() == 0
    assert all(torch.equal(a, b) for a, b in zip(views(grad), plain))


def test_the_same_call_gives_the_same_bits():
    for ql, kl in (([300, 513], [300, 513]), ([1, 1], [4000, 777]), ([40], [3000])):
        p = problem(ql, kl, P=2, Hq=8, Hkv=2, D=128, seed=13)
        first = forward(p)
        do = rand(p["g"], *p["q"].shape)

        def grads():
            out = [torch.empty_like(x) for x in (p["q"], p["k"], p["v"])]
            rc.attn_bwd(p["q"], p["k"], p["v"], *first, do, *out, ints(p["cu_q"]), ints(p["cu_k"]))
            return out
        g0 = grads()
        for _ in range(5):
            assert all(torch.equal(a, b) for a, b in zip(first, forward(p)))
            assert all(torch.equal(a, b) for a, b in zip(g0, grads()))


def test_batching_does_not_change_a_prompt():
    p = problem([200, 77, 300], [200, 77, 300], Hq=4, Hkv=2, D=128, seed=14)
    out, lse = forward(p)
    for b in range(3):
        s = slice(int(p["cu_q"][b]), int(p["cu_q"][b + 1]))
        one = dict(p, q=p["q"][:, s].contiguous(), k=p["k"][:, s].contiguous(), v=p["v"][:, s].contiguous(),
                   cu_q=np.array([0, s.stop - s.start]), cu_k=np.array([0, s.stop - s.start]))
        o1, l1 = forward(one)
        assert torch.equal(o1, out[:, s]) and torch.equal(l1, lse[:, s])


def test_cache_beyond_32_bit_offsets():
    """A cache of over 2^32 bytes whose sequence lies at its end."""
    T, n = (1 << 22) + 5000, 700
    k = torch.zeros((1, T, 4, 128), dtype=BF, device=DEV)
    v = torch.zeros((1, T, 4, 128), dtype=BF, device=DEV)
    assert k.numel() * 2 > 1 << 32
    g = torch.Generator(device=DEV).manual_seed(15)
    k[:, T - n:], v[:, T - n:] = rand(g, 1, n, 4, 128), rand(g, 1, n, 4, 128)
    for m in (1, n):
        q = rand(g, 1, m, 8, 128)
        p = dict(q=q, k=k, v=v, cu_q=np.array([0, m]), cu_k=np.array([T - n, T]), used=None, g=g)
        out, lse = forward(p)
        small = dict(p, k=k[:, T - n:].contiguous(), v=v[:, T - n:].contiguous(), cu_k=np.array([0, n]))
        a, b = forward(small)
        assert torch.equal(out, a) and torch.equal(lse, b)
    do = rand(g, *q.shape)
    dk, dv = torch.zeros_like(k), torch.zeros_like(v)
    rc.attn_bwd(q, k, v, out, lse, do, torch.empty_like(q), dk, dv, ints([0, n]), ints([T - n, T]))
    sk, sv = torch.empty_like(small["k"]), torch.empty_like(small["v"])
    rc.attn_bwd(q, small["k"], small["v"], out, lse, do, torch.empty_like(q), sk, sv, ints([0, n]), ints([0, n]))
    assert rc.ring_status() == 0
    assert torch.equal(dk[:, T - n:], sk) and torch.equal(dv[:, T - n:], sv)


def test_offsets_outside_the_tensors_are_clamped():
    p = problem([100], [100], seed=16)
    out, lse = forward(p)
    wild = dict(p, cu_q=np.array([-5, 1 << 30]), cu_k=np.array([0, 1 << 30]), used=[1 << 30])
    a, b = forward(wild)
    assert torch.equal(a, out) and torch.equal(b, lse)


@pytest.mark.parametrize("B, tokens, keys", [(599, 1, 16500), (9, 128, 9000), (75, 5, 4097)])
def test_decreasing_offsets_stay_inside_the_workspace(B, tokens, keys):
    """Offsets that go back and forth give every other sequence all tokens: more units than
    disjoint sequences could have.  The call writes nothing past its workspace, and equal
    sequences write equal rows."""
    p = problem([tokens], [keys], P=1, Hq=2, Hkv=1, D=64, seed=23)
    want, wlse, ob, lb = oa.attn_fwd(f64(p["q"]), f64(p["k"]), f64(p["v"]), seqs(p))
    size = rc.attn_fwd_workspace_bytes(1, B, tokens, keys, 2, 1, 64)
    space = torch.full((size + 4096,), 0x5A, dtype=torch.uint8, device=DEV)
    space[:size] = 0
    back = dict(p, cu_q=[tokens * (b & 1) for b in range(B + 1)], cu_k=[keys * (b & 1) for b in range(B + 1)])
    out, lse = forward(back, workspace=space[:size])
    assert rc.ring_status_ex(space) == 0
    assert bool((space[size:] == 0x5A).all())
    inside(out, want, ob, "out")
    inside(lse, wlse, lb, "lse")


def test_streams_and_workspaces():
    """Calls with their own workspaces on two streams, tensors made on the default stream."""
    ps = [problem([1] * 5, [3000, 20, 900, 1, 4000], P=2, Hq=8, Hkv=2, D=128, seed=s) for s in (17, 18)]
    want = [forward(p) for p in ps]
    streams = [torch.cuda.Stream() for _ in ps]
    P, T, Hq, D = ps[0]["q"].shape
    size = rc.attn_fwd_workspace_bytes(P, 5, T, ps[0]["k"].size(1), Hq, 2, D)
    spaces = [torch.zeros(size, dtype=torch.uint8, device=DEV) for _ in ps]
    args = [(ints(p["cu_q"]), ints(p["cu_k"]), torch.empty_like(p["q"]), torch.empty(p["q"].shape[:3], device=DEV)) for p in ps]
    torch.cuda.synchronize()
    for _ in range(20):
        for p, s, w, (cq, ck, out, lse) in zip(ps, streams, spaces, args):
            rc.attn_fwd(p["q"], p["k"], p["v"], out, lse, cq, ck, workspace=w, stream=s)
    for s, w, (_, _, out, lse), (a, b) in zip(streams, spaces, args, want):
        assert rc.ring_status_ex(w, s) == 0
        assert torch.equal(out, a) and torch.equal(lse, b)
    with pytest.raises(rc.RingError):
        rc.attn_fwd(ps[0]["q"], ps[0]["k"], ps[0]["v"], args[0][2], None, args[0][0], args[0][1], workspace=spaces[0][:1024])
    with torch.cuda.stream(streams[0]):
        o2, _ = forward(ps[0])
    assert torch.equal(o2, want[0][0])


def test_graph_replay_follows_the_lengths():
    """A captured call reads lengths and offsets when it runs."""
    p = problem([1, 1, 1], [600, 600, 600], Hq=4, Hkv=1, D=64, cap=600, seed=19)
    used, cu_q, cu_k = ints([600, 1, 300]), ints(p["cu_q"]), ints(p["cu_k"])
    out, lse = torch.empty_like(p["q"]), torch.empty(p["q"].shape[:3], device=DEV)
    call = lambda: rc.attn_fwd(p["q"], p["k"], p["v"], out, lse, cu_q, cu_k, used_k=used)  # noqa: E731
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for lens in ([600, 1, 300], [5, 599, 0], [128, 129, 127]):
        used.copy_(ints(lens))
        graph.replay()
        torch.cuda.synchronize()
        want = oa.attn_fwd(f64(p["q"]), f64(p["k"]), f64(p["v"]), oa.sequences(p["cu_q"], p["cu_k"], lens))
        inside(out, want[0], want[2], "out")
        inside(lse, want[1], want[3], "lse")


def test_gradients_against_differences():
    """The directional derivative of sum(out * do) along random directions, from 64-bit
    differences of the definition at the kernel's own bf16 inputs, against the inner
    product with the kernel's gradients; its error is bounded by the gradients' bounds."""
    p = problem([65, 20], [65, 150], Hq=4, Hkv=2, D=64, seed=20)
    out, lse = forward(p)
    do = rand(p["g"], *p["q"].shape)
    grads = [torch.empty_like(p[n]) for n in "qkv"]
    rc.attn_bwd(p["q"], p["k"], p["v"], out, lse, do, *grads, ints(p["cu_q"]), ints(p["cu_k"]))
    assert rc.ring_status() == 0
    x, d = {n: f64(p[n]) for n in "qkv"}, f64(do)
    _, bounds = oa.attn_bwd(x["q"], x["k"], x["v"], f64(out), f64(lse), d, seqs(p))
    # delta uses the rounded output: |o - out| is within the forward bound
    _, _, ob, _ = oa.attn_fwd(x["q"], x["k"], x["v"], seqs(p))
    rng = np.random.default_rng(0)
    f = lambda y: (oa.attn_fwd(y["q"], y["k"], y["v"], seqs(p))[0] * d).sum()  # noqa: E731
    for n, g, b in zip("qkv", grads, bounds):
        t = rng.standard_normal(x[n].shape)
        h = 1e-5
        want = (f(dict(x, **{n: x[n] + h * t})) - f(dict(x, **{n: x[n] - h * t}))) / (2 * h)
        extra = 0.0 if n == "v" else 65 * 0.125 * np.abs(ob * d).sum() * np.abs(t).max() * 6   # delta's share: p |d delta| scale |k or q| |t|
        assert abs((f64(g) * t).sum() - want) <= (b * np.abs(t)).sum() + extra + 1e-6 * abs(want)


def test_binding_refuses_what_does_not_fit():
    p = problem([4], [4])
    cu = ints([0, 4])
    out, lse = torch.empty_like(p["q"]), torch.empty(p["q"].shape[:3], device=DEV)
    with pytest.raises(TypeError):
        rc.attn_fwd(p["q"].float(), p["k"], p["v"], out, lse, cu, cu)
    with pytest.raises(TypeError):
        rc.attn_fwd(p["q"].cpu(), p["k"], p["v"], out, lse, cu, cu)
    with pytest.raises(ValueError):
        rc.attn_fwd(p["q"], p["k"], p["v"][:, :3], out, lse, cu, cu)
    with pytest.raises(ValueError):
        rc.attn_fwd(p["q"], p["k"], p["v"], out.transpose(2, 3).contiguous().transpose(2, 3), lse, cu, cu)
    with pytest.raises(TypeError):
        rc.attn_fwd(p["q"], p["k"], p["v"], out, lse[:, :2], cu, cu)
    with pytest.raises(TypeError):
        rc.attn_fwd(p["q"], p["k"], p["v"], out, lse, cu, cu.long())
    with pytest.raises(rc.RingError):
        rc.attn_fwd(p["q"], p["k"], p["v"], p["q"], lse, cu, cu)
    assert rc.attn_fwd(p["q"], p["k"], p["v"], out, None, cu, cu) is out
    assert rc.ring_status() == 0
