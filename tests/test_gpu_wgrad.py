"""GPU weight gradient from 8-bit activations against 64 bits (needs a GB300)."""
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


def problem(P, T, N, K, seed=0, share=""):
    """dy [P, T, N] and the pair of x [P, T, K]; what `share` names has one slot for all ranks."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    dy = torch.randn((1 if "y" in share else P, T, N), generator=g, device=DEV).to(BF)
    x = torch.randn((1 if "x" in share else P, T, K), generator=g, device=DEV) * torch.exp(torch.randn((1, T, 1), generator=g, device=DEV))
    x8 = rc.act8_pack(x.to(BF), rc.act8_empty(x.shape, DEV))
    return dy.expand(P, -1, -1), tuple(t.expand(P, -1, -1) for t in x8)


def values(x8):
    return ob.act8_values(*(t.cpu().numpy() for t in x8))


def check(dy, x8, dtype=BF, workspace=None):
    P, _, N = dy.shape
    dw = torch.full((P, N, x8[0].shape[2]), float("nan"), dtype=dtype, device=DEV)
    assert rc.gemm_wgrad(dy, x8, dw, workspace=workspace) is dw
    inside(dw, *ob.gemm_wgrad(f64(dy), values(x8), 2.0 ** -8 if dtype is BF else 2.0 ** -24))
    assert rc.ring_status() == 0
    return dw


SHAPES = [(1, 1, 8, 8), (1, 64, 256, 256), (1, 65, 264, 248), (2, 63, 128, 64), (1, 200, 520, 1000), (3, 129, 72, 200), (1, 1031, 520, 1000),
          (1, 640, 8, 2048), (2, 333, 1032, 40), (1, 4100, 256, 256), (8, 300, 96, 512)]


@pytest.mark.parametrize("dtype", [BF, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("P,T,N,K", SHAPES)
def test_shapes(P, T, N, K, dtype):
    check(*problem(P, T, N, K, seed=T), dtype)


@pytest.mark.parametrize("P,T,N,K", [(1, 8192, 512, 512), (5, 4096, 768, 1024), (1, 16000, 264, 272), (20, 2048, 512, 512), (10, 4096, 512, 1024)])
def test_tokens_divided_over_the_pairs(P, T, N, K):
    """Few tiles, or some left over after the last whole round, over many tokens: parts that reach over a
    tile's end, and as many parts as pairs."""
    dy, x8 = problem(P, T, N, K, seed=K)
    want = check(dy, x8, torch.float32)
    assert torch.equal(want, check(dy, x8, torch.float32))            # the same bits every time


@pytest.mark.parametrize("share", ["x", "y", "xy"])
def test_operands_of_all_ranks(share):
    check(*problem(4, 150, 136, 264, seed=1, share=share))


@pytest.mark.parametrize("dtype", [BF, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("T", [70, 8192])
def test_accumulates(dtype, T):
    dy, x8 = problem(1, T, 264, 520, seed=2)
    dw = torch.randn((1, 264, 520), device=DEV).to(dtype)
    old = f64(dw)
    rc.gemm_wgrad(dy, x8, dw, accumulate=True)
    u = 2.0 ** -8 if dtype is BF else 2.0 ** -24
    want, bound = ob.gemm_wgrad(f64(dy), values(x8), u)
    inside(dw, old + want, bound + (u + 2.0 ** -24) * (np.abs(old) + np.abs(want)))


def test_strided_views_leave_the_rest():
    P, T, N, K = 2, 140, 72, 136
    dy, (q, e) = problem(P, T, N, K, seed=3)
    want = check(dy, (q, e))
    wide = torch.zeros((T, P, 3 * N), dtype=BF, device=DEV).transpose(0, 1)
    wide[..., N:2 * N] = dy
    bytes_ = torch.zeros((T, P, K + 24), dtype=torch.int8, device=DEV).transpose(0, 1)
    bytes_[..., 8:8 + K] = q
    groups = torch.zeros((P, T, 9), dtype=torch.uint8, device=DEV)
    groups[..., 3:8] = e
    room = torch.full((P, N + 3, K + 8), 7.0, dtype=BF, device=DEV)
    rc.gemm_wgrad(wide[..., N:2 * N], (bytes_[..., 8:8 + K], groups[..., 3:8]), room[:, 1:N + 1, :K])
    assert torch.equal(room[:, 1:N + 1, :K], want)
    room[:, 1:N + 1, :K] = 7
    assert (room == 7).all()


@pytest.mark.parametrize("dtype", [BF, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("N,K", [(264, 256), (136, 520), (256, 776)])
def test_rows_of_dw_off_whole_sectors(N, K, dtype):
    """Whole and partial tiles whose rows start 16 bytes off a multiple of 32: all of them, none, or every other
    one; what lies between them stays as it was."""
    dy, x8 = problem(2, 70, N, K, seed=K)
    unit = 8 if dtype is BF else 4
    want, bound = ob.gemm_wgrad(f64(dy), values(x8), 2.0 ** -8 if dtype is BF else 2.0 ** -24)
    for shift, pad in ((0, unit), (unit, 2 * unit), (unit, unit), (0, 2 * unit)):
        room = torch.full((2, N, shift + K + pad), 7.0, dtype=dtype, device=DEV)
        dw = room[..., shift:shift + K]
        for turn in (1, 2):
            rc.gemm_wgrad(dy, x8, dw, accumulate=turn == 2)
            # twice: the first result's error, this sum's, the addition's in binary32 and the last rounding
            u = (2.0 ** -8 if dtype is BF else 2.0 ** -24) + 2.0 ** -24
            inside(dw, turn * want, bound if turn == 1 else 2 * bound + u * (2 * np.abs(want) + 2 * bound))
        room[..., shift:shift + K] = 7
        assert (room == 7).all()


def test_workspace_is_for_parts():
    assert rc.gemm_wgrad_workspace_bytes(1, 16384, 256, 512) > 256 and rc.gemm_wgrad_workspace_bytes(38, 16384, 256, 512) == 256
    assert rc.gemm_wgrad_workspace_bytes(1, 64, 256, 256) == 256 and rc.gemm_wgrad_workspace_bytes(1, 64, 257, 256) == 0


def test_no_tokens():
    dy = torch.empty((2, 0, 64), dtype=BF, device=DEV)
    x8 = rc.act8_empty((2, 0, 72), DEV)
    dw = torch.ones((2, 66, 80), device=DEV)
    rc.gemm_wgrad(dy, x8, dw[:, 1:65, :72], accumulate=True)
    assert (dw == 1).all()
    rc.gemm_wgrad(dy, x8, dw[:, 1:65, :72])
    assert (dw[:, 1:65, :72] == 0).all() and dw.sum() == 2 * (66 * 80 - 64 * 72)


def test_non_finite_values_reach_their_row_or_column_only():
    dy, x8 = problem(1, 100, 264, 264, seed=4)
    want = check(dy, x8)
    dy = dy.clone()
    dy[0, 99, 260] = float("inf")
    x8[1][0, 7, 3] = 255                                                # channels 96..127 of a token
    x8[0][0, 7, 96:128] = 0
    dw = torch.empty_like(want)
    rc.gemm_wgrad(dy, x8, dw)
    bad = torch.zeros_like(dw, dtype=torch.bool)
    bad[0, 260], bad[0, :, 96:128] = True, True
    assert torch.isnan(dw[0, :, 96:128]).all() and not torch.isfinite(dw[0, 260]).any() and torch.equal(dw[~bad], want[~bad])


def test_huge_and_tiny_groups():
    """Groups near both ends of the range: their values, products and sums are all numbers."""
    dy, (q, e) = problem(1, 96, 72, 136, seed=9)
    dy = (dy * 2.0 ** -20).contiguous()
    e[0, 5], e[0, 70], e[0, 71] = 240, 228, 231
    e[0, 30:40] = 2
    dw = check(dy, (q, e), torch.float32)
    assert torch.isfinite(dw).all() and dw.abs().max() > 1e30


@pytest.mark.parametrize("K", [200, 208])
def test_a_rank_does_not_reach_another(K):
    """Tokens come 64 at a time, the last of a rank with the next rank's first; marked groups there stay there."""
    dy, (q, e) = problem(3, 129, 136, K, seed=8)
    want = check(dy, (q, e))
    q[1], e[1] = 0, 255
    dy[2] = float("nan")
    dw = torch.empty_like(want)
    rc.gemm_wgrad(dy, (q, e), dw)
    assert torch.equal(dw[0], want[0]) and torch.isnan(dw[1:]).all()


@pytest.mark.parametrize("K,pad", [(72, 0), (72, 8), (80, 8), (256, 8), (264, 16), (1000, 0)])
def test_rows_of_every_alignment(K, pad):
    """Rows of bytes on 16-byte boundaries, every other on one, and neither; slots that follow one another or not."""
    P, T, N = 2, 131, 72
    dy, (q, e) = problem(P, T, N, K, seed=K)
    want = check(dy, (q, e))
    for gap in (0, 1):
        room = torch.full((P, T + gap, K + pad), 99, dtype=torch.int8, device=DEV)
        view = room[:, :T, :K]
        view.copy_(q)
        assert torch.equal(check(dy, (view, e)), want)
        flat = torch.full((room.numel() + 16,), 99, dtype=torch.int8, device=DEV)
        shifted = flat[8:].as_strided((P, T, K), room.stride())
        shifted.copy_(q)
        assert torch.equal(check(dy, (shifted, e)), want)


def test_workspace_streams_and_graph():
    P, T, N, K = 1, 6000, 512, 768
    a, b = problem(P, T, N, K, seed=5), problem(P, T, N, K, seed=6)
    want = [check(*x, torch.float32) for x in (a, b)]
    size = rc.gemm_wgrad_workspace_bytes(P, T, N, K)
    spaces = [torch.zeros(size, dtype=torch.uint8, device=DEV) for _ in range(2)]
    got = [torch.empty_like(want[0]) for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    for s, x, ws, dw in zip(streams, (a, b), spaces, got):              # two calls at once, a workspace each
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            for _ in range(3):
                rc.gemm_wgrad(*x, dw, workspace=ws)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(want, got))
    assert all((ws[256:] == 0).all() for ws in spaces) and rc.ring_status_ex(spaces[0]) == 0
    with pytest.raises(rc.RingError):
        rc.gemm_wgrad(*a, got[0], workspace=spaces[0][:-256])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        rc.gemm_wgrad(*a, got[0])
    a[0].copy_(b[0]), a[1][0].copy_(b[1][0]), a[1][1].copy_(b[1][1])
    check(*problem(2, 9000, 768, 1024, seed=7))                         # a call that may outgrow the library's space
    graph.replay()
    assert torch.equal(got[0], want[1])
