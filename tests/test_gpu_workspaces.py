"""One caller-owned workspace shared by different calls in stream order (needs a GB300).

The signalling calls keep words after the 128-byte header that compare with
the header's epoch, so whatever other calls put there has to be gone when they
return: zero is a word that no launch has signalled yet.
"""
import numpy as np
import pytest
import torch

import ring_collectives_gb300 as rc

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
BF = torch.bfloat16
HEADER = 128


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(DEV)
    rc.ring_set_timeout_ms(2000)


def ints(x):
    return torch.tensor([int(v) for v in x], dtype=torch.int32, device=DEV)


class Attention:
    """One attention problem, forward and backward, on the library's workspace or a caller's."""

    def __init__(self, ql, kl, P, Hq, Hkv, D, seed):
        g = torch.Generator(device=DEV).manual_seed(seed)
        r = lambda T, H: torch.randn(P, T, H, D, generator=g, device=DEV).to(BF)  # noqa: E731
        self.q, self.dout = r(sum(ql), Hq), r(sum(ql), Hq)
        self.k, self.v = r(sum(kl), Hkv), r(sum(kl), Hkv)
        self.cu = ints(np.cumsum([0] + ql)), ints(np.cumsum([0] + kl))
        self.sizes = P, len(ql), sum(ql), sum(kl), Hq, Hkv, D

    def forward(self, ws=None):
        out, lse = torch.empty_like(self.q), torch.empty(self.q.shape[:3], device=DEV)
        rc.attn_fwd(self.q, self.k, self.v, out, lse, *self.cu, workspace=ws)
        return out, lse

    def backward(self, out, lse, ws=None):
        grads = [torch.empty_like(x) for x in (self.q, self.k, self.v)]
        rc.attn_bwd(self.q, self.k, self.v, out, lse, self.dout, *grads, *self.cu, workspace=ws)
        return grads


def equal(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


# Few rows on long key ranges, which are divided: single tokens, few and many rows, both row forms and head classes
DIVIDED = [([1], [9000], 2, 4, 1, 128), ([1, 1, 1], [5000, 20, 3100], 1, 8, 8, 64), ([40, 3], [3000, 2600], 1, 8, 2, 96),
           ([300], [4097], 1, 4, 2, 128)]


@pytest.mark.parametrize("shape", DIVIDED, ids=str)
def test_attention_leaves_no_words_behind(shape):
    a = Attention(*shape, seed=1)
    want = a.forward()
    grads = a.backward(*want)
    size = max(rc.attn_fwd_workspace_bytes(*a.sizes), rc.attn_bwd_workspace_bytes(*a.sizes))
    assert rc.attn_fwd_workspace_bytes(*a.sizes) > 4096
    ws = torch.zeros(size, dtype=torch.uint8, device=DEV)
    for _ in range(2):
        assert equal(a.forward(ws), want)
        assert rc.ring_status_ex(ws) == 0
        assert not ws[HEADER:].any()
        assert equal(a.backward(*want, ws), grads)
        assert rc.ring_status_ex(ws) == 0
        assert not ws[HEADER:].any()


def test_attention_and_signalling_calls_share_a_workspace():
    """The layers of a block on one workspace: gather + matmul of new shards each time (a wait that
    ended early would use the rows gathered before), attention, and a ring all-reduce."""
    P, M_r, N, K = 4, 256, 512, 256
    a = Attention([1, 40], [9000, 3000], P, 4, 1, 128, seed=2)
    want = a.forward()
    grads = a.backward(*want)
    size = max(rc.attn_fwd_workspace_bytes(*a.sizes), rc.attn_bwd_workspace_bytes(*a.sizes),
               rc.ag_gemm_workspace_bytes(P, M_r), rc.ring_allreduce_workspace_bytes(P, 64 * P * 300, torch.float32))
    ws = torch.zeros(size, dtype=torch.uint8, device=DEV)
    g = torch.Generator(device=DEV).manual_seed(3)
    B = torch.randn(N, K, generator=g, device=DEV).to(BF)
    gathered, C = torch.empty(P * M_r, K, dtype=BF, device=DEV), torch.empty(P * M_r, N, dtype=BF, device=DEV)
    wanted, Cw = torch.empty_like(gathered), torch.empty_like(C)
    for it in range(6):
        shards = torch.randn(P, M_r, K, generator=g, device=DEV).to(BF)
        x = torch.randn(P, 64 * P * 300, generator=g, device=DEV)
        y = x.clone()
        rc.ag_gemm(shards, wanted, B, Cw, rank=it % P)
        rc.ring_allreduce(y)
        gathered.fill_(float(it))
        rc.ag_gemm_ex(shards, gathered, B, C, it % P, ws)
        assert equal(a.forward(ws), want)
        rc.ring_allreduce_ex(x, ws)
        assert equal(a.backward(*want, ws), grads)
        assert rc.ring_status_ex(ws) == 0, rc.ring_last_error()
        assert torch.equal(gathered, shards.view(P * M_r, K)) and torch.equal(C, Cw) and torch.equal(x, y)


class Norm:
    """One gradient of the query/key norm, on the library's workspace or a caller's."""

    def __init__(self, P, T, Hq, Hkv, D, seed):
        g = torch.Generator(device=DEV).manual_seed(seed)
        r = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
        self.heads = [r(P, T, h, D).to(BF) for h in (Hq, Hkv, Hq, Hkv)]
        angle = r(T, D // 2)
        self.rest = r(D), r(D), angle.cos(), angle.sin(), torch.arange(T, dtype=torch.int32, device=DEV)
        self.sizes = P, T, Hq, Hkv, D

    def backward(self, ws=None):
        q, k, dqo, dko = self.heads
        P, D = q.size(0), q.size(3)
        res = [torch.empty_like(q), torch.empty_like(k), torch.empty(P, D, device=DEV), torch.empty(P, D, device=DEV)]
        rc.qk_norm_rope_bwd(q, k, *self.rest, dqo, dko, *res, workspace=ws)
        return res


@pytest.mark.parametrize("shape", [(1, 3, 2, 1, 64), (4, 700, 4, 2, 128), (2, 45, 3, 1, 24)], ids=str)
def test_norm_gradient_leaves_the_header_and_no_words_behind(shape):
    n = Norm(*shape, seed=4)
    want = n.backward()
    ws = torch.zeros(rc.qk_norm_rope_bwd_workspace_bytes(*n.sizes), dtype=torch.uint8, device=DEV)
    ws[:HEADER] = 0x5A
    for _ in range(2):
        assert equal(n.backward(ws), want)
        assert (ws[:HEADER] == 0x5A).all() and not ws[HEADER:].any()


def test_norm_and_attention_share_a_workspace():
    n = Norm(4, 700, 4, 2, 128, seed=5)
    a = Attention([1, 40], [9000, 3000], 4, 4, 1, 128, seed=6)
    dx, want = n.backward(), a.forward()
    grads = a.backward(*want)
    size = max(rc.qk_norm_rope_bwd_workspace_bytes(*n.sizes), rc.attn_fwd_workspace_bytes(*a.sizes),
               rc.attn_bwd_workspace_bytes(*a.sizes))
    ws = torch.zeros(size, dtype=torch.uint8, device=DEV)
    for _ in range(3):
        assert equal(n.backward(ws), dx)
        assert equal(a.forward(ws), want) and equal(a.backward(*want, ws), grads)
        assert rc.ring_status_ex(ws) == 0, rc.ring_last_error()


def captured(a, out, lse):
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        rc.attn_fwd(a.q, a.k, a.v, out, lse, *a.cu)
    return graph


def test_the_library_space_grows_while_a_stream_is_captured():
    """A long prompt needs no space for parts, eight tokens do: their first call may be a captured one."""
    rc.ring_finalize()
    prompt, tokens = Attention([4096], [4096], 1, 32, 8, 128, seed=7), Attention([8], [4096], 1, 32, 8, 128, seed=8)
    assert rc.attn_fwd_workspace_bytes(*prompt.sizes) < 1024 < rc.attn_fwd_workspace_bytes(*tokens.sizes)
    prompt.forward()
    out, lse = torch.zeros_like(tokens.q), torch.zeros(tokens.q.shape[:3], device=DEV)
    captured(tokens, out, lse).replay()
    assert rc.ring_status() == 0, rc.ring_last_error()
    assert equal((out, lse), tokens.forward())


def test_captured_calls_outlive_larger_ones():
    """Calls that outgrow the library's space (parts) and its signal words (the header that
    attention counts its units in) leave what a captured call uses in place."""
    rc.ring_finalize()
    tokens = Attention([8], [4096], 1, 32, 8, 128, seed=9)
    want = tokens.forward()
    out, lse = torch.zeros_like(tokens.q), torch.zeros(tokens.q.shape[:3], device=DEV)
    graph = captured(tokens, out, lse)
    larger = Attention([2048], [2048], 1, 32, 8, 128, seed=10)
    assert rc.attn_fwd_workspace_bytes(*larger.sizes) > 2 * rc.attn_fwd_workspace_bytes(*tokens.sizes)
    wide = larger.forward()
    assert rc.ring_allreduce_workspace_bytes(64, 64 * 4096, torch.float32) > 1 << 20
    x = torch.randn(64, 64 * 4096, device=DEV)
    total = x.double().sum(0)
    rc.ring_allreduce(x)
    assert (x[3].double() - total).abs().max() <= 64 * 2.0 ** -24 * 64 * 6
    for _ in range(3):
        out.zero_(), lse.zero_()
        graph.replay()
        assert rc.ring_status() == 0, rc.ring_last_error()
        assert equal((out, lse), want) and equal(larger.forward(), wide)
