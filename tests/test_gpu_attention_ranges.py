"""Attention at lengths where index arithmetic could leave 32 bits (needs a GB300)."""
import numpy as np
import pytest
import torch

import ring_collectives_gb300 as rc
from oracle import attention as oa
from tests.test_gpu_attention import BF, DEV, f64, inside, ints, rand

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(DEV)
    rc.ring_set_timeout_ms(10000)
    yield
    rc.ring_set_timeout_ms(2000)


def test_gradient_of_a_large_group_on_a_long_key_range():
    """Two tokens of 128 heads on one key head and over 2^31 / 128 keys: the distance of a key
    from the tokens, in rows of a tile, passes 32 bits.  dK and dV of a key depend on the other
    keys through lse and the output only, so they are checked at the keys of both ends and
    around the distance where 32 bits end."""
    G, D, T = 128, 8, (1 << 24) + 3000
    g = torch.Generator(device=DEV).manual_seed(1)
    q, dout = rand(g, 1, 2, G, D), rand(g, 1, 2, G, D)
    k, v = (torch.zeros(1, T, 1, D, dtype=BF, device=DEV) for _ in range(2))
    edge = T - (1 << 24)
    some = torch.cat([torch.arange(0, 700), torch.arange(edge - 300, edge + 300), torch.arange(T - 300, T)]).to(DEV)
    k[:, some], v[:, some] = rand(g, 1, some.numel(), 1, D), rand(g, 1, some.numel(), 1, D)
    cq, ck = ints([0, 2]), ints([0, T])
    out, lse = torch.empty_like(q), torch.empty(q.shape[:3], device=DEV)
    rc.attn_fwd(q, k, v, out, lse, cq, ck)
    dq, dk, dv = torch.empty_like(q), torch.full_like(k, float("nan")), torch.full_like(v, float("nan"))
    rc.attn_bwd(q, k, v, out, lse, dout, dq, dk, dv, cq, ck)
    assert rc.ring_status() == 0, rc.ring_last_error()
    # the last key is seen by the second token only, so the oracle's mask is that of the sub-sequence
    want, bound = oa.attn_bwd(f64(q), f64(k[:, some]), f64(v[:, some]), f64(out), f64(lse), f64(dout),
                              [(0, 2, 0, some.numel())])
    inside(dk[:, some], want[1], bound[1], "dk")
    inside(dv[:, some], want[2], bound[2], "dv")
    rest = torch.ones(T, dtype=torch.bool, device=DEV)
    rest[some] = False
    assert torch.isfinite(dk).all() and (dv[0, rest] == dv[0, rest][:1]).all() and (dv[0, rest][0] != 0).any()
