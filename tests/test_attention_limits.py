"""Sizes at which the attention and norm kernels' 32-bit indices would end are refused (CPU).

Calls that are not refused would be launched, so those here run only where there is no GPU:
they have to get as far as finding none.
"""
import pytest
import torch

import ring_collectives_gb300 as rc
from tests.test_attention_refusals import _attn, _norm, lib  # noqa: F401  (fixture)

no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="would launch")
MOST = 2**31 - 1 - 2**20


@pytest.mark.parametrize("fn", ["attn_fwd", "attn_bwd"])
@pytest.mark.parametrize("change", [dict(Tq=2**31 - 1), dict(Tk=2**31 - 1), dict(Tq=MOST + 1), dict(Tk=MOST + 1),
                                    dict(P=64, Hq=65536, Hkv=65536, B=600, Tq=600, Tk=600, D=8)], ids=str)
def test_attention_refuses_sizes_beyond_its_indices(lib, fn, change):  # noqa: F811
    assert getattr(lib, fn)(_attn(**change), None) == rc.RC_ERR_INVALID
    assert getattr(lib, fn + "_workspace_bytes")(_attn(**change)) == 0


@pytest.mark.parametrize("fn", ["qk_norm_rope", "qk_norm_rope_bwd"])
@pytest.mark.parametrize("T", [2**31 - 1, MOST + 1])
def test_norm_refuses_sizes_beyond_its_indices(lib, fn, T):  # noqa: F811
    assert getattr(lib, fn)(_norm(T=T), None) == rc.RC_ERR_INVALID


@no_gpu
def test_the_largest_sizes_are_taken(lib):  # noqa: F811
    far = {n: [(i + 1) << 44, 1 << 38, 1024, 128] for i, n in enumerate(("q", "k", "v", "out", "dout", "dq", "dk", "dv"))}
    for fn in (lib.attn_fwd, lib.attn_bwd):
        assert fn(_attn(Tq=MOST, Tk=MOST, P=1, **far), None) == rc.RC_ERR_UNSUPPORTED
        assert fn(_attn(P=64, Hq=64, Hkv=64, B=4096, Tq=4096, Tk=4096, **{n: [x[0], 1 << 30, 1 << 16, 128] for n, x in far.items()}),
                  None) == rc.RC_ERR_UNSUPPORTED
    far = {n: [(i + 1) << 44, 1 << 38, 1024, 128] for i, n in enumerate(("q", "k", "q_out", "k_out", "dq", "dk"))}
    for fn in (lib.qk_norm_rope, lib.qk_norm_rope_bwd):
        assert fn(_norm(T=MOST, P=1, **far), None) == rc.RC_ERR_UNSUPPORTED
