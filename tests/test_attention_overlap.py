"""Results that share bytes with an input, with one another or within themselves are refused (CPU).

The layouts are strided, so their spans may cross without a shared byte (heads inside one
fused buffer): the answer is compared with the sets of bytes themselves.  Calls that are not
refused would be launched, so those run only where there is no GPU.
"""
import random

import pytest
import torch

import ring_collectives_gb300 as rc
from tests.test_attention_refusals import HEADS, NORM_HEADS, _attn, _norm, lib  # noqa: F401  (fixture)

no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="would launch")
FAR = {n: [(i + 1) << 36, 1 << 20, 1 << 14, 128] for i, n in enumerate(HEADS)}
NORM_FAR = {n: [(i + 1) << 36, 1 << 20, 1 << 14, 128] for i, n in enumerate(NORM_HEADS)}
Q = FAR["q"][0]
K = FAR["k"][0]


def at(base, slot=1 << 20, token=1 << 14, head=128):
    return [base, slot, token, head]


FUSED = 12 * 128   # a token of one rank: 4 query, 2 key, 2 value heads of 64 and room for 4 more


@pytest.mark.parametrize("change", [
    dict(out=at(Q + 16)), dict(out=at(Q + 128)), dict(out=at(Q + (1 << 14))), dict(out=at(Q - (1 << 20))),
    dict(out=at(Q + 64, 1 << 21, 1 << 15)), dict(out=at(K + 128)), dict(out=at(FAR["v"][0] + 5 * (1 << 14))),
    dict(out=at(Q, 1 << 20, 1 << 14, 256)), dict(out=at(Q - 512, 4096, 512, 128)),
    dict(lse=Q), dict(lse=Q + (1 << 20) + 7 * (1 << 14) + 508), dict(lse=FAR["out"][0]),
    dict(out=at(FAR["out"][0], 1 << 20, 256, 128)), dict(out=at(FAR["out"][0], 1 << 20, 1 << 20, 128)),
    dict(out=at(FAR["out"][0], 1 << 20, 384, 256))], ids=str)
def test_forward_refuses_results_on_inputs(lib, change):  # noqa: F811
    assert lib.attn_fwd(_attn(**{**FAR, **change}), None) == rc.RC_ERR_INVALID
    assert "overlap" in rc.ring_last_error()


@pytest.mark.parametrize("change", [
    dict(dq=at(Q + 16)), dict(dq=at(FAR["out"][0] + 128)), dict(dq=at(FAR["dout"][0])), dict(dk=at(FAR["dv"][0] + 128)),
    dict(dk=at(FAR["dq"][0] + 3 * (1 << 14) + 384)), dict(dv=at(K + (1 << 20))), dict(dk=at(0x9000 & ~15, 1 << 20, 1 << 14)),
    dict(dv=at(FAR["dv"][0], 1 << 14, 1 << 14))], ids=str)
def test_backward_refuses_results_on_inputs(lib, change):  # noqa: F811
    assert lib.attn_bwd(_attn(**{**FAR, **change}), None) == rc.RC_ERR_INVALID
    assert "overlap" in rc.ring_last_error()


@pytest.mark.parametrize("change", [dict(q_out=at(NORM_FAR["q"][0] + 128)), dict(q_out=at(NORM_FAR["k"][0])),
                                    dict(k_out=at(NORM_FAR["q"][0])), dict(q_out=at(NORM_FAR["q"][0], 1 << 20, 1 << 13)),
                                    dict(k_out=at(NORM_FAR["q_out"][0] + 256))], ids=str)
def test_norm_refuses_results_on_inputs(lib, change):  # noqa: F811
    assert lib.qk_norm_rope(_norm(**{**NORM_FAR, **change}), None) == rc.RC_ERR_INVALID
    assert "overlap" in rc.ring_last_error()


@pytest.mark.parametrize("change", [dict(dq=at(NORM_FAR["q"][0] + 128)), dict(dq=at(NORM_FAR["k_out"][0])), dict(dk=at(NORM_FAR["dq"][0] + 128)),
                                    dict(dgamma_q=NORM_FAR["q"][0]), dict(dgamma_k=NORM_FAR["dk"][0] + (1 << 14)),
                                    dict(dgamma_q=0x9500, dgamma_k=0x9500 + 2 * 64 * 4 - 4)], ids=str)
def test_norm_gradient_refuses_results_on_inputs(lib, change):  # noqa: F811
    base = {**NORM_FAR, "dgamma_q": 0x100000, "dgamma_k": 0x200000}
    assert lib.qk_norm_rope_bwd(_norm(**{**base, **change}), None) == rc.RC_ERR_INVALID
    assert "overlap" in rc.ring_last_error()


@no_gpu
def test_heads_of_one_fused_buffer_are_taken(lib):  # noqa: F811
    """Views of one activation buffer: the spans cross, no byte is shared."""
    def view(first, base=0, P=2):
        return [Q + base + first * 128, FUSED, P * FUSED, 128]

    assert lib.attn_fwd(_attn(**{**FAR, "q": view(0), "k": view(4), "v": view(6), "out": view(8)}), None) == rc.RC_ERR_UNSUPPORTED
    assert lib.attn_fwd(_attn(**{**FAR, "q": view(0), "k": view(4), "v": view(6), "out": view(7)}), None) == rc.RC_ERR_INVALID
    grads = {"dq": view(0, 1 << 30), "dk": view(4, 1 << 30), "dv": view(6, 1 << 30)}
    assert lib.attn_bwd(_attn(**{**FAR, **grads}), None) == rc.RC_ERR_UNSUPPORTED
    long = dict(Tq=1 << 24, Tk=1 << 24, P=2, **{n: [x[0] << 8, 1 << 38, 2 * FUSED, 128] for n, x in FAR.items()})
    for n, first in (("dq", 0), ("dk", 4), ("dv", 6)):
        long[n] = [(9 << 44) + first * 128, FUSED, 2 * FUSED, 128]
    assert lib.attn_bwd(_attn(**long), None) == rc.RC_ERR_UNSUPPORTED
    long["dv"][0] -= 128
    assert lib.attn_bwd(_attn(**long), None) == rc.RC_ERR_INVALID
    q, k = view(0), view(4)
    assert lib.qk_norm_rope(_norm(**{**NORM_FAR, "q": q, "k": k, "q_out": q, "k_out": k}), None) == rc.RC_ERR_UNSUPPORTED
    base = {**NORM_FAR, "dgamma_q": 0x100000, "dgamma_k": 0x200000}
    assert lib.qk_norm_rope_bwd(_norm(**{**base, "dq": base["q_out"], "dk": base["k_out"]}), None) == rc.RC_ERR_UNSUPPORTED
    assert lib.qk_norm_rope_bwd(_norm(**{**base, "dq": base["q"], "dk": base["k"]}), None) == rc.RC_ERR_UNSUPPORTED


def _units(h, P, T, H, D):
    """The 16-byte units of an operand, and whether two of its heads share one."""
    s = [u for r in range(P) for t in range(T) for i in range(H)
         for u in range((h[0] + r * h[1] + t * h[2] + i * h[3]) // 16, (h[0] + r * h[1] + t * h[2] + i * h[3] + 2 * D) // 16)]
    return set(s), len(set(s)) < len(s)


@no_gpu
def test_refused_exactly_where_bytes_are_shared(lib):  # noqa: F811
    """Random layouts of q and out, fused, nested, crossing and of unrelated strides."""
    rng = random.Random(5)
    seen = {True: 0, False: 0}
    for _ in range(6000):
        P, T, G, D = rng.choice([1, 2, 3]), rng.choice([1, 2, 4, 7]), rng.choice([1, 2, 4]), rng.choice([8, 16, 24])

        def strides():
            x = [rng.choice([1, 1, 2, 3]) * 2 * D]
            for n in rng.sample([G, T, P], 3):
                x.append(max(2 * D, x[-1] * n + rng.choice([0, 0, 16, -16, 64, 160])))
            order = rng.choice([(2, 1, 0), (2, 1, 0), (1, 2, 0), (2, 0, 1), (0, 1, 2)])
            return [x[i] // 16 * 16 for i in order]

        base = 1 << 36
        q = [base] + strides()
        out = [base + 16 * rng.randrange(-60, 200)] + (q[1:] if rng.random() < 0.5 else strides())
        ext = [(n, s) for n, s in ((P, 1), (T, 2), (G, 3))]
        for h in (q, out):                          # what the library takes for an extent of 1
            for n, s in ext:
                h[s] = 2 * D if n == 1 else max(h[s], 2 * D)
        (a, _), (b, self_) = _units(q, P, T, G, D), _units(out, P, T, G, D)
        want = bool(a & b) or self_
        seen[want] += 1
        far = {n: [(i + 1) << 40, 1 << 20, 1 << 14, 128] for i, n in enumerate(HEADS)}
        got = lib.attn_fwd(_attn(**{**far, "q": q, "out": out, "P": P, "Tq": T, "Hq": G, "Hkv": 1, "D": D}), None)
        assert got == (rc.RC_ERR_INVALID if want else rc.RC_ERR_UNSUPPORTED), (q, out, P, T, G, D, rc.ring_last_error())
    assert min(seen.values()) > 1000, seen
