"""What the attention and query/key norm calls refuse, before any CUDA call (CPU)."""
import ctypes

import pytest

import ring_collectives_gb300 as rc

HEADS = ("q", "k", "v", "out", "dout", "dq", "dk", "dv")
NORM_HEADS = ("q", "k", "q_out", "k_out", "dq", "dk")


@pytest.fixture(scope="module")
def lib():
    from ring_collectives_gb300 import _build
    _build.build()
    return rc.load()


def _attn(**change):
    """Packed arguments of one valid call (addresses are never followed), with changes."""
    a = dict(P=2, B=3, Tq=8, Tk=16, Hq=4, Hkv=2, D=64, causal=1, scale=0.125, reserved=0, lse=0x9000, cu_q=0xA000,
             cu_k=0xB000, used_k=0, ws=0, ws_bytes=0)
    for i, n in enumerate(HEADS):
        a[n] = [0x100000 * (i + 1), 1 << 20, 1024, 128]
    a.update(change)
    return rc._ATTN_ARGS.pack(*sum((list(a[n]) for n in HEADS), []), a["lse"], a["cu_q"], a["cu_k"], a["used_k"], a["ws"],
                              a["ws_bytes"], a["P"], a["B"], a["Tq"], a["Tk"], a["Hq"], a["Hkv"], a["D"], a["causal"],
                              a["scale"], a["reserved"])


def _norm(**change):
    a = dict(P=2, T=8, Hq=4, Hkv=2, D=64, npos=9, layout=0, eps=1e-6, gamma_q=0x9000, gamma_k=0x9100, cos=0x9200,
             sin=0x9300, pos=0x9400, dgamma_q=0x9500, dgamma_k=0x9600, ws=0, ws_bytes=0)
    for i, n in enumerate(NORM_HEADS):
        a[n] = [0x100000 * (i + 1), 1 << 20, 1024, 128]
    a.update(change)
    return rc._QK_NORM_ARGS.pack(*sum((list(a[n]) for n in NORM_HEADS), []), a["gamma_q"], a["gamma_k"], a["cos"],
                                 a["sin"], a["pos"], a["dgamma_q"], a["dgamma_k"], a["ws"], a["ws_bytes"], a["P"], a["T"],
                                 a["Hq"], a["Hkv"], a["D"], a["npos"], a["layout"], a["eps"])


SIZES = [dict(P=0), dict(P=65), dict(B=0), dict(Tq=-1), dict(Tk=-1), dict(Hq=0), dict(Hkv=0), dict(Hq=5), dict(Hq=258),
         dict(D=0), dict(D=4), dict(D=68), dict(D=136), dict(scale=0.0), dict(scale=-1.0), dict(scale=float("inf")),
         dict(scale=float("nan")), dict(causal=2), dict(reserved=1)]
LAYOUT = [dict(q=[0, 1 << 20, 1024, 128]), dict(k=[0x200008, 1 << 20, 1024, 128]), dict(v=[0x300000, 1 << 20, 1032, 128]),
          dict(out=[0x400000, 1 << 20, 1024, 64]), dict(q=[0x100000, 1 << 20, 64, 128]), dict(cu_q=0), dict(cu_k=0),
          dict(k=[0x200000, 1 << 41, 1024, 128])]


@pytest.mark.parametrize("fn", ["attn_fwd", "attn_bwd"])
@pytest.mark.parametrize("change", SIZES + LAYOUT, ids=str)
def test_attention_refuses(lib, fn, change):
    assert getattr(lib, fn)(_attn(**change), None) == rc.RC_ERR_INVALID
    assert rc.ring_last_error()


@pytest.mark.parametrize("change", [dict(out=[0x100000, 1 << 20, 1024, 128]), dict(out=[0x300000, 1 << 20, 1024, 128])], ids=str)
def test_forward_output_may_not_be_an_input(lib, change):
    assert lib.attn_fwd(_attn(**change), None) == rc.RC_ERR_INVALID


@pytest.mark.parametrize("change", [dict(lse=0), dict(dout=[0, 1 << 20, 1024, 128]), dict(dk=[0x800000, 1 << 20, 1024, 128]),
                                    dict(dq=[0x100000, 1 << 20, 1024, 128]), dict(dv=[0x300000, 1 << 20, 1024, 120])], ids=str)
def test_backward_refuses(lib, change):
    assert lib.attn_bwd(_attn(**change), None) == rc.RC_ERR_INVALID


@pytest.mark.parametrize("fn", ["qk_norm_rope", "qk_norm_rope_bwd"])
@pytest.mark.parametrize("change", [dict(P=0), dict(P=65), dict(T=-1), dict(Hq=0), dict(Hkv=0), dict(D=0), dict(D=12),
                                    dict(D=264), dict(npos=0), dict(layout=2), dict(eps=-1.0), dict(eps=float("inf")),
                                    dict(gamma_q=0), dict(gamma_k=0x9104), dict(cos=0), dict(sin=0x9308), dict(pos=0),
                                    dict(q=[0, 1 << 20, 1024, 128]), dict(k_out=[0x400002, 1 << 20, 1024, 128]),
                                    dict(q_out=[0x300000, 1 << 20, 1024, 96])], ids=str)
def test_norm_refuses(lib, fn, change):
    assert getattr(lib, fn)(_norm(**change), None) == rc.RC_ERR_INVALID


@pytest.mark.parametrize("change", [dict(dgamma_q=0), dict(dgamma_k=0), dict(dq=[0, 1 << 20, 1024, 128])], ids=str)
def test_norm_gradient_refuses(lib, change):
    assert lib.qk_norm_rope_bwd(_norm(**change), None) == rc.RC_ERR_INVALID


def test_null_arguments_and_empty_work(lib):
    for fn in (lib.attn_fwd, lib.attn_bwd, lib.qk_norm_rope, lib.qk_norm_rope_bwd):
        assert fn(None, None) == rc.RC_ERR_INVALID
    assert lib.attn_fwd(_attn(Tq=0), None) == rc.RC_OK
    assert lib.attn_bwd(_attn(Tq=0, Tk=0), None) == rc.RC_OK
    assert lib.qk_norm_rope(_norm(T=0), None) == rc.RC_OK
    for fn in (lib.attn_fwd_workspace_bytes, lib.attn_bwd_workspace_bytes, lib.qk_norm_rope_bwd_workspace_bytes):
        assert fn(None) == 0
    assert lib.attn_bwd_workspace_bytes(_attn(D=12)) == 0


def test_argument_structs_match_the_header(lib):
    """The packed layouts are those of the C structs (no padding is lost)."""
    class Heads(ctypes.Structure):
        _fields_ = [("base", ctypes.c_void_p)] + [(n, ctypes.c_size_t) for n in ("slot", "token", "head")]

    class Attn(ctypes.Structure):
        _fields_ = ([(n, Heads) for n in HEADS] + [(n, ctypes.c_void_p) for n in ("lse", "cu_q", "cu_k", "used_k", "workspace")]
                    + [("ws_bytes", ctypes.c_size_t)] + [(n, ctypes.c_int) for n in ("P", "B", "Tq", "Tk", "Hq", "Hkv", "D", "causal")]
                    + [("scale", ctypes.c_float), ("reserved", ctypes.c_int)])

    class Norm(ctypes.Structure):
        _fields_ = ([(n, Heads) for n in NORM_HEADS]
                    + [(n, ctypes.c_void_p) for n in ("gamma_q", "gamma_k", "cos", "sin", "pos", "dgamma_q", "dgamma_k", "workspace")]
                    + [("ws_bytes", ctypes.c_size_t)] + [(n, ctypes.c_int) for n in ("P", "T", "Hq", "Hkv", "D", "npos", "layout")]
                    + [("eps", ctypes.c_float)])

    a = Attn.from_buffer_copy(_attn(reserved=7))
    assert ctypes.sizeof(Attn) == rc._ATTN_ARGS.size and (a.dv.head, a.cu_k, a.P, a.causal, a.scale, a.reserved) == (
        128, 0xB000, 2, 1, 0.125, 7)
    n = Norm.from_buffer_copy(_norm(layout=1))
    assert ctypes.sizeof(Norm) == rc._QK_NORM_ARGS.size and (n.dk.base, n.dgamma_k, n.npos, n.layout) == (0x600000, 0x9600, 9, 1)
