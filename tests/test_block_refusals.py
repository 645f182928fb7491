"""What the 8-bit, block norm and gated activation calls refuse, before any CUDA call (CPU)."""
import pytest

import ring_collectives_gb300 as rc

ROWS = [1 << 20, 128]          # slot and row strides of the default operands: rows of 64 bf16


@pytest.fixture(scope="module")
def lib():
    from ring_collectives_gb300 import _build
    _build.build()
    return rc.load()


def _packed(base):
    return [base, 1 << 20, 64, base + 0x80000, 1 << 20, 2]


def _act8(**change):
    """Packed arguments of one valid call (addresses are never followed), with changes."""
    a = dict(x=[0x100000000, *ROWS], x8=_packed(0x200000000), P=2, T=8, N=64, reserved=0)
    a.update(change)
    return rc._ACT8_ARGS.pack(*a["x"], *a["x8"], a["P"], a["T"], a["N"], a["reserved"])


NORM = ("y", "res", "h", "z", "dh", "dz", "dy", "dres")
WEIGHTS = ("gamma_post", "gate", "gamma_pre", "dgamma_post", "dgate", "dgamma_pre")


def _norm(**change):
    a = dict(P=2, T=8, N=64, y_cols=0, dy_cols=0, dz_cols=0, alpha=1.0, eps=1e-6, ws=0, ws_bytes=0, y8=[0] * 6, res8=[0] * 6, z8=[0] * 6)
    for i, n in enumerate(NORM):
        a[n] = [0x100000000 * (i + 1), *ROWS]
    for i, n in enumerate(WEIGHTS):
        a[n] = 0xA000 + 0x1000 * i
    a.update(change)
    return rc._BLOCK_NORM_ARGS.pack(*sum((list(a[n]) for n in NORM + ("y8", "res8", "z8")), []), *(a[n] for n in WEIGHTS),
                                    a["ws"], a["ws_bytes"], a["P"], a["T"], a["N"], a["y_cols"], a["dy_cols"], a["alpha"],
                                    a["eps"], a["dz_cols"])


GLU = ("a", "b", "h", "dh", "da", "db")


def _glu(**change):
    a = dict(P=2, T=8, N=64, act=0, reserved=[0, 0], a8=[0] * 6, b8=[0] * 6, h8=[0] * 6)
    for i, n in enumerate(GLU):
        a[n] = [0x100000000 * (i + 1), *ROWS]
    a.update(change)
    return rc._GLU_ARGS.pack(*sum((list(a[n]) for n in GLU + ("a8", "b8", "h8")), []), a["P"], a["T"], a["N"], a["act"], *a["reserved"])


SIZES = [dict(P=0), dict(P=65), dict(T=-1), dict(T=1 << 30), dict(N=0), dict(N=4), dict(N=68)]
CHUNKED = 16384 * 2


@pytest.mark.parametrize("fn", ["act8_pack", "act8_unpack"])
@pytest.mark.parametrize("change", SIZES + [
    dict(N=(1 << 20) + 8), dict(reserved=1), dict(x=[0, *ROWS]), dict(x=[0x100000008, *ROWS]), dict(x=[0x100000000, 1 << 20, 136]),
    dict(x=[0x100000000, 1 << 20, 112]), dict(x=[0x100000000, 0, 128]), dict(x8=[0] * 6), dict(x8=_packed(0x200000000)[:3] + [0] * 3),
    dict(x8=_packed(0x200000004)), dict(x8=[0x200000000, 1 << 20, 56, 0x300000000, 1 << 20, 2]),
    dict(x8=[0x200000000, 1 << 20, 64, 0x300000000, 1 << 20, 1]), dict(x8=_packed(0x100000000)), dict(x=[0x100000000, 1 << 41, 128])], ids=str)
def test_act8_refuses(lib, fn, change):
    assert getattr(lib, fn)(_act8(**change), None) == rc.RC_ERR_INVALID
    assert rc.ring_last_error()


@pytest.mark.parametrize("fn", ["block_norm", "block_norm_bwd"])
@pytest.mark.parametrize("change", SIZES + [
    dict(N=16392), dict(dz_cols=2), dict(y_cols=2), dict(dy_cols=-1), dict(alpha=float("inf")), dict(alpha=float("nan")), dict(eps=-1.0),
    dict(eps=float("inf")), dict(P=3, N=64, y_cols=1), dict(y=[0, *ROWS]), dict(res=[0x200000008, *ROWS]), dict(gate=0xB004),
    dict(y_cols=1, y=[0x100000000, 1 << 20, 48])], ids=str)
def test_block_norm_refuses(lib, fn, change):
    assert getattr(lib, fn)(_norm(**change), None) == rc.RC_ERR_INVALID
    assert rc.ring_last_error()


@pytest.mark.parametrize("change", [
    dict(z=[0, 0, 0]), dict(gamma_pre=0), dict(z8=_packed(0x2000000000), z=[0, 0, 0], gamma_pre=0), dict(h=[0, *ROWS]),
    dict(h=[0x100000000, *ROWS]), dict(z=[0x200000000, *ROWS]), dict(z=[0x300000000, *ROWS]), dict(h=[0x200000080, *ROWS]),
    dict(y8=_packed(0x200000000)), dict(res8=_packed(0x2000000000), y8=_packed(0x2000000000)), dict(y8=_packed(0x2000000004)),
    dict(h=[0xA000 - 128, *ROWS])], ids=str)
def test_block_norm_forward_refuses(lib, change):
    assert lib.block_norm(_norm(**change), None) == rc.RC_ERR_INVALID


@pytest.mark.parametrize("change", [
    dict(dz=[0, 0, 0]), dict(gamma_pre=0), dict(dgamma_pre=0), dict(gate=0), dict(dgate=0), dict(gamma_post=0), dict(dgamma_post=0),
    dict(dy=[0, *ROWS]), dict(dres=[0, *ROWS]), dict(res8=_packed(0x2000000000)), dict(y8=_packed(0x2000000000)),
    dict(dy=[0x100000000, *ROWS]), dict(dy=[0x800000000, *ROWS]), dict(dres=[0x600000080, *ROWS]), dict(dgate=0xF000),
    dict(dy_cols=1, dy=[0x500000000, 1 << 20, 64]), dict(dz_cols=1, dz=[0x600000000, 1 << 20, 48]),
    dict(dz_cols=1, dz=[0x600000000, 1 << 20, 128], dres=[0x600000000, 1 << 20, 128]), dict(ws=0x1000080, ws_bytes=1 << 40)], ids=str)
def test_block_norm_gradient_refuses(lib, change):
    assert lib.block_norm_bwd(_norm(**change), None) == rc.RC_ERR_INVALID


@pytest.mark.parametrize("fn", ["glu", "glu_bwd"])
@pytest.mark.parametrize("change", SIZES + [
    dict(N=(1 << 20) + 8), dict(act=2), dict(act=-1), dict(reserved=[0, 1]), dict(a=[0, *ROWS]), dict(b=[0x200000008, *ROWS]),
    dict(h8=_packed(0x2000000004)), dict(h8=_packed(0x300000000))], ids=str)
def test_glu_refuses(lib, fn, change):
    assert getattr(lib, fn)(_glu(**change), None) == rc.RC_ERR_INVALID
    assert rc.ring_last_error()


@pytest.mark.parametrize("fn,change", [
    ("glu", dict(h=[0, *ROWS])), ("glu", dict(h=[0x100000080, *ROWS])), ("glu", dict(a8=_packed(0x300000000))),
    ("glu_bwd", dict(da=[0, *ROWS])), ("glu_bwd", dict(db=[0x500000000, *ROWS])), ("glu_bwd", dict(h=[0x400000000, *ROWS])),
    ("glu_bwd", dict(a8=_packed(0x2000000000))), ("glu_bwd", dict(b8=_packed(0x2000000000))), ("glu_bwd", dict(dh=[0, *ROWS])), ("glu_bwd", dict(da=[0x400000040, *ROWS]))], ids=str)
def test_glu_places_refused(lib, fn, change):
    assert getattr(lib, fn)(_glu(**change), None) == rc.RC_ERR_INVALID


def test_null_arguments(lib):
    for fn in ("act8_pack", "act8_unpack", "block_norm", "block_norm_bwd", "glu", "glu_bwd"):
        assert getattr(lib, fn)(None, None) == rc.RC_ERR_INVALID
    assert lib.block_norm_bwd_workspace_bytes(None) == 0 and lib.block_norm_bwd_workspace_bytes(_norm(N=4)) == 0


def test_nothing_to_do_is_no_error(lib):
    """T = 0 returns before any operand or device is looked at (the gradient still writes sums of 0)."""
    for fn, args in (("act8_pack", _act8), ("act8_unpack", _act8), ("block_norm", _norm), ("glu", _glu), ("glu_bwd", _glu)):
        assert getattr(lib, fn)(args(T=0), None) == rc.RC_OK


def _wgrad(**change):
    a = dict(dy=[0x100000000, *ROWS], x8=[0x200000000, 1 << 20, 72, 0x300000000, 1 << 20, 3], dw=[0x400000000, 1 << 20, 144], ws=0, ws_bytes=0,
             P=2, T=8, N=64, K=72, dw_type=1, accumulate=0, reserved=[0, 0])
    a.update(change)
    return rc._WGRAD_ARGS.pack(*a["dy"], *a["x8"], *a["dw"], a["ws"], a["ws_bytes"], a["P"], a["T"], a["N"], a["K"], a["dw_type"],
                               a["accumulate"], *a["reserved"])


@pytest.mark.parametrize("change", [
    dict(P=0), dict(P=65), dict(T=-1), dict(T=0x7FFFFFFF), dict(N=0), dict(N=60), dict(K=4), dict(K=76), dict(N=(1 << 20) + 8),
    dict(N=1 << 20, K=1 << 20, dw=[0x400000000, 1 << 38, 1 << 21]), dict(dw_type=2), dict(accumulate=2), dict(reserved=[1, 0]),
    dict(dy=[0, *ROWS]), dict(dy=[0x100000008, *ROWS]), dict(dy=[0x100000000, 64, 128]), dict(x8=[0] * 6),
    dict(x8=[0x200000000, 1 << 20, 76, 0x300000000, 1 << 20, 3]), dict(x8=[0x200000000, 1 << 20, 72, 0x300000000, 1 << 20, 2]),
    dict(dw=[0, 1 << 20, 144]), dict(dw=[0x400000008, 1 << 20, 144]), dict(dw=[0x400000000, 0, 144]), dict(dw=[0x400000000, 1 << 20, 128]),
    dict(dw_type=0), dict(dw=[0x100000000, 1 << 20, 144]), dict(dw=[0x300000000, 1 << 20, 144]), dict(ws=0x1000080, ws_bytes=1 << 40)], ids=str)
def test_wgrad_refuses(lib, change):
    assert lib.gemm_wgrad(_wgrad(**change), None) == rc.RC_ERR_INVALID
    assert rc.ring_last_error()
    assert lib.gemm_wgrad(None, None) == rc.RC_ERR_INVALID and lib.gemm_wgrad_workspace_bytes(None) == 0
