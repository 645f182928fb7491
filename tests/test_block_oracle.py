"""The 64-bit definitions of the block operators: their gradients against differences, the 8-bit form's
properties, and bounds that a mistake does not pass (CPU)."""
import numpy as np
import pytest

from oracle import block as ob


def bf16(x):
    """Nearest bf16, in float64 (ties to even)."""
    b = np.asarray(x, np.float32).view(np.uint32).astype(np.uint64)
    b = (b + 0x7FFF + ((b >> 16) & 1)) >> 16 << 16
    return b.astype(np.uint32).view(np.float32).astype(np.float64)


@pytest.fixture
def rng():
    return np.random.default_rng(5)


@pytest.mark.parametrize("N", [8, 32, 40, 64, 1000])
def test_8_bits_are_the_nearest_multiples(rng, N):
    x = bf16(rng.standard_normal((2, 9, N)) * 2.0 ** rng.integers(-30, 30, (2, 9, 1)))
    x[0, 0] = 0
    q, e = ob.act8_pack(x)
    v = ob.act8_values(q, e)
    assert q.min() >= -127 and e.shape == (2, 9, -(-N // 32)) and (e[0, 0] == 1).all()
    step = 2.0 ** (e.astype(float) - 127)[..., np.arange(N) // 32]
    assert (np.abs(v - x) <= step / 2).all()
    for g in range(0, N, 32):                         # no smaller power of two would do, and the error stays below 1/127
        top = np.abs(x[..., g:g + 32]).max(-1)
        assert ((top > 127 * step[..., g] / 2) | (top == 0)).all() and (np.abs(v - x)[..., g:g + 32].max(-1) <= top / 127).all()
    again = ob.act8_pack(v)
    assert np.array_equal(ob.act8_values(*again), v)  # values that 8 bits hold stay what they are


def test_8_bits_at_the_ends_of_the_range():
    x = np.zeros((1, 4, 32))
    big = bf16(3.3895e38)
    x[0, 0, 0], x[0, 1, 0], x[0, 2, 0], x[0, 3, 5] = big, 2.0 ** -133, np.nan, -np.inf
    q, e = ob.act8_pack(x)
    assert q[0, 0, 0] == 127 and e[0, 0, 0] == 248 and e[0, 1, 0] == 1 and (e[0, 2:] == 255).all()
    v = ob.act8_values(q, e)
    assert abs(v[0, 0, 0] - big) <= big / 127 and v[0, 1, 0] == 0 and np.isnan(v[0, 2:]).all()


@pytest.mark.parametrize("post,gate,pre", [(1, 1, 1), (1, 0, 1), (0, 1, 1), (0, 0, 1), (1, 1, 0), (1, 0, 0), (0, 1, 0), (0, 0, 0)])
def test_block_norm_gradient_against_differences(rng, post, gate, pre):
    P, T, N, alpha, eps = 2, 3, 24, 0.7, 1e-3
    y, res, dh, dz = (rng.standard_normal((P, T, N)) for _ in range(4))
    w = [rng.standard_normal(N) if on else None for on in (post, gate, pre)]

    def value(y, res, w):
        (h, z), _ = ob.block_norm(y, res, *w, alpha=alpha, eps=eps)
        return (h * dh).sum() + (0.0 if z is None else (z * dz).sum())

    g, _ = ob.block_norm_bwd(y, res, dh, dz, *w, alpha=alpha, eps=eps)
    step = 1e-5
    for i, name in enumerate(("dy", "dres", "dgamma_post", "dgate", "dgamma_pre")):
        if name not in g:
            assert i > 1 and w[i - 2] is None
            continue
        at = [y, res, *w]
        v = rng.standard_normal(at[i].shape)
        ends = []
        for sign in (1, -1):
            moved = list(at)
            moved[i] = at[i] + sign * step * v
            ends.append(value(moved[0], moved[1], moved[2:]))
        slope = (g[name] * v).sum()
        assert abs((ends[0] - ends[1]) / (2 * step) - slope) <= 1e-7 * (1 + abs(g[name] * v).sum())


@pytest.mark.parametrize("kind", ["silu", "gelu"])
def test_glu_gradient_against_differences(rng, kind):
    a, b, dh = (2 * rng.standard_normal((1, 4, 16)) for _ in range(3))
    (da, db, h), _ = ob.glu_bwd(a, b, dh, kind)
    assert np.array_equal(h, ob.glu(a, b, kind)[0])
    for g, move in ((da, (1e-5, 0)), (db, (0, 1e-5))):
        up, down = (ob.glu(a + s * move[0], b + s * move[1], kind)[0] for s in (1, -1))
        assert np.abs((up - down) / 2e-5 * dh - g).max() <= 1e-7


def test_activations_match_their_usual_form(rng):
    x = np.linspace(-9, 9, 999)[None, None]
    one = np.ones_like(x)
    tanh = 0.5 * x * (1 + np.tanh(np.sqrt(2 / np.pi) * (x + 0.044715 * x ** 3)))
    assert np.abs(ob.glu(x, one, "gelu")[0] - tanh).max() < 1e-14
    assert np.abs(ob.glu(x, one, "silu")[0] - x / (1 + np.exp(-x))).max() < 1e-14


def test_column_chunks_and_rows_are_inverse(rng):
    y = rng.standard_normal((4, 3, 64))
    c = ob.to_cols(y)
    assert c.shape == (4, 12, 16) and np.array_equal(ob.from_cols(c, 3), y)
    assert c[2, 3 * 1 + 2, 5] == y[1, 2, 2 * 16 + 5]        # chunk 2, row 2 of rank 1


def test_bounds_fail_a_wrong_result(rng):
    """A mistake planted in the formulas leaves their bounds: eps dropped, a mean over N - 1, a gate
    applied twice, the second norm of the rounded sum's gradient left out."""
    y, res, dh, dz = (bf16(rng.standard_normal((1, 5, 64))) for _ in range(4))
    g = [1 + 0.2 * rng.standard_normal(64) for _ in range(3)]
    (h, z), (hb, zb) = ob.block_norm(y, res, *g, eps=1e-2)
    assert (np.abs(ob.block_norm(y, res, *g, eps=0.0)[0][0] - h) > hb).any()
    assert (np.abs(z * np.sqrt(63 / 64) - z) > zb).any()
    (want, off), (bad, _) = (ob.block_norm_bwd(y, res, dh, dz, *w) for w in (g, (g[0], g[1] ** 2, g[2])))
    assert all((np.abs(want[k] - bad[k]) > off[k]).any() for k in want)
    short, _ = ob.block_norm_bwd(y, res, dh, 0 * dz, *g)
    assert (np.abs(want["dres"] - short["dres"]) > off["dres"]).any()
