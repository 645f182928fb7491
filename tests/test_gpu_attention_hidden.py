"""Few hidden values that are not finite: single rows and single elements, wherever they lie in a
tile (needs a GB300)."""
import pytest
import torch

import ring_collectives_gb300 as rc
from tests.test_gpu_attention import DEV, check_forward, forward, problem

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(DEV)
    rc.ring_set_timeout_ms(2000)


@pytest.mark.parametrize("D", [64, 72, 128])
@pytest.mark.parametrize("rows", [1, 3])
@pytest.mark.parametrize("keys", [1, 57, 127, 130, 255, 1081])
def test_a_row_behind_the_used_ones(keys, rows, D):
    """A cache with one or three rows too many, which hold infinities."""
    p = problem([1, 1], [keys, keys], Hq=7, Hkv=1, D=D, cap=keys + rows, seed=41)
    for b in range(2):
        end = int(p["cu_k"][b + 1])
        p["k"][:, end - rows:end] = float("nan")
        p["v"][:, end - rows:end] = float("inf")
    check_forward(p)


@pytest.mark.parametrize("D", [48, 96, 128])
def test_single_elements_in_a_prompt(D):
    """One value that is not finite, at every eighth key and in changing columns: rows before it are
    what they are without it, in every bit, and the later ones are off in its column only."""
    T = 300
    p = problem([T], [T], Hq=2, Hkv=1, D=D, seed=42)
    clean, _ = forward(p)
    v = p["v"].clone()
    for n, key in enumerate(range(0, T, 8)):
        column = (n * 29 + 3) % D
        p["v"] = v.clone()
        p["v"][0, key, 0, column] = float("-inf") if n & 1 else float("nan")
        out, _ = forward(p)
        assert torch.equal(out[0, :key], clean[0, :key]), (key, column)
        rest = torch.arange(D, device=DEV) != column
        assert torch.equal(out[0, key:, :, rest], clean[0, key:, :, rest]), (key, column)
        assert not torch.isfinite(out[0, key:, :, column]).any(), (key, column)
