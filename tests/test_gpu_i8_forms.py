"""The 8-bit integer products at sizes chosen for the kernel that takes them,
against the formula in 64 bits (tolerances: those derived in test_gpu_i8_mm)."""

import pytest
import torch

from test_gpu_i8_mm import ACTS, Group, Linear

pytestmark = pytest.mark.gpu

DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    torch.cuda.init()


def at_the_end(t):
    """The same values at the end of an allocation of their own that is no longer
    than it has to be (a multiple of 512 bytes)."""
    n = t.numel()
    whole = torch.full(((n + 511) // 512 * 512,), 99, dtype=t.dtype, device=DEV)
    start = whole.numel() - n
    start -= start % 16
    whole[start:start + n] = t.reshape(-1)
    return whole[start:start + n].view(t.shape)


@pytest.mark.parametrize("act", list(ACTS))
@pytest.mark.parametrize("K", [16, 32, 48, 64, 80])
@pytest.mark.parametrize("M", [1, 20, 33, 60])
def test_few_rows_and_the_least_contractions(M, K, act):
    """Contractions shorter than a step of the few-rows kernel, the last weight row at
    the end of its buffer."""
    p = Linear(M, 34, K, act, dtype="f16" if K % 32 else "bf16")
    p.w = at_the_end(p.w)
    p.check(p())
    g = Group(M, 3, 34, K, 2, 16, act, per_route=K % 32 == 0)
    g.w = at_the_end(g.w)
    g.check(g())
