"""The 8-bit integer products at sizes chosen for the kernel that takes them,
against the formula in 64 bits (tolerances: those derived in test_gpu_i8_mm)."""

import pytest
import torch

import fp8_block_scale_amd as moe
from test_gpu_i8_mm import ACTS, Group, Linear

pytestmark = pytest.mark.gpu

DEV = "cuda"

# Sizes of every kernel form, by (rows of a few-rows pass, rows and weight rows of a
# tile), without SwiGLU and with it; test_i8_host checks that each takes its form.
# Contractions are no multiple of a step, output columns no multiple of 8 where the
# form has code for that.
LINEAR = {  # M, N, K, act
    (16, 0, 0): [(9, 34, 1136, "none"), (9, 40, 1232, "swiglu")],
    (32, 0, 0): [(20, 2282, 1136, "silu"), (18, 2170, 1440, "swiglu")],
    (48, 0, 0): [(37, 2390, 1120, "none"), (75, 1470, 1104, "swiglu")],
    (64, 0, 0): [(54, 2202, 1184, "silu"), (53, 2436, 1184, "swiglu")],
    (0, 64, 64): [(1366, 34, 720, "gelu"), (1193, 40, 784, "swiglu")],
    (0, 64, 128): [(4344, 210, 704, "gelu"), (5869, 148, 720, "swiglu")],
    (0, 128, 128): [(1218, 1770, 736, "none"), (407, 5000, 704, "swiglu")],
    (0, 128, 256): [(1745, 2646, 1104, "silu"), (1753, 2494, 1040, "swiglu")],
    (0, 256, 256): [(4620, 3040, 976, "silu"), (2103, 4480, 1968, "swiglu")],
}
GROUP = {   # M, E, N, K, top_k, block_m, act
    (16, 0, 0): [(33, 2, 34, 1200, 1, 32, "gelu"), (7, 2, 38, 1456, 3, 64, "swiglu")],
    (32, 0, 0): [(56, 7, 324, 1120, 3, 32, "silu"), (83, 11, 218, 1120, 3, 32, "swiglu")],
    (48, 0, 0): [(372, 11, 244, 1632, 1, 128, "silu"), (31, 3, 1208, 1232, 3, 64, "swiglu")],
    (64, 0, 0): [(2397, 4, 36, 1104, 2, 128, "gelu"), (404, 7, 328, 1488, 1, 64, "swiglu")],
    (0, 64, 64): [(300, 4, 1494, 720, 1, 16, "silu"), (1886, 2, 132, 704, 2, 32, "swiglu")],
    (0, 64, 128): [(459, 11, 798, 736, 2, 32, "gelu"), (2952, 6, 74, 736, 3, 64, "swiglu")],
    (0, 128, 128): [(214, 4, 3014, 720, 3, 32, "none"), (207, 4, 2868, 736, 3, 128, "swiglu")],
    (0, 128, 256): [(985, 9, 3782, 944, 1, 128, "gelu"), (466, 9, 4066, 992, 2, 64, "swiglu")],
    (0, 256, 256): [(1550, 5, 2720, 976, 3, 64, "none"), (1334, 6, 5680, 1168, 1, 64, "swiglu")],
}
ALL_LINEAR = [(form, p) for form, ps in LINEAR.items() for p in ps]
ALL_GROUP = [(form, p) for form, ps in GROUP.items() for p in ps]


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


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("form,size", ALL_LINEAR)
def test_every_dense_form(form, size, dtype):
    M, N, K, act = size
    p = Linear(M, N, K, act, dtype=dtype, pad=3)
    p.check(p())
    p = Linear(M, N, K, act, dtype=dtype, bias=False, residual=False)
    p.check(p())


@pytest.mark.parametrize("per_route", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("form,size", ALL_GROUP)
def test_every_grouped_form(form, size, dtype, per_route):
    M, E, N, K, k, bm, act = size
    p = Group(M, E, N, K, k, bm, act, dtype=dtype, per_route=per_route, bias=per_route, pad=3)
    p.check(p())


@pytest.mark.parametrize("M,N,K", [(5, 40, 48), (40, 256, 512), (1366, 34, 720), (4620, 3040, 976)])
def test_dense_products_need_no_workspace(M, N, K):
    p = Linear(M, N, K)
    out = torch.full((M, N), 3.0, dtype=torch.bfloat16, device=DEV)
    moe.moe_i8_linear(p.xq, p.xs, p.w, p.ws, out, p.bias, p.res)
    assert torch.equal(out, p())
