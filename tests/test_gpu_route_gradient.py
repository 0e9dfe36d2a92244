"""moe_route_scored_bwd where terms of its formula nearly cancel, against the
formula in 64 bits with the differences taken first.

Tolerances, derived, in units of 2^-24 and relative to the magnitudes of the
differences.  A weight p: exp 2, its argument's rounding |argument|, the sum over E
experts E / 64 + 6, a division and a product 2: at most |argument| + E / 64 + 10.
A term has two of them, a difference (1), a product (1) and at most `slots` + 6
additions.  Together 2 |argument| + E / 32 + slots + 28 <= 2 |argument| + E / 32 +
slots + 40.  d_weights are small multiples of 2^-6, so that the sums over slots of
one expert are exact."""

import pytest
import torch

import fp8_block_scale_amd as moe

pytestmark = pytest.mark.gpu

DEV = "cuda"
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    torch.cuda.init()


def inputs(M, E, slots, dtype, seed, gap):
    """Logits with one expert `gap` above about the mean, ids without repetition, the
    dominant expert first in two tokens of three, in no slot in the third."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    l = torch.randn((M, E), generator=g, device=DEV)
    ids = torch.rand((M, E), generator=g, device=DEV).argsort(1)
    top = torch.where(torch.arange(M, device=DEV) % 3 < 2, ids[:, 0], ids[:, -1])
    l.scatter_(1, top[:, None], gap)
    dw = torch.randint(-200, 201, (M, slots), generator=g, device=DEV).float() / 64
    return l.to(DT[dtype]), ids[:, :slots].to(torch.int32).contiguous(), dw


def softmax_ref(l, ids, dw):
    """(dl, the magnitudes that it adds): p_e sum_f p_f (A_e - A_f)"""
    z = l.double()
    p = torch.softmax(z, 1)
    ok = (ids >= 0) & (ids < l.shape[1])
    at = torch.where(ok, ids, 0).long()
    A = torch.zeros_like(p).scatter_add_(1, at, torch.where(ok, dw.double(), 0.0))
    hit = torch.zeros_like(p).scatter_add_(1, at, ok.double()) > 0
    # over the experts in a slot, the others together (their A is 0)
    rest = torch.where(hit, 0.0, p).sum(1, keepdim=True)
    ref, mag = A * rest, A.abs() * rest
    for t in range(l.shape[0]):
        f = torch.nonzero(hit[t]).flatten()
        d = A[t][:, None] - A[t][f][None, :]
        ref[t] += (d * p[t][f]).sum(1)
        mag[t] += (d.abs() * p[t][f]).sum(1)
    return p * ref, p * mag


def check_softmax(l, ids, dw):
    d = torch.full_like(l, 7.0)
    moe.moe_route_scored_bwd(l, ids, dw, d, moe.MOE_SCORE_SOFTMAX, renorm=False)
    ref, mag = softmax_ref(l, ids, dw)
    z = l.double()
    arg = (z - z.amax(1, keepdim=True)).abs().amax()
    half = torch.finfo(l.dtype).eps / 2 if l.dtype != torch.float32 else 0.0
    tiny = 2.0 ** -25 if l.dtype == torch.float16 else 2.0 ** -130
    tol = half * ref.abs() + (2 * arg + l.shape[1] / 32 + ids.shape[1] + 40) * 2.0 ** -24 * mag * (1 + half) + tiny
    err = (d.double() - ref).abs()
    assert (err <= tol).all(), (err / tol).max().item()


@pytest.mark.parametrize("gap", [9.0, 17.0, 40.0])
@pytest.mark.parametrize("E,slots", [(40, 1), (40, 4), (130, 17), (512, 10), (1000, 33)])
def test_softmax_beside_a_dominant_expert(E, slots, gap):
    """The dominant expert's gradient is p times the rest's sum of differences: small
    beside d_weights, and no difference of numbers of their size."""
    check_softmax(*inputs(60, E, slots, "f32", E + slots, gap))


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_softmax_beside_a_dominant_expert_16_bits(dtype):
    check_softmax(*inputs(60, 288, 8, dtype, 3, 12.0))


def test_softmax_with_the_dominant_expert_listed_twice():
    l, ids, dw = inputs(90, 64, 6, "f32", 5, 17.0)
    ids[:, 3] = ids[:, 0]
    ids[::2, 4] = ids[::2, 1]
    ids[1::4, 5] = -1
    ids[2::4, 2] = 64
    check_softmax(l, ids, dw)


def renormalised_ref(l, ids, dw, score):
    """(dl, the magnitudes that it adds): sum_{j: e_j = e} f_j sum_{i: e_i != e} s_i
    (a_j - a_i), the differences between slots of one expert, which cancel, left out"""
    z, a = l.double().gather(1, ids.long()), dw.double()
    s = torch.sigmoid(z) if score == "sigmoid" else torch.softmax(z, 1)
    f = (s * torch.sigmoid(-z) if score == "sigmoid" else s) / s.sum(1, keepdim=True) ** 2
    d = a[:, :, None] - a[:, None, :]
    d = torch.where(ids[:, :, None] == ids[:, None, :], 0.0, d) * s[:, None, :]
    ref, mag = torch.zeros_like(l, dtype=torch.float64), torch.zeros_like(l, dtype=torch.float64)
    return ref.scatter_add_(1, ids.long(), f * d.sum(2)), mag.scatter_add_(1, ids.long(), f * d.abs().sum(2))


@pytest.mark.parametrize("slots", [2, 4, 16, 20])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("gap", [5.0, 17.0])
def test_renormalised_with_the_dominant_expert_listed_twice(score, slots, gap):
    """Its two slots' weights hold nearly the whole sum: what they take from each other
    is far more than their expert's gradient."""
    l, ids, dw = inputs(90, 40, slots, "f32", slots, gap)
    l -= 12
    ids[:, -1] = ids[:, 0]
    if slots > 3:
        ids[::2, 2] = ids[::2, 1]
    d = torch.full_like(l, 7.0)
    moe.moe_route_scored_bwd(l, ids, dw, d, {"softmax": moe.MOE_SCORE_SOFTMAX, "sigmoid": moe.MOE_SCORE_SIGMOID}[score])
    ref, mag = renormalised_ref(l, ids, dw, score)
    arg = l.abs().amax().item()
    tol = (2 * arg + slots + 40 + slots) * 2.0 ** -24 * mag + 2.0 ** -130      # (and a slot's sum over its expert's slots)
    err = (d.double() - ref).abs()
    assert (err <= tol).all(), (err / tol).max().item()
