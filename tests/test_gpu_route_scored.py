"""Routing by scores (moe_route_scored) and its gradient against their
definitions in 64 bits.

Tolerances, derived.  The forward computes in 64 bits and rounds a weight once:
half a step of FP32, 2^-24 relative (2^-150 below its normal numbers), and
2^-40 for the roundings in 64 bits.  The choice is compared exactly: logits are
drawn so that no two scores agree to 64-bit rounding unless they are equal.

The gradient is FP32: its value is a product of terms each within a few units of
2^-24 (exp and division within 2 each, sums over at most 64 lanes in 6 levels,
E / 64 additions in a lane, the exponent's argument rounded once, which exp
turns into |argument| 2^-24 relative), applied to the magnitudes that it adds:
(48 + E / 64 + the largest |argument|) 2^-24 of them, then one rounding to the
output's type."""

import numpy as np
import pytest
import torch

import fp8_block_scale_amd as moe
from oracle.router import route_scored_ref, router_ref

pytestmark = pytest.mark.gpu

DEV = "cuda"
SCORE = {"sigmoid": moe.MOE_SCORE_SIGMOID, "softmax": moe.MOE_SCORE_SOFTMAX}
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    torch.cuda.init()


def logits_of(M, E, seed, dtype="f32", spread=1.5, pad=0):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    l = (torch.randn((M, E + pad), generator=g, device=DEV) * spread).to(DT[dtype])
    return l[:, :E]


def bias_of(E, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed + 99)
    return torch.randn(E, generator=g, device=DEV) * 0.05


def route(l, k, score, bias=None, n_shared=0, **kw):
    ids = torch.full((l.shape[0], k + n_shared), -77, dtype=torch.int32, device=DEV)
    w = torch.full((l.shape[0], k + n_shared), -7.0, device=DEV)
    moe.moe_route_scored(l, k, ids, w, SCORE[score], bias=bias, n_shared=n_shared, **kw)
    return ids, w


def check_route(l, k, score, bias=None, **kw):
    ids, w = route(l, k, score, bias, **kw)
    rid, rw = route_scored_ref(l.float().cpu().numpy(), k, score, None if bias is None else bias.cpu().numpy(),
                               **kw)
    assert np.array_equal(ids.cpu().numpy(), rid)
    w = w.double().cpu().numpy()
    assert np.all(np.abs(w - rw) <= (2.0 ** -24 + 2.0 ** -40) * np.abs(rw) + 2.0 ** -149)
    return ids


CASES = [  # M, E, k, score, bias, n_group, topk_group, group_top, renorm, scale, shared, dtype
    (1, 1, 1, "sigmoid", False, 1, 1, 2, True, 1.0, 0, "f32"),
    (1, 1, 1, "softmax", True, 1, 1, 1, False, 2.5, 1, "bf16"),
    (3, 2, 2, "sigmoid", True, 2, 2, 2, True, 1.0, 1, "f16"),
    (5, 8, 2, "softmax", False, 4, 1, 2, False, 1.0, 0, "f32"),
    (16, 256, 8, "sigmoid", True, 8, 4, 2, True, 2.5, 1, "f32"),
    (300, 256, 8, "sigmoid", True, 8, 4, 2, True, 2.5, 1, "bf16"),
    (65, 160, 6, "softmax", False, 8, 3, 1, False, 16.0, 0, "f32"),
    (130, 288, 8, "softmax", True, 1, 1, 2, True, 1.0, 0, "f16"),
    (77, 320, 5, "sigmoid", True, 5, 2, 2, False, -1.0, 0, "f32"),
    (31, 1023, 32, "softmax", True, 11, 4, 2, True, 0.75, 1, "f32"),
    (33, 1024, 32, "sigmoid", True, 64, 2, 1, True, 1.0, 0, "bf16"),
    (9, 1023, 31, "sigmoid", False, 33, 1, 2, True, 1.0, 0, "f32"),
    (40, 512, 10, "softmax", False, 1, 1, 2, False, 1.0, 0, "bf16"),
    (21, 63, 3, "sigmoid", True, 21, 1, 2, True, 1.0, 0, "f32"),
    (12, 65, 7, "softmax", True, 13, 13, 2, False, 1.0, 1, "f32"),
    (4, 64, 1, "sigmoid", True, 64, 1, 2, True, 1.0, 0, "f32"),
]


@pytest.mark.parametrize("M,E,k,score,bias,G,tg,gt,renorm,scale,ns,dtype", CASES)
def test_choice_and_weights(M, E, k, score, bias, G, tg, gt, renorm, scale, ns, dtype):
    l = logits_of(M, E, M + 7 * E, dtype, pad=(M % 3) * 5)
    check_route(l, k, score, bias_of(E, E) if bias else None, n_group=G, topk_group=tg, group_top=gt,
                renorm=renorm, routed_scaling=scale, n_shared=ns)


@pytest.mark.parametrize("score", list(SCORE))
@pytest.mark.parametrize("E,k,G,tg,gt", [(64, 8, 1, 1, 2), (96, 12, 8, 3, 2), (96, 12, 8, 3, 1), (300, 32, 4, 2, 2)])
def test_ties_go_to_the_lowest(score, E, k, G, tg, gt):
    """Few distinct logits, -0 and +0 among them, and few distinct biases: ties of
    experts and of groups everywhere."""
    g = torch.Generator(device=DEV)
    g.manual_seed(E + k)
    l = torch.randint(-2, 3, (200, E), generator=g, device=DEV).float()
    l = torch.where((l == 0) & (torch.rand((200, E), generator=g, device=DEV) < 0.5), -0.0, l)
    check_route(l, k, score, n_group=G, topk_group=tg, group_top=gt)
    check_route(l, k, score, torch.full((E,), 0.25, device=DEV), n_group=G, topk_group=tg, group_top=gt)
    check_route(torch.zeros((3, E), device=DEV), k, score, n_group=G, topk_group=tg, group_top=gt)


@pytest.mark.parametrize("score", list(SCORE))
@pytest.mark.parametrize("E,k,G,tg,gt", [(64, 8, 1, 1, 2), (128, 6, 8, 4, 2), (128, 6, 8, 4, 1), (288, 16, 1, 1, 1)])
@pytest.mark.parametrize("gap", [0.0, 1e-12, 1e-9, 1e-7, 1e-5])
def test_choices_that_nearly_agree(score, E, k, G, tg, gt, gap):
    """Choice scores within some gaps of each other, by a bias that evens the
    scores out as far as FP32 goes, and by logits that differ by little."""
    g = torch.Generator(device=DEV)
    g.manual_seed(E + k)
    l = torch.randn((1, E), generator=g, device=DEV) * 2
    s = torch.sigmoid(l.double()) if score == "sigmoid" else torch.softmax(l.double(), 1)
    bias = (0.5 - s + gap * torch.randn((1, E), generator=g, device=DEV).double())[0].float()
    kw = dict(n_group=G, topk_group=tg, group_top=gt)
    check_route(l, k, score, bias, **kw)
    for base in (0.0, 1.0, -30.0):
        near = (base + gap * torch.randn((40, E), generator=g, device=DEV).double()).float()
        check_route(near, k, score, **kw)
        check_route(near, k, score, torch.zeros(E, device=DEV), **kw)


@pytest.mark.parametrize("score", list(SCORE))
def test_wide_logits(score):
    """Far apart: scores that underflow in FP32, and beyond where 64 bits tell them apart."""
    for spread in (15.0, 80.0, 300.0, 900.0):
        l = torch.linspace(-1, 1, 96, device=DEV).repeat(3, 1) * spread
        l = l[:, torch.randperm(96, generator=torch.Generator().manual_seed(3)).to(DEV)].contiguous()
        check_route(l, 12, score)
        check_route(l, 12, score, n_group=8, topk_group=2)
        check_route(l, 12, score, bias_of(96, 1), n_group=8, topk_group=4)


def test_softmax_renormalised_is_the_plan_router():
    l = logits_of(500, 288, 4)
    ids, w = route(l, 8, "softmax", n_shared=1, routed_scaling=2.5)
    rid, rw = router_ref(l.cpu().numpy(), 8, 1, 2.5)
    assert np.array_equal(ids.cpu().numpy(), rid)
    assert np.all(np.abs(w.double().cpu().numpy() - rw) <= 2.0 ** -23 * rw)


@pytest.mark.parametrize("score", list(SCORE))
@pytest.mark.parametrize("renorm", [False, True])
def test_masked_experts(score, renorm):
    """-infinity and NaN logits are never chosen; rows with fewer experts than
    slots, and with none; +infinity; far apart and far below zero."""
    inf, nan = float("inf"), float("nan")
    l = logits_of(12, 16, 3)
    l[0, :] = -inf
    l[1, :] = nan
    l[2, 3:] = -inf
    l[3, ::2] = nan
    l[4, 5] = inf
    l[5, 5] = l[5, 9] = inf
    l[6, :] = -200.0 - torch.arange(16, device=DEV)
    l[7, :] = -1000.0
    l[7, 2] = -990.0
    l[8, :8] = -inf
    l[9, :] = -3.0e38
    l[10, :] = torch.linspace(-30, 30, 16, device=DEV)
    for kw in (dict(), dict(n_group=4, topk_group=2), dict(n_group=4, topk_group=1, group_top=1)):
        check_route(l, 4, score, renorm=renorm, n_shared=1, **kw)
    bias = torch.zeros(16, device=DEV)
    bias[4] = -inf
    bias[7] = nan
    bias[11] = inf
    bias[12] = -5.0
    check_route(l, 4, score, bias, renorm=renorm, n_group=4, topk_group=2)


def test_a_bias_moves_the_choice_and_no_weight():
    l = torch.tensor([[1.0, 0.5, 0.0, -0.5]], device=DEV)
    ids, w = route(l, 2, "sigmoid", torch.tensor([0.0, 0.0, 0.0, 1.0], device=DEV), renorm=False)
    assert ids.tolist() == [[3, 0]]
    ref = torch.sigmoid(l.double()[0, [3, 0]])
    assert ((w[0].double() - ref).abs() <= 2.0 ** -24 * ref * 1.001).all()


# ----------------------------------------------------------------- gradient --

def weights64(l, ids, score, renorm, scale):
    """The weights of these slots in 64 bits, differentiable."""
    E = l.shape[1]
    ok = (ids >= 0) & (ids < E)
    at = ids.long().clamp(0, E - 1)
    z = l.gather(1, at)
    dead = z == -float("inf")
    ok = ok & ~dead.detach()
    if score == "sigmoid":
        w = torch.where(ok, torch.sigmoid(z), 0.0)
        if renorm:
            w = w / w.sum(1, keepdim=True).clamp_min(1e-300)
    elif renorm:
        z = torch.where(ok, z, -1e300)
        w = torch.where(ok, torch.softmax(z, 1), 0.0)
    else:
        w = torch.where(ok, torch.softmax(l, 1).gather(1, at), 0.0)
    return w * scale


def bwd(l, ids, dw, score, renorm, scale, pad=0):
    d = torch.full((l.shape[0], l.shape[1] + pad), 7.0, dtype=l.dtype, device=DEV)
    moe.moe_route_scored_bwd(l, ids, dw, d[:, :l.shape[1]], SCORE[score], renorm=renorm, routed_scaling=scale)
    assert (d[:, l.shape[1]:] == 7.0).all()
    return d[:, :l.shape[1]]


def check_bwd(l, ids, dw, score, renorm, scale, pad=0):
    got = bwd(l, ids, dw, score, renorm, scale, pad).double()
    l64 = l.double().requires_grad_(True)
    (ref,) = torch.autograd.grad((weights64(l64, ids, score, renorm, scale) * dw.double()).sum(), l64)
    ref = torch.nan_to_num(ref, 0.0)
    # the magnitudes that are added: |value factor| (|a_j| + sum |a| p)
    E = l.shape[1]
    ok = (ids >= 0) & (ids < E)
    at = ids.long().clamp(0, E - 1)
    z = torch.where(ok, l.double().gather(1, at), -float("inf"))
    a = torch.where(ok, dw.double().abs() * abs(scale), 0.0)
    if score == "softmax" and not renorm:
        p = torch.softmax(l.double(), 1)
        mag = p * (torch.zeros_like(p).scatter_add_(1, at, a) + (a * p.gather(1, at)).sum(1, keepdim=True))
        arg = (l.double() - l.double().amax(1, keepdim=True)).abs().clamp(max=110).amax()
    else:
        s = torch.sigmoid(z) if score == "sigmoid" else torch.softmax(z.clamp_min(-1e300), 1)
        s = torch.where(ok, s, 0.0)
        f = torch.where(ok, s * torch.sigmoid(-z), 0.0) if score == "sigmoid" else s
        if renorm or score == "softmax":
            S = s.sum(1, keepdim=True).clamp_min(1e-300)
            v = f * (a + (a * s).sum(1, keepdim=True) / S) / S
        else:
            v = f * a
        mag = torch.zeros_like(ref).scatter_add_(1, at, torch.where(ok, v, 0.0))
        arg = torch.where(ok, z, 0.0).abs().clamp(max=110).amax() * 2
    half = torch.finfo(l.dtype).eps / 2
    tiny = {torch.float32: 2.0 ** -120, torch.bfloat16: 2.0 ** -120, torch.float16: 2.0 ** -25}[l.dtype]
    tol = half * ref.abs() + (48 + E / 64 + arg) * 2.0 ** -24 * mag * (1 + half) + tiny
    err = (got - ref).abs()
    assert (err <= tol).all(), (err / tol).max().item()
    return got


@pytest.mark.parametrize("score", list(SCORE))
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("M,E,k,ns,dtype,pad", [(1, 1, 1, 0, "f32", 0), (7, 8, 2, 1, "bf16", 3), (130, 256, 8, 1, "f32", 0),
                                               (66, 288, 8, 0, "f16", 8), (33, 513, 10, 0, "bf16", 1),
                                               (10, 1023, 32, 1, "f32", 0), (5, 64, 32, 1, "f16", 0)])
def test_gradient(score, renorm, M, E, k, ns, dtype, pad):
    l = logits_of(M, E, M + E, dtype, pad=pad)
    ids, _ = route(l, k, score, bias_of(E, 5), n_shared=ns, renorm=renorm)
    g = torch.Generator(device=DEV)
    g.manual_seed(k)
    dw = torch.randn(ids.shape, generator=g, device=DEV)
    d = check_bwd(l, ids, dw, score, renorm, 2.5, pad)
    if score == "softmax":  # adding a number to all logits changes nothing
        assert (d.sum(1).abs() <= (2.0 ** -8 + 2.0 ** -12) * d.abs().sum(1) + 1e-6).all()


@pytest.mark.parametrize("score", list(SCORE))
@pytest.mark.parametrize("renorm", [False, True])
def test_gradient_of_any_ids(score, renorm):
    """Masked slots, a row of them, an expert listed twice, ids beyond the
    experts, and logits of -infinity (chosen or not)."""
    l = logits_of(6, 12, 8)
    l[4, 3] = -float("inf")
    ids = torch.tensor([[0, -1, 5], [-1, -1, -1], [7, 7, 2], [12, 900, 3], [3, 4, 5], [11, 0, 2 ** 31 - 1]],
                       dtype=torch.int32, device=DEV)
    dw = torch.tensor([[1.0, 50.0, -2.0]] * 6, device=DEV)
    got = bwd(l, ids, dw, score, renorm, 1.5).double()
    l64 = l.double().requires_grad_(True)
    (ref,) = torch.autograd.grad((weights64(l64, ids, score, renorm, 1.5) * dw.double()).sum(), l64)
    ref = torch.nan_to_num(ref, 0.0)
    assert torch.isfinite(got).all()
    # magnitudes at most 50 * 1.5 * 2: (48 + 12 / 64 + 8) 2^-24 of it
    assert ((got - ref).abs() <= 57 * 2.0 ** -24 * 150).all()
    assert (got[1] == 0).all()


@pytest.mark.parametrize("score", list(SCORE))
@pytest.mark.parametrize("renorm", [False, True])
def test_gradient_by_differences(score, renorm):
    """Against differences of the forward's own weights with the ids held."""
    l = logits_of(4, 16, 21)
    ids, _ = route(l, 4, score, renorm=renorm)
    dw = torch.randn(ids.shape, generator=torch.Generator(device=DEV).manual_seed(2), device=DEV)
    d = bwd(l, ids, dw, score, renorm, 1.0).double()
    h = 2.0 ** -10
    for e in range(16):
        lp, lm = l.double().clone(), l.double().clone()
        lp[:, e] += h
        lm[:, e] -= h
        diff = ((weights64(lp, ids, score, renorm, 1.0) - weights64(lm, ids, score, renorm, 1.0)) * dw.double()).sum(1) / (2 * h)
        # third derivatives of these weights are below 1: h^2 / 6 times sum |dw|
        assert ((diff - d[:, e]).abs() <= (h * h + 1e-5) * dw.abs().sum(1).double()).all()


@pytest.mark.parametrize("renorm", [False, True])
def test_gradient_far_from_zero(renorm):
    l = torch.tensor([[60.0, -60.0, 20.0, 3.0], [-200.0, -201.0, -199.5, -900.0], [-95.0, -96.0, 0.0, 1.0]], device=DEV)
    ids = torch.tensor([[0, 1, 2], [0, 1, 2], [0, 1, 1]], dtype=torch.int32, device=DEV)
    dw = torch.tensor([[1.0, -2.0, 3.0]] * 3, device=DEV)
    for score in SCORE:
        got = bwd(l, ids, dw, score, renorm, 1.0).double()
        l64 = l.double().requires_grad_(True)
        (ref,) = torch.autograd.grad((weights64(l64, ids, score, renorm, 1.0) * dw.double()).sum(), l64)
        # exponents up to 900 whose rounding exp multiplies: 2^-24 * 260 where the value is not below FP32
        assert ((got - ref).abs() <= 2.0 ** -15 * ref.abs() + 2.0 ** -23).all(), (score, got, ref)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("score", list(SCORE))
def test_gradient_of_a_single_choice(score, dtype):
    """Renormalised, one expert's weight is the scale whatever its logit."""
    l = logits_of(200, 40, 3, dtype)
    ids, w = route(l, 1, score, renorm=True)
    dw = torch.randn(ids.shape, generator=torch.Generator(device=DEV).manual_seed(1), device=DEV)
    assert (bwd(l, ids, dw, score, True, 2.5) == 0).all()
    wide = torch.full((200, 20), -1, dtype=torch.int32, device=DEV)
    wide[:, 17] = ids[:, 0]
    assert (bwd(l, wide, dw.expand(200, 20).contiguous(), score, True, 2.5) == 0).all()


@pytest.mark.parametrize("slots", [4, 16, 20])
@pytest.mark.parametrize("score", list(SCORE))
def test_gradient_beside_a_dominant_choice(score, slots):
    """One slot holds nearly the whole sum.  Its gradient is s' / S^2 sum_j s_j (a_i -
    a_j): against the magnitudes of that sum (scale 1: the differences have one
    rounding), not against those of a_i, 2^17 times larger."""
    g = torch.Generator(device=DEV).manual_seed(slots)
    l = torch.randn((300, 40), generator=g, device=DEV) - 12
    ids = torch.rand((300, 40), generator=g, device=DEV).argsort(1)[:, :slots].to(torch.int32).contiguous()
    l.scatter_(1, ids[:, 1:2].long(), 0.25)
    dw = torch.randn(ids.shape, generator=g, device=DEV)
    got = bwd(l, ids, dw, score, True, 1.0).double().gather(1, ids.long())
    z, a = l.double().gather(1, ids.long()), dw.double()
    s = torch.sigmoid(z) if score == "sigmoid" else torch.softmax(z, 1)
    f = (s * torch.sigmoid(-z) if score == "sigmoid" else s) / s.sum(1, keepdim=True) ** 2
    diff = a[:, :, None] - a[:, None, :]
    ref, mag = f * (diff * s[:, None, :]).sum(2), f * (diff.abs() * s[:, None, :]).sum(2)
    assert ((got - ref).abs() <= (48 + 2 * 20) * 2.0 ** -24 * mag).all()


def test_graph_streams_and_bits():
    l = logits_of(700, 256, 1, "bf16")
    bias = bias_of(256, 1)
    ids, w = route(l, 8, "sigmoid", bias, n_group=8, topk_group=4, n_shared=1)
    dw = torch.randn(ids.shape, device=DEV)
    d = bwd(l, ids, dw, "sigmoid", True, 1.0)
    ids2, w2, d2 = torch.zeros_like(ids), torch.zeros_like(w), torch.zeros_like(d)

    def both(stream=None):
        moe.moe_route_scored(l, 8, ids2, w2, SCORE["sigmoid"], bias=bias, n_group=8, topk_group=4, n_shared=1,
                             stream=stream)
        moe.moe_route_scored_bwd(l, ids2, dw, d2, SCORE["sigmoid"], stream=stream)

    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        both()
    for _ in range(3):
        for t in (ids2, w2, d2):
            t.fill_(3)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(ids, ids2) and torch.equal(w, w2) and torch.equal(d, d2)
    for t in (ids2, w2, d2):
        t.fill_(3)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    both(s)
    s.synchronize()
    assert torch.equal(ids, ids2) and torch.equal(w, w2) and torch.equal(d, d2)


def test_no_tokens():
    l = torch.empty((0, 8), device=DEV)
    ids, w = route(l, 2, "sigmoid")
    moe.moe_route_scored_bwd(l, ids, w, torch.empty((0, 8), device=DEV))


def test_more_tokens_than_a_launch_counts():
    """More workgroups than a launch takes: the kernels go round (67.2 million tokens
    whose logits repeat every 1000)."""
    n, times = 1000, 67200
    l = logits_of(n, 8, 17, "bf16")
    ids, w = route(l, 2, "sigmoid")
    dw = torch.randn(ids.shape, generator=torch.Generator(device=DEV).manual_seed(3), device=DEV)
    d = bwd(l, ids, dw, "sigmoid", True, 1.0)
    dd = bwd(l, ids, dw, "softmax", False, 1.0)
    big = l.repeat(times, 1)
    bi, bw = route(big, 2, "sigmoid")
    assert (bi.view(times, -1) == ids.view(1, -1)).all() and (bw.view(times, -1) == w.view(1, -1)).all()
    bdw = dw.repeat(times, 1)
    assert (bwd(big, bi, bdw, "sigmoid", True, 1.0).view(times, -1) == d.reshape(1, -1)).all()
    assert (bwd(big, bi, bdw, "softmax", False, 1.0).view(times, -1) == dd.reshape(1, -1)).all()
