"""The operators around the experts as they are used together.

Serving: route by scores, plan, quantise the tokens, 8-bit gate/up with SwiGLU,
quantise the routes' rows, 8-bit down product, weighted sum with the residual --
against the same chain in 64 bits that takes over the codes (their rounding is
tested elsewhere).  Training: route, plan, 16-bit grouped products, weighted sum,
and the gradients back to x, the weights and the router's logits, against
differentiating the formula in 64 bits and against differences."""

import pytest
import torch

import fp8_block_scale_amd as moe
from oracle import plan_ref, route_scored_ref

pytestmark = pytest.mark.gpu

DEV = "cuda"
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    torch.cuda.init()


def plan_of(ids, E, bm):
    M, k = ids.shape
    sc, bc = moe.moe_plan_capacity(M, k, E, bm)
    p = (torch.zeros(sc, dtype=torch.int32, device=DEV), torch.zeros(bc, dtype=torch.int32, device=DEV),
         torch.zeros(1, dtype=torch.int32, device=DEV))
    n = moe.moe_plan_workspace_size(M, k, E, bm)
    moe.moe_plan(ids, E, bm, *p, workspace=torch.empty(n, dtype=torch.uint8, device=DEV) if n else None)
    return p


def ws(n):
    return torch.empty(max(n, 256), dtype=torch.uint8, device=DEV)


@pytest.mark.parametrize("M,Er,k,K,I,bm,ns", [(1, 32, 4, 512, 256, 16, 1), (37, 16, 3, 256, 144, 32, 0),
                                              (900, 24, 4, 768, 272, 64, 1)])
def test_int8_layer(M, Er, k, K, I, bm, ns):
    g = torch.Generator(device=DEV)
    g.manual_seed(M)
    E, kk = Er + ns, k + ns
    x = torch.randn((M, K), generator=g, device=DEV).to(BF)
    wg = torch.randn((Er, K), generator=g, device=DEV) / K ** 0.5
    bias = torch.randn(Er, generator=g, device=DEV) * 0.02
    q13, s13 = torch.empty((E * 2 * I, K), dtype=torch.int8, device=DEV), torch.empty(E * 2 * I, device=DEV)
    moe.moe_quant_i8((torch.randn((E * 2 * I, K), generator=g, device=DEV) * K ** -0.5).to(BF), q13, s13)
    q2, s2 = torch.empty((E * K, I), dtype=torch.int8, device=DEV), torch.empty(E * K, device=DEV)
    moe.moe_quant_i8((torch.randn((E * K, I), generator=g, device=DEV) * I ** -0.5).to(BF), q2, s2)
    w13, w2 = (q13.view(E, 2 * I, K), s13.view(E, 2 * I)), (q2.view(E, K, I), s2.view(E, K))

    logits = x.float() @ wg.t()
    ids = torch.empty((M, kk), dtype=torch.int32, device=DEV)
    tw = torch.empty((M, kk), device=DEV)
    h = torch.full((M * kk, I), 9.0, dtype=BF, device=DEV)
    y = torch.full((M * kk, K), 9.0, dtype=BF, device=DEV)
    xq, xs = torch.empty((M, K), dtype=torch.int8, device=DEV), torch.empty(M, device=DEV)
    hq, hs = torch.empty((M * kk, I), dtype=torch.int8, device=DEV), torch.empty(M * kk, device=DEV)
    out = torch.empty((M, K), dtype=BF, device=DEV)
    cap = moe.moe_plan_capacity(M, kk, E, bm)[0]
    work = ws(max(moe.moe_i8_group_mm_workspace_size(M, K, 2 * I, E, kk, bm, cap, moe.MOE_ACT_SWIGLU),
                  moe.moe_i8_group_mm_workspace_size(M, I, K, E, kk, bm, cap, x_per_route=True)))
    moe.moe_route_scored(logits, k, ids, tw, bias=bias, n_group=4, topk_group=2, routed_scaling=1.5, n_shared=ns)
    plan = plan_of(ids, E, bm)
    moe.moe_quant_i8(x, xq, xs)
    moe.moe_i8_group_mm(xq, xs, *w13, *plan, kk, bm, h, act=moe.MOE_ACT_SWIGLU, workspace=work, x_per_route=False)
    moe.moe_quant_i8(h, hq, hs)
    moe.moe_i8_group_mm(hq, hs, *w2, *plan, kk, bm, y, workspace=work, x_per_route=True)
    moe.moe_combine(y, tw, out, ids, E, residual=x)

    rid, rw = route_scored_ref(logits.cpu().numpy(), k, "sigmoid", bias.cpu().numpy(), 4, 2, routed_scaling=1.5,
                               n_shared=ns)
    assert (ids.cpu().numpy() == rid).all()
    rs, rx, P = plan_ref(rid, E, bm)
    assert int(plan[2]) == P and (plan[0][:P].cpu().numpy() == rs).all()
    ref = x.double()
    xd, hd = xq.double() * xs.double()[:, None], hq.double() * hs.double()[:, None]
    for t in range(M) if M < 100 else range(0, M, 97):
        acc, mag = x[t].double(), torch.zeros(K, dtype=torch.float64, device=DEV)
        for j in range(kk):
            e, r = int(rid[t, j]), t * kk + j
            z = (w13[0][e].double() * w13[1][e].double()[:, None]) @ xd[t]
            a = z[:I] * torch.sigmoid(z[:I]) * z[I:]
            # SwiGLU in FP32 (2^-16 of the terms covers it) and one rounding to BF16
            assert ((h[r].double() - a).abs() <= 2.0 ** -8 * a.abs() + 2.0 ** -16 * (z[:I].abs() * z[I:].abs() + 2.0 ** -16)).all()
            d = (w2[0][e].double() * w2[1][e].double()[:, None]) @ hd[r]
            acc = acc + float(rw[t, j]) * d
            mag = mag + abs(float(rw[t, j])) * d.abs()
        # each route's row is rounded to BF16 once, and the sum once more
        assert ((out[t].double() - acc).abs() <= 2.0 ** -8 * acc.abs() + (2.0 ** -8 + 2.0 ** -16) * mag + 2.0 ** -16).all()


@pytest.mark.parametrize("score,renorm", [("sigmoid", True), ("sigmoid", False), ("softmax", True), ("softmax", False)])
def test_training_step(score, renorm):
    """out = residual + sum_j w_j (x W_e^T): gradients of x, W and the logits."""
    M, E, k, K, N, bm = 60, 8, 3, 64, 48, 16
    f16 = torch.float16
    code = moe.MOE_SCORE_SIGMOID if score == "sigmoid" else moe.MOE_SCORE_SOFTMAX
    g = torch.Generator(device=DEV)
    g.manual_seed(5)
    x = torch.randn((M, K), generator=g, device=DEV).to(f16)
    W = (torch.randn((E, N, K), generator=g, device=DEV) / 8).to(f16)
    logits = torch.randn((M, E), generator=g, device=DEV)
    res = torch.randn((M, N), generator=g, device=DEV).to(f16)
    dout = torch.randn((M, N), generator=g, device=DEV).to(f16)
    ids, tw = torch.empty((M, k), dtype=torch.int32, device=DEV), torch.empty((M, k), device=DEV)
    moe.moe_route_scored(logits, k, ids, tw, code, renorm=renorm)
    plan = plan_of(ids, E, bm)
    cap = plan[0].numel()
    work = ws(max(moe.moe_group_mm_workspace_size(op, M, K, N, E, k, bm, cap)
                  for op in (moe.MOE_GMM_FWD, moe.MOE_GMM_DX, moe.MOE_GMM_DW)))
    y, out = torch.zeros((M * k, N), dtype=f16, device=DEV), torch.zeros((M, N), dtype=f16, device=DEV)
    moe.moe_group_mm(x, W, *plan, k, bm, y, work, x_per_route=False)
    moe.moe_combine(y, tw, out, ids, E, residual=res)
    dy, dw = torch.zeros_like(y), torch.zeros_like(tw)
    dl, dx = torch.zeros_like(logits), torch.zeros_like(x)
    dW = torch.zeros((E, N, K), dtype=torch.float32, device=DEV)
    moe.moe_combine_bwd(dout, y, tw, dy, dw, ids, E)
    moe.moe_route_scored_bwd(logits, ids, dw, dl, code, renorm=renorm)
    moe.moe_group_mm_dx(dy, W, *plan, k, bm, dx, work, x_per_route=False)
    moe.moe_group_mm_dw(dy, x, *plan, k, bm, dW, work, x_per_route=False)

    def formula(x, W, l):
        z = l.gather(1, ids.long())
        if score == "sigmoid":
            w = torch.sigmoid(z)
            w = w / w.sum(1, keepdim=True) if renorm else w
        else:
            w = torch.softmax(z, 1) if renorm else torch.softmax(l, 1).gather(1, ids.long())
        rows = torch.stack([(W[ids[:, j].long()] * x[:, None, :]).sum(2) for j in range(k)], 1)
        return res.double() + (w[..., None] * rows).sum(1)

    a = [t.double().requires_grad_(True) for t in (x, W, logits)]
    o = formula(*a)
    rdx, rdW, rdl = torch.autograd.grad((o * dout.double()).sum(), a)
    # FP16 rows (2^-11 each) enter linearly: y, dy, then the results' own rounding;
    # the 2-norm of independent roundings stays within 2^-11 of the terms' norm each
    def near(got, ref, steps):
        assert (got.double() - ref).norm() <= steps * 2.0 ** -11 * ref.norm(), \
            ((got.double() - ref).norm() / ref.norm()).item()

    near(out, o, 3)
    near(dx, rdx, 3)
    near(dW, rdW, 2)
    # differences of experts' scalar products: their terms' norm, not the result's
    rows = torch.stack([(W.double()[ids[:, j].long()] * x.double()[:, None, :]).sum(2) for j in range(k)], 1)
    scale = (rows.abs() * dout.double().abs()[:, None]).sum()
    assert (dl.double() - rdl).abs().sum() <= 2 * 2.0 ** -11 * scale
    # by differences, along one random direction of the logits
    with torch.no_grad():
        v = torch.randn((M, E), generator=g, device=DEV, dtype=torch.float64)
        h = 1e-4
        d = ((formula(a[0], a[1], a[2] + h * v) - formula(a[0], a[1], a[2] - h * v)) * dout.double()).sum() / (2 * h)
    assert (d - (dl.double() * v).sum()).abs() <= 2 * 2.0 ** -11 * scale * v.abs().max() + 1e-3
