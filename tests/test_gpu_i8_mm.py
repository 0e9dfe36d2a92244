"""8-bit integer codes of rows (moe_quant_i8) and their products, dense
(moe_i8_linear) and grouped by expert (moe_i8_group_mm), against their formulas
in 64 bits.

Tolerances, derived.  The codes are compared exactly: FP32 division, product and
rounding are IEEE operations on both sides.  The products' sums are exact
integers; turning one into FP32, times two scales, plus the bias is at most 4
roundings of 2^-24 of the product's magnitude and one of the sum's.  The
activations have slope at most 1.13 (SwiGLU: the product rule) and are evaluated
within 2^-18 of their value and argument; a residual adds one rounding, and the
result is rounded once (half a step: 2^-8 BF16, 2^-11 FP16, 2^-25 below FP16's
normal numbers)."""

import math

import numpy as np
import pytest
import torch

import fp8_block_scale_amd as moe

pytestmark = pytest.mark.gpu

DEV = "cuda"
DT = {"bf16": torch.bfloat16, "f16": torch.float16}
ACTS = {"none": moe.MOE_ACT_NONE, "silu": moe.MOE_ACT_SILU, "gelu": moe.MOE_ACT_GELU,
        "swiglu": moe.MOE_ACT_SWIGLU}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    torch.cuda.init()


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


# -------------------------------------------------------------------- codes --

def quant(x):
    q = torch.full(x.shape, 99, dtype=torch.int8, device=DEV)
    s = torch.full((x.shape[0],), -1.0, device=DEV)
    moe.moe_quant_i8(x, q, s)
    return q, s


def quant_ref(x):
    f = x.float().cpu().numpy()
    s = np.maximum(np.abs(f).max(axis=1) / np.float32(127), np.float32(2.0 ** -126)).astype(np.float32)
    f = np.where(np.isfinite(s)[:, None], f, 0)  # (rows that are not finite: codes 0)
    return np.rint(f * (np.float32(1) / s)[:, None]).astype(np.int8), s


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("M,K,pad", [(1, 16, 0), (3, 48, 8), (5, 256, 0), (4, 2048, 16), (7, 2064, 0), (9, 4096, 8),
                                     (2, 7168, 0), (3, 8192, 0), (2, 8208, 8), (1, 131056, 0), (1001, 512, 0)])
def test_codes(M, K, pad, dtype):
    g = gen(M + K)
    x = torch.randn((M, K + pad), generator=g, device=DEV) * torch.exp(torch.randn((M, 1), generator=g, device=DEV) * 3)
    x = x.to(DT[dtype])[:, :K]
    q, s = quant(x)
    rq, rs = quant_ref(x)
    assert np.array_equal(s.cpu().numpy(), rs) and np.array_equal(q.cpu().numpy(), rq)


@pytest.mark.parametrize("dtype", list(DT))
def test_codes_at_the_edges(dtype):
    """Zero rows, one value, ties, the largest and smallest values of the type."""
    x = torch.zeros((6, 64), dtype=DT[dtype], device=DEV)
    x[1, 63] = -2.0
    x[2] = torch.arange(64, device=DEV).to(x.dtype) - 32.5
    x[2, 0] = 127.0                              # scale 1: every half is a tie
    x[3] = torch.finfo(x.dtype).max
    x[4, 5] = 2.0 ** -24 if dtype == "f16" else 2.0 ** -133
    x[5] = -0.0
    q, s = quant(x)
    rq, rs = quant_ref(x)
    assert np.array_equal(s.cpu().numpy(), rs) and np.array_equal(q.cpu().numpy(), rq)


def test_rows_that_are_not_finite():
    x = torch.ones((5, 32), dtype=torch.bfloat16, device=DEV)
    x[1, 3], x[2, 31], x[3, 0] = float("inf"), float("nan"), -float("inf")
    q, s = quant(x)
    assert (q[1:4] == 0).all() and (q[0] == 127).all() and (q[4] == 127).all()
    assert torch.isfinite(s).tolist() == [True, False, False, False, True]
    w = torch.ones((8, 32), dtype=torch.int8, device=DEV)
    out = torch.zeros((5, 8), dtype=torch.bfloat16, device=DEV)
    moe.moe_i8_linear(q, s, w, torch.ones(8, device=DEV), out)
    assert torch.isnan(out[1:4]).all() and torch.isfinite(out[0]).all() and torch.isfinite(out[4]).all()


def test_more_rows_than_a_launch_counts():
    """More workgroups than a launch takes: the kernel goes round (33.6 million rows
    that repeat every 1000)."""
    x = torch.randn((1000, 16), generator=gen(1), device=DEV).to(torch.bfloat16)
    q, s = quant(x)
    bq, bs = quant(x.repeat(33600, 1))
    assert (bq.view(33600, -1) == q.view(1, -1)).all() and (bs.view(33600, -1) == s.view(1, -1)).all()


# ----------------------------------------------------------------- products --

def codes(shape, g):
    return torch.randint(-128, 128, shape, generator=g, device=DEV, dtype=torch.int32).to(torch.int8)


def epilogue64(z, mag, act, bias, res):
    """(result, bound of the error before the last rounding)"""
    d = 4 * 2.0 ** -24 * mag
    if bias is not None:
        z = z + bias.double()
        d = d + 2.0 ** -24 * z.abs()
    if act == "silu":
        d, z = 1.13 * d + 2.0 ** -18 * z.abs(), z * torch.sigmoid(z)
    elif act == "gelu":
        u = math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)
        d, z = 1.13 * d + 2.0 ** -18 * z.abs(), 0.5 * z * (1 + torch.tanh(u))
    elif act == "swiglu":
        gt, up = z.chunk(2, dim=1)
        dg, du = d.chunk(2, dim=1)
        dg = 1.13 * dg + 2.0 ** -18 * gt.abs()
        gt = gt * torch.sigmoid(gt)
        d, z = gt.abs() * du + up.abs() * dg + dg * du + 2.0 ** -23 * (gt * up).abs(), gt * up
    if res is not None:
        z = z + res.double()
        d = d + 2.0 ** -24 * z.abs()
    return z, d


def check(got, z, d):
    h = torch.finfo(got.dtype).eps / 2
    tol = h * z.abs() + d * (1 + h) + (2.0 ** -25 if got.dtype == torch.float16 else 2.0 ** -120)
    err = (got.double() - z).abs()
    bad = ~(err <= tol)
    if got.dtype == torch.float16:               # from 65520 on (half a step past the largest) rounding gives infinity
        bad &= ~((z.abs() + d >= 65520) & (got.double() == torch.sign(z) * math.inf))
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} off, first at {torch.nonzero(bad)[0].tolist()}: " \
        f"err {err[bad][0].item():.3g} tol {tol[bad][0].item():.3g}"


class Linear:
    def __init__(self, M, N, K, act="none", bias=True, residual=True, dtype="bf16", seed=0, pad=0):
        g = gen(seed + 3 * M + 7 * N + K)
        self.M, self.N, self.K, self.act, self.dtype = M, N, K, act, DT[dtype]
        self.n_out = N // 2 if act == "swiglu" else N
        self.xq, self.w = codes((M, K), g), codes((N, K), g)
        self.xs = torch.exp(torch.randn(M, generator=g, device=DEV)) * 0.01
        self.ws = torch.exp(torch.randn(N, generator=g, device=DEV)) * 0.01 / K ** 0.5
        self.bias = torch.randn(N, generator=g, device=DEV) if bias else None
        self.res = torch.randn((M, self.n_out + pad), generator=g, device=DEV).to(self.dtype)[:, :self.n_out] \
            if residual else None
        self.pad = pad

    def workspace(self):
        n = moe.moe_i8_linear_workspace_size(self.M, self.N, self.K, ACTS[self.act])
        return torch.full((max(n, 256),), 0xFF, dtype=torch.uint8, device=DEV)

    def __call__(self, out=None, residual="own", workspace=None, stream=None):
        full = torch.full((self.M, self.n_out + self.pad), 3.0, dtype=self.dtype, device=DEV)
        o = full[:, :self.n_out] if out is None else out
        moe.moe_i8_linear(self.xq, self.xs, self.w, self.ws, o, self.bias,
                          self.res if isinstance(residual, str) else residual, ACTS[self.act],
                          self.workspace() if workspace is None else workspace, stream)
        if out is None:
            assert (full[:, self.n_out:] == 3.0).all()
        return o

    def check(self, got):
        z = self.xq.double() @ self.w.double().t() * self.xs.double()[:, None] * self.ws.double()
        check(got, *epilogue64(z, z.abs(), self.act, self.bias, self.res))


SIZES = [(1, 1, 16), (1, 64, 256), (1, 4096, 7168), (2, 130, 400), (5, 257, 1024), (16, 512, 2048), (17, 96, 528),
         (33, 1000, 640), (48, 2048, 4096), (64, 128, 112), (100, 300, 896), (129, 2048, 240), (256, 256, 1024),
         (300, 1026, 512), (1000, 1002, 2048), (513, 4096, 384)]


@pytest.mark.parametrize("act", list(ACTS))
@pytest.mark.parametrize("M,N,K", SIZES)
def test_linear(M, N, K, act):
    if act == "swiglu" and N % 2:
        N += 1
    p = Linear(M, N, K, act, bias=(M + N) % 3 != 0, residual=(M + K // 16) % 2 == 0,
               dtype=["bf16", "f16"][(M + K // 16 + len(act)) % 2], pad=(N + M) % 4)
    p.check(p())


@pytest.mark.parametrize("act", ["gelu", "swiglu"])
@pytest.mark.parametrize("M,N,K", [(2500, 4096, 256), (2501, 4130, 272), (2500, 1026, 384), (1100, 264, 400),
                                   (1100, 520, 1024), (1000, 1024, 2048), (1030, 264, 2432), (70, 200, 4992),
                                   (700, 1024, 4096), (4100, 1040, 16), (6000, 1026, 256), (2500, 2048, 2048),
                                   (9000, 66, 528), (40, 20000, 128)])
def test_linear_larger(M, N, K, act):
    p = Linear(M, N, K, act, dtype="f16" if N % 4 else "bf16")
    p.check(p())


@pytest.mark.parametrize("M,N,K,act", [(3000, 5000, 2064, "none"), (700, 20000, 1024, "swiglu"), (300, 30000, 1040, "silu"),
                                       (5000, 4000, 640, "swiglu")])
def test_several_tiles_a_workgroup(M, N, K, act):
    p = Linear(M, N, K, act)
    p.check(p())


@pytest.mark.parametrize("M,N,K", [(1, 16, 131056), (40, 64, 131056), (300, 70, 131056)])
def test_largest_sums(M, N, K):
    """-128 times -128 over the longest contraction: 2147221504, no overflow."""
    xq = torch.full((M, K), -128, dtype=torch.int8, device=DEV)
    w = torch.full((N, K), -128, dtype=torch.int8, device=DEV)
    w[1::2] = 127
    out = torch.zeros((M, N), dtype=torch.bfloat16, device=DEV)
    n = moe.moe_i8_linear_workspace_size(M, N, K)
    moe.moe_i8_linear(xq, torch.ones(M, device=DEV), w, torch.ones(N, device=DEV), out,
                      workspace=torch.empty(max(n, 256), dtype=torch.uint8, device=DEV))
    ref = torch.tensor([16384.0 * K, -16256.0 * K], device=DEV).repeat(N // 2).float().to(torch.bfloat16)
    assert (out == ref).all()


@pytest.mark.parametrize("M,N,K", [(1, 257, 1024), (3, 1000, 128), (40, 1001, 2048), (100, 520, 4096),
                                   (700, 1024, 4096), (1000, 1001, 2048), (3000, 1026, 512)])
def test_linear_exact(M, N, K):
    """Scales of 1 and small sums: every form gives the integers themselves."""
    g = gen(K)
    p = Linear(M, N, K, bias=False, residual=False)
    p.xq = torch.where(torch.rand((M, K), generator=g, device=DEV) < 32 / K, codes((M, K), g) % 2, 0).to(torch.int8)
    p.w = (codes((N, K), g) % 3).to(torch.int8)
    p.xs.fill_(1.0)
    p.ws.fill_(1.0)
    ref = p.xq.double() @ p.w.double().t()
    assert ref.abs().max() <= 256
    assert torch.equal(p().double(), ref)


def test_linear_out_may_be_the_residual():
    for M in (3, 200, 3000):
        p = Linear(M, 330, 512, "silu", pad=6)
        ref = p()
        acc = p.res.clone()
        p(acc, acc)
        assert torch.equal(acc, ref)


class Group:
    def __init__(self, M, E, N, K, k, bm, act="none", bias=True, dtype="bf16", per_route=False, routing="even", seed=0,
                 pad=0):
        g = gen(seed + M + 5 * E + 3 * N + K)
        self.__dict__.update(M=M, E=E, N=N, K=K, k=k, bm=bm, act=act, dtype=DT[dtype], per_route=per_route, pad=pad)
        self.n_out = N // 2 if act == "swiglu" else N
        if routing == "even":
            ids = torch.rand((M, E + 2), generator=g, device=DEV).argsort(1)[:, :k] - 1     # -1 and E: masked
        elif routing == "one":
            ids = torch.full((M, k), E // 2, device=DEV)
        else:                                    # "masked": no routes at all
            ids = torch.full((M, k), -1, device=DEV)
        self.ids = ids.to(torch.int32).contiguous()
        sc, bc = moe.moe_plan_capacity(M, k, E, bm)
        self.srt = torch.full((sc,), 0x7F7F7F7F, dtype=torch.int32, device=DEV)
        self.eids = torch.full((bc,), 0x7F7F7F7F, dtype=torch.int32, device=DEV)
        self.ntp = torch.zeros(1, dtype=torch.int32, device=DEV)
        moe.moe_plan(self.ids, E, bm, self.srt, self.eids, self.ntp)
        self.xq = codes((M * k if per_route else M, K), g)
        self.xs = torch.exp(torch.randn(self.xq.shape[0], generator=g, device=DEV)) * 0.01
        self.w = codes((E, N, K), g)
        self.ws = torch.exp(torch.randn((E, N), generator=g, device=DEV)) * 0.01 / K ** 0.5
        self.bias = torch.randn((E, N), generator=g, device=DEV) if bias else None

    def workspace(self):
        n = moe.moe_i8_group_mm_workspace_size(self.M, self.K, self.N, self.E, self.k, self.bm, self.srt.numel(),
                                               ACTS[self.act], self.per_route)
        return torch.full((max(n, 256),), 0xFF, dtype=torch.uint8, device=DEV)

    def __call__(self, out=None, workspace=None, stream=None):
        full = torch.full((self.M * self.k, self.n_out + self.pad), 3.0, dtype=self.dtype, device=DEV)
        o = full[:, :self.n_out] if out is None else out
        moe.moe_i8_group_mm(self.xq, self.xs, self.w, self.ws, self.srt, self.eids, self.ntp, self.k, self.bm, o,
                            self.bias, ACTS[self.act], self.workspace() if workspace is None else workspace,
                            stream, self.per_route)
        if out is None:
            assert (full[:, self.n_out:] == 3.0).all()
        return o

    def check(self, got):
        flat = self.ids.reshape(-1)
        for e in range(self.E):
            r = torch.nonzero(flat == e).flatten()
            if not r.numel():
                continue
            t = r if self.per_route else r // self.k
            z = self.xq[t].double() @ self.w[e].double().t() * self.xs[t].double()[:, None] * self.ws[e].double()
            check(got[r], *epilogue64(z, z.abs(), self.act, None if self.bias is None else self.bias[e], None))
        assert (got[(flat < 0) | (flat >= self.E)] == 3.0).all()


GROUPS = [  # M, E, N, K, k, bm, act, per_route, routing
    (1, 1, 1, 16, 1, 8, "none", False, "even"), (1, 257, 512, 7168, 9, 16, "swiglu", False, "even"),
    (4, 8, 512, 256, 2, 16, "swiglu", True, "even"), (16, 64, 130, 400, 8, 8, "gelu", False, "even"),
    (7, 3, 33, 112, 2, 128, "silu", True, "even"), (64, 8, 264, 1024, 2, 64, "none", False, "even"),
    (200, 24, 712, 528, 4, 32, "swiglu", True, "even"), (333, 24, 1288, 720, 4, 32, "none", True, "even"),
    (500, 7, 250, 640, 3, 16, "swiglu", False, "even"), (1000, 4, 1026, 384, 2, 128, "silu", False, "even"),
    (2048, 64, 512, 256, 10, 64, "none", False, "even"), (3000, 5, 300, 144, 3, 8, "gelu", True, "even"),
    (900, 3, 520, 2048, 2, 64, "swiglu", False, "one"), (50, 16, 64, 256, 4, 16, "none", False, "masked"),
    (2000, 1, 1000, 1040, 1, 128, "swiglu", False, "even"), (300, 1024, 64, 64, 8, 8, "none", False, "even"),
    (4000, 6, 2050, 256, 2, 128, "swiglu", True, "even"), (1, 4, 48, 131056, 2, 16, "none", False, "even"),
    (600, 2, 96, 40016, 1, 64, "silu", False, "one"),
]


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("M,E,N,K,k,bm,act,per_route,routing", GROUPS)
def test_group(M, E, N, K, k, bm, act, per_route, routing, dtype):
    p = Group(M, E, N, K, k, bm, act, bias=(M + N) % 2 == 0, dtype=dtype, per_route=per_route, routing=routing,
              pad=M % 3)
    p.check(p())


@pytest.mark.parametrize("M,N,K,act", [(142, 1920, 1536, "none"), (229, 704, 720, "swiglu"), (213, 920, 1280, "silu"),
                                       (232, 1000, 1232, "swiglu"), (142, 1914, 1552, "gelu"), (231, 1002, 1232, "swiglu")])
def test_linear_between(M, N, K, act):
    """Between few rows and many: passes of 48 and 64 rows."""
    p = Linear(M, N, K, act, dtype="f16" if M % 2 else "bf16")
    p.check(p())


@pytest.mark.parametrize("per_route", [False, True])
@pytest.mark.parametrize("M,E,N,K,k,bm,act", [
    (63, 9, 464, 1472, 4, 64, "none"), (270, 5, 128, 256, 2, 128, "swiglu"), (329, 6, 336, 2736, 3, 128, "gelu"),
    (131, 8, 1392, 960, 2, 64, "swiglu"), (308, 1, 1264, 2640, 1, 128, "silu"), (461, 9, 880, 384, 1, 128, "swiglu"),
    (844, 6, 3104, 1968, 2, 128, "swiglu"), (1163, 3, 3680, 816, 3, 16, "silu"), (1278, 3, 2720, 2944, 3, 64, "swiglu"),
    (461, 9, 890, 384, 1, 128, "swiglu"), (844, 6, 3106, 1968, 2, 128, "swiglu")])
def test_group_between(M, E, N, K, k, bm, act, per_route):
    """Few-rows passes of 32 to 64 rows over plan blocks, and the tiles' sizes with
    either kind of activation."""
    p = Group(M, E, N, K, k, bm, act, bias=M % 2 == 0, dtype="f16" if K % 32 else "bf16", per_route=per_route, pad=2)
    p.check(p())


def test_group_of_one_is_the_dense_product():
    p = Group(700, 1, 320, 512, 1, 64, "swiglu")
    d = Linear(700, 320, 512, "swiglu", residual=False)
    d.xq, d.xs, d.w, d.ws, d.bias = p.xq, p.xs, p.w[0], p.ws[0], p.bias[0]
    p.ids.zero_()
    moe.moe_plan(p.ids, 1, 64, p.srt, p.eids, p.ntp)
    assert torch.equal(p(), d())


def test_plan_beyond_its_buffers_and_foreign_entries():
    """A device-side plan length above sorted_cap is taken as sorted_cap, entries
    that are no route or expert are skipped."""
    p = Group(40, 4, 64, 128, 2, 16)
    ref = p()
    n = int(p.ntp)
    p.srt[n:] = 0x7F7F7F7F
    p.eids[n // 16:] = 0x7F7F7F7F
    p.ntp.fill_(0x7FFFFFFF)
    assert torch.equal(p(), ref)


def test_graph_streams_and_bits():
    for p in (Linear(3, 300, 512, "silu"), Linear(900, 1024, 4096, "swiglu"), Linear(3000, 1030, 512, "gelu"),
              Group(6, 32, 256, 1024, 4, 16, "swiglu"), Group(900, 8, 512, 512, 2, 64, "swiglu")):
        ref, ws = p().clone(), p.workspace()
        out = torch.full_like(ref, 3.0)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            p(out=out, workspace=ws)
        for _ in range(3):
            out.fill_(3.0)
            ws.fill_(0xAB)
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, ref)
        out.fill_(3.0)
        torch.cuda.synchronize()
        s = torch.cuda.Stream()
        p(out=out, workspace=ws, stream=s)
        s.synchronize()
        assert torch.equal(out, ref)


def test_nothing_to_do():
    p = Linear(0, 64, 128)
    p()
    g = Group(4, 4, 64, 128, 2, 16)
    out = torch.full((8, 64), 3.0, dtype=torch.bfloat16, device=DEV)
    moe.moe_i8_group_mm(g.xq, g.xs, g.w, g.ws, g.srt[:0], g.eids[:0], g.ntp, 2, 16, out)     # sorted_cap 0
    assert (out == 3.0).all()


def test_weights_past_4_gib():
    """Offsets past 32 bits in the experts' weights."""
    E, N, K = 33, 16384, 8192
    w = torch.zeros((E, N, K), dtype=torch.int8, device=DEV)
    w[-1, -1] = 1
    for M, bm in ((2, 16), (600, 64)):
        ids = torch.full((M, 1), E - 1, dtype=torch.int32, device=DEV)
        sc, bc = moe.moe_plan_capacity(M, 1, E, bm)
        srt, eids = torch.zeros(sc, dtype=torch.int32, device=DEV), torch.zeros(bc, dtype=torch.int32, device=DEV)
        ntp = torch.zeros(1, dtype=torch.int32, device=DEV)
        moe.moe_plan(ids, E, bm, srt, eids, ntp)
        x = torch.ones((M, K), dtype=torch.int8, device=DEV)
        out = torch.full((M, N), 3.0, dtype=torch.bfloat16, device=DEV)
        n = moe.moe_i8_group_mm_workspace_size(M, K, N, E, 1, bm, sc)
        moe.moe_i8_group_mm(x, torch.ones(M, device=DEV), w, torch.ones((E, N), device=DEV), srt, eids, ntp, 1, bm,
                            out, workspace=torch.empty(max(n, 256), dtype=torch.uint8, device=DEV))
        assert (out[:, -1] == K).all() and (out[:, :-1] == 0).all()
