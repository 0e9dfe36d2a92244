"""The grouped 16-bit products (moe_group_mm, moe_group_mm_dx, moe_group_mm_dw)
against their formulas in 64 bits on the same inputs.

Tolerance, derived: a result is an FP32 sum of n products, each exact in FP32
(11-bit by 11-bit or 8-bit by 8-bit significands), then one rounding to the
output's type.  A sum of n terms in any order is off by at most
(n - 1) 2^-23 S, S the sum of the magnitudes (one whole FP32 step allowed per
addition); the rounding adds eps / 2 of the value (FP16: half its smallest
subnormal, 2^-25, below its normal range).  S comes from the same product of
absolute values in 64 bits."""

import pytest
import torch

import fp8_block_scale_amd as moe

pytestmark = pytest.mark.gpu

DEV = "cuda"
BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    torch.cuda.init()


def make_plan(ids, E, bm):
    M, k = ids.shape
    sc, bc = moe.moe_plan_capacity(M, k, E, bm)
    srt = torch.full((sc,), -7, dtype=torch.int32, device=DEV)
    eid = torch.full((bc,), -7, dtype=torch.int32, device=DEV)
    ntp = torch.zeros(1, dtype=torch.int32, device=DEV)
    n = moe.moe_plan_workspace_size(M, k, E, bm)
    ws = torch.empty(n, dtype=torch.uint8, device=DEV) if n else None
    moe.moe_plan(ids.to(torch.int32).contiguous(), E, bm, srt, eid, ntp, ws)
    return srt, eid, ntp


def workspace(op, M, K, N, E, k, bm, sc, per_route):
    n = moe.moe_group_mm_workspace_size(op, M, K, N, E, k, bm, sc, per_route)
    return torch.full((max(n, 256),), 0xFF, dtype=torch.uint8, device=DEV)


class Problem:
    def __init__(self, dt, M, E, K, N, k, bm, per_route=False, routing="random", seed=0, scale=0.05):
        g = torch.Generator(device=DEV)
        g.manual_seed(seed + 17 * M + 31 * E + K + 5 * N)
        self.dt, self.M, self.E, self.K, self.N, self.k, self.bm = dt, M, E, K, N, k, bm
        self.per_route, self.R = per_route, M * k
        if routing == "random":                      # masked routes, repeats, empty experts
            ids = torch.randint(-1, E, (M, k), generator=g, device=DEV)
            if E > 3:
                ids[ids == 2] = E + 5
        elif routing == "one":
            ids = torch.full((M, k), E - 1, device=DEV)
        elif routing == "none":
            ids = torch.full((M, k), -1, device=DEV)
        elif routing == "full":
            ids = torch.randint(0, E, (M, k), generator=g, device=DEV)
        self.ids = ids
        rows = self.R if per_route else M
        self.x = torch.randn((rows, K), generator=g, device=DEV).to(dt)
        self.dy = torch.randn((self.R, N), generator=g, device=DEV).to(dt)
        self.w = (torch.randn((E, N, K), generator=g, device=DEV) * scale).to(dt)
        self.plan = make_plan(ids, E, bm)

    def ws(self, op):
        return workspace(op, self.M, self.K, self.N, self.E, self.k, self.bm, self.plan[0].numel(),
                         self.per_route)

    def groups(self):
        flat = self.ids.reshape(-1)
        for e in range(self.E):
            r = torch.nonzero(flat == e).flatten()
            yield e, r, (r if self.per_route else r // self.k)

    def valid(self):
        flat = self.ids.reshape(-1)
        return (flat >= 0) & (flat < self.E)

    # ---- formulas in 64 bits: (value, sum of magnitudes, terms)
    def ref_y(self):
        v = torch.zeros((self.R, self.N), dtype=torch.float64, device=DEV)
        s = torch.zeros_like(v)
        for e, r, t in self.groups():
            a, b = self.x[t].double(), self.w[e].double()
            v[r], s[r] = a @ b.t(), a.abs() @ b.abs().t()
        return v, s, self.K

    def ref_dx(self):
        rows = self.R if self.per_route else self.M
        v = torch.zeros((rows, self.K), dtype=torch.float64, device=DEV)
        s = torch.zeros_like(v)
        for e, r, t in self.groups():
            a, b = self.dy[r].double(), self.w[e].double()
            v.index_add_(0, t, a @ b)
            s.index_add_(0, t, a.abs() @ b.abs())
        return v, s, self.N * (1 if self.per_route else self.k)

    def ref_dw(self):
        v = torch.zeros((self.E, self.N, self.K), dtype=torch.float64, device=DEV)
        s = torch.zeros_like(v)
        for e, r, t in self.groups():
            a, b = self.dy[r].double(), self.x[t].double()
            v[e], s[e] = a.t() @ b, a.abs().t() @ b.abs()
        return v, s, max(self.R, 1)

    # ---- calls
    def y(self, out=None, x=None):
        out = torch.full((self.R, self.N), 3.0, dtype=self.dt, device=DEV) if out is None else out
        moe.moe_group_mm(self.x if x is None else x, self.w, *self.plan, self.k, self.bm, out,
                         self.ws(moe.MOE_GMM_FWD), x_per_route=self.per_route)
        return out

    def dx(self, out=None, dy=None):
        rows = self.R if self.per_route else self.M
        out = torch.full((rows, self.K), 3.0, dtype=self.dt, device=DEV) if out is None else out
        moe.moe_group_mm_dx(self.dy if dy is None else dy, self.w, *self.plan, self.k, self.bm, out,
                            self.ws(moe.MOE_GMM_DX), x_per_route=self.per_route)
        return out

    def dw(self, dtype=None, out=None, accumulate=False):
        if out is None:
            out = torch.full((self.E, self.N, self.K), 3.0, dtype=dtype or self.dt, device=DEV)
        moe.moe_group_mm_dw(self.dy, self.x, *self.plan, self.k, self.bm, out, self.ws(moe.MOE_GMM_DW),
                            accumulate, x_per_route=self.per_route)
        return out


def check(got, ref, dt):
    v, s, n = ref
    tol = torch.finfo(dt).eps / 2 * v.abs() + n * 2.0 ** -23 * s * (1 + torch.finfo(dt).eps)
    if dt == HF:
        tol = tol + 2.0 ** -25
    err = (got.double() - v).abs()
    bad = ~(err <= tol)
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} off, first at {torch.nonzero(bad)[0].tolist()}: " \
        f"err {err[bad][0].item():.3g} tol {tol[bad][0].item():.3g}"


def check_all(p):
    y = p.y()
    valid = p.valid()
    v, s, n = p.ref_y()
    check(y[valid], (v[valid], s[valid], n), p.dt)
    assert (y[~valid] == 3.0).all(), "rows of masked routes changed"
    dx = p.dx()
    v, s, n = p.ref_dx()
    if p.per_route:
        check(dx[valid], (v[valid], s[valid], n), p.dt)
        assert (dx[~valid] == 3.0).all(), "dx rows of masked routes changed"
    else:
        check(dx, (v, s, n), p.dt)
    ref = p.ref_dw()
    check(p.dw(), ref, p.dt)
    check(p.dw(F32), ref, F32)


SIZES = [  # M, E, K, N, top_k, block_m
    (1, 1, 8, 8, 1, 8), (1, 8, 64, 64, 2, 16), (4, 8, 256, 512, 2, 16), (5, 3, 72, 40, 2, 8),
    (1, 40, 1032, 72, 9, 16), (3, 16, 4096, 200, 5, 16), (16, 33, 7168, 512, 9, 16),
    (37, 7, 264, 136, 3, 32), (130, 4, 128, 256, 2, 64), (61, 5, 520, 328, 4, 128),
    (257, 2, 64, 520, 1, 128), (600, 4, 712, 264, 2, 32), (1500, 3, 320, 776, 2, 64),
    (700, 2, 1000, 1016, 3, 8), (2100, 2, 256, 512, 1, 16), (900, 1, 2048, 136, 2, 128)]


@pytest.mark.parametrize("M,E,K,N,k,bm", SIZES)
@pytest.mark.parametrize("dt", [BF, HF])
@pytest.mark.parametrize("per_route", [False, True])
def test_formulas(M, E, K, N, k, bm, dt, per_route):
    check_all(Problem(dt, M, E, K, N, k, bm, per_route))


@pytest.mark.parametrize("bm", [8, 16, 32, 64, 128])
@pytest.mark.parametrize("routing", ["one", "none", "full"])
def test_routings(bm, routing):
    check_all(Problem(BF, 150, 6, 200, 104, 3, bm, False, routing))
    check_all(Problem(HF, 9, 6, 200, 104, 3, bm, True, routing))


@pytest.mark.parametrize("M,E,K,N,k,bm", [(3000, 4, 1024, 1032, 2, 64), (2048, 12, 520, 2048, 4, 128),
                                          (5000, 1, 136, 256, 1, 32)])
@pytest.mark.parametrize("dt", [BF, HF])
def test_larger(M, E, K, N, k, bm, dt):
    check_all(Problem(dt, M, E, K, N, k, bm, routing="full"))


@pytest.mark.parametrize("M,E,K,N,k,bm", [
    (4500, 2, 1032, 1032, 2, 64), (9000, 2, 264, 264, 2, 128),      # 256-row tiles
    (70001, 3, 8, 16, 1, 16),                                       # many tokens, short rows
    (300, 1024, 136, 264, 8, 16), (2000, 1024, 64, 40, 4, 8),       # the most experts
    (40, 6, 72, 136, 6, 128), (3, 6, 264, 8, 6, 64)])               # every expert for every token
@pytest.mark.parametrize("dt", [BF, HF])
def test_ranges(M, E, K, N, k, bm, dt):
    check_all(Problem(dt, M, E, K, N, k, bm))


# Contractions of one, two and more stages of 64 with many items a workgroup,
# in each row-tile form (by the rule on sizes: 256, 128, 64 or 32 rows, 6 to
# 12 items on each of 256 workgroups): (op, rows of the form, M, E, the
# contraction's sizes, output columns).  The forward takes 32 rows only above
# one stage.
MANY = [("fwd", 256, 35496, 256, (8, 64, 72, 128), 520), ("fwd", 256, 35496, 64, (200,), 1032),
        ("fwd", 128, 28397, 1024, (8, 64), 520), ("fwd", 128, 14540, 512, (72, 128), 1032),
        ("fwd", 128, 35496, 256, (200,), 520),
        ("fwd", 64, 4765, 256, (8, 64), 2056), ("fwd", 64, 1562, 128, (72, 128), 4104),
        ("fwd", 64, 3812, 256, (200,), 2056),
        ("fwd", 32, 2440, 256, (72,), 2056), ("fwd", 32, 1250, 128, (128,), 4104),
        ("fwd", 32, 1562, 256, (200,), 2056),
        ("dx", 256, 35496, 256, (8, 64, 72, 128), 520), ("dx", 256, 35496, 64, (200,), 1032),
        ("dx", 128, 28397, 1024, (8, 64), 520), ("dx", 128, 14540, 512, (72, 128), 1032),
        ("dx", 128, 35496, 256, (200,), 520),
        ("dx", 64, 5956, 512, (8, 64), 1032), ("dx", 64, 1562, 128, (72, 128), 4104),
        ("dx", 64, 3812, 256, (200,), 2056),
        ("dx", 32, 1000, 1024, (8, 64, 72, 128, 200), 520)]


@pytest.mark.parametrize("op,rows,M,E,red,cols",
                         [(op, rows, M, E, c, n) for op, rows, M, E, cs, n in MANY for c in cs])
@pytest.mark.parametrize("per_route", [False, True])
def test_many_items_and_few_stages(op, rows, M, E, red, cols, per_route):
    """Each tile is stored to its own rows while the routes of the items after
    it are fetched; twice, with the same bits."""
    K, N = (red, cols) if op == "fwd" else (cols, red)
    p = Problem(HF if E == 256 else BF, M, E, K, N, 2, 8, per_route)
    valid = p.valid()
    call, (v, s, n) = (p.y, p.ref_y()) if op == "fwd" else (p.dx, p.ref_dx())
    got = call()
    if op == "fwd" or per_route:
        check(got[valid], (v[valid], s[valid], n), p.dt)
        assert (got[~valid] == 3.0).all(), "rows of masked routes changed"
    else:
        check(got, (v, s, n), p.dt)
    assert torch.equal(got, call())


@pytest.mark.parametrize("K", [8, 64])
def test_one_stage_forward_with_a_long_plan_buffer(K):
    """A plan buffer of more blocks than a grid takes goes to the row tiles
    (32 rows) at any size; blocks past the plan's length are never read."""
    p = Problem(BF, 1000, 1024, K, 520, 2, 8)
    srt, eid, ntp = p.plan
    blocks = 65536 + 8
    p.plan = (torch.cat([srt, torch.full((blocks * 8 - srt.numel(),), -9, dtype=torch.int32, device=DEV)]),
              torch.cat([eid, torch.full((blocks - eid.numel(),), 1 << 30, dtype=torch.int32, device=DEV)]), ntp)
    valid = p.valid()
    v, s, n = p.ref_y()
    got = p.y()
    check(got[valid], (v[valid], s[valid], n), BF)
    assert (got[~valid] == 3.0).all()
    assert torch.equal(got, p.y())


@pytest.mark.parametrize("K,N", [(1 << 20, 8), (8, 1 << 20), ((1 << 20) - 8, 24)])
@pytest.mark.parametrize("M,k,bm", [(1, 1, 8), (5, 2, 16), (150, 2, 32)])
def test_longest_contractions_and_rows(K, N, M, k, bm):
    """K and N up to 2^20, on whole numbers of at most 1: sums of fewer than
    2^24, so every result equals the value in 64 bits, rounded once."""
    p = Problem(BF, M, 2, K, N, k, bm, routing="full")
    g = torch.Generator(device=DEV)
    g.manual_seed(2)
    p.x, p.dy, p.w = (torch.randint(-1, 2, t.shape, generator=g, device=DEV, dtype=torch.int8).to(BF)
                      for t in (p.x, p.dy, p.w))
    assert torch.equal(p.y(), p.ref_y()[0].to(BF))
    assert torch.equal(p.dx(), p.ref_dx()[0].to(BF))
    assert torch.equal(p.dw(F32), p.ref_dw()[0].float())


def test_no_tokens():
    p = Problem(BF, 4, 3, 64, 32, 2, 16)
    e = torch.empty((0, 64), dtype=BF, device=DEV)
    z = torch.empty((0, 32), dtype=BF, device=DEV)
    plan = (torch.empty(0, dtype=torch.int32, device=DEV), torch.empty(0, dtype=torch.int32, device=DEV),
            torch.zeros(1, dtype=torch.int32, device=DEV))
    moe.moe_group_mm(e, p.w, *plan, 2, 16, z)
    moe.moe_group_mm_dx(z, p.w, *plan, 2, 16, e)
    for dt in (BF, F32):
        dw = torch.full((3, 32, 64), 5.0, dtype=dt, device=DEV)
        moe.moe_group_mm_dw(z, e, *plan, 2, 16, dw, accumulate=True)
        assert (dw == 5.0).all()
        moe.moe_group_mm_dw(z, e, *plan, 2, 16, dw)
        assert (dw == 0).all()


@pytest.mark.parametrize("M,K", [(5, 64), (1, 8), (700, 2056)])
@pytest.mark.parametrize("dt", [BF, HF])
def test_tokens_and_an_empty_plan(M, K, dt):
    """Plan buffers of length 0 (whose pointers are NULL): every route is
    masked, so y and dx rows of routes stay, dx of the tokens and dw are 0."""
    none = torch.empty(0, dtype=torch.int32, device=DEV)
    plan = none, none, torch.zeros(1, dtype=torch.int32, device=DEV)
    w = torch.randn((3, 32, K), device=DEV).to(dt)
    x, dy = torch.randn((M, K), device=DEV).to(dt), torch.randn((2 * M, 32), device=DEV).to(dt)
    y = torch.full((2 * M, 32), 3.0, dtype=dt, device=DEV)
    moe.moe_group_mm(x, w, *plan, 2, 16, y)
    assert (y == 3.0).all()
    dx = torch.full((2 * M, K), 3.0, dtype=dt, device=DEV)
    moe.moe_group_mm_dx(dy, w, *plan, 2, 16, dx)
    assert (dx == 3.0).all()
    wide = torch.full((M, K + 8), 3.0, dtype=dt, device=DEV)
    moe.moe_group_mm_dx(dy, w, *plan, 2, 16, wide[:, :K])
    assert not wide[:, :K].view(torch.int16).any() and (wide[:, K:] == 3.0).all()
    dw = torch.full((3, 32, K), 3.0, dtype=dt, device=DEV)
    moe.moe_group_mm_dw(dy, x, *plan, 2, 16, dw, accumulate=True)
    assert (dw == 3.0).all()
    moe.moe_group_mm_dw(dy, x, *plan, 2, 16, dw)
    assert not dw.view(torch.int16).any()


@pytest.mark.parametrize("dt", [BF, HF, F32])
def test_accumulate(dt):
    p = Problem(HF if dt == HF else BF, 210, 5, 136, 72, 2, 16)
    before = torch.randn((5, 72, 136), device=DEV).to(dt)
    got = p.dw(dt, before.clone(), accumulate=True)
    v, s, n = p.ref_dw()
    check(got, (v + before.double(), s + before.double().abs(), n + 1), dt)


@pytest.mark.parametrize("M,E,K,N,bm", [(210, 5, 136, 72, 16), (9000, 3, 264, 264, 64), (2100, 190, 152, 240, 16)])
@pytest.mark.parametrize("dt", [BF, HF, F32])
def test_accumulate_leaves_experts_without_routes(M, E, K, N, bm, dt):
    """Their dw is not rewritten: negative zeros and the bits of a NaN stay."""
    p = Problem(HF if dt == HF else BF, M, E, K, N, 2, bm)
    p.ids[(p.ids == 0) | (p.ids == E - 1)] = 1
    p.plan = make_plan(p.ids, E, bm)
    dw = torch.zeros((E, N, K), dtype=dt, device=DEV)
    bits = dw.view(torch.int32 if dt == F32 else torch.int16)
    bits[0] = torch.iinfo(bits.dtype).min                             # -0
    bits[E - 1] = {BF: 0x7F81, HF: 0x7C01, F32: 0x7F800001}[dt]       # a signalling NaN
    before = bits.clone()
    p.dw(dt, dw, accumulate=True)
    assert torch.equal(bits[0], before[0]) and torch.equal(bits[E - 1], before[E - 1])
    check(dw[1:E - 1], tuple(t[1:E - 1] for t in p.ref_dw()[:2]) + (2 * M,), dt)


@pytest.mark.parametrize("M,K,N", [(40, 72, 40), (1, 520, 136), (700, 328, 264)])
def test_strides_and_neighbours(M, K, N):
    """Operands inside larger buffers whose other values are NaN: none enters
    a sum, and output columns past the last stay as they were."""
    p = Problem(BF, M, 4, K, N, 2, 16)

    def pad(t, extra):
        b = torch.full((t.shape[0] + 2, t.shape[1] + extra), float("nan"), dtype=t.dtype, device=DEV)
        b[1:-1, :t.shape[1]] = t
        return b[1:-1, :t.shape[1]]

    ref = p.y(), p.dx(), p.dw()
    wbuf = torch.full((6, N, K), float("nan"), dtype=BF, device=DEV)
    wbuf[1:5] = p.w
    p.x, p.dy, p.w = pad(p.x, 24), pad(p.dy, 8), wbuf[1:5]
    yb = torch.full((2 * M, N + 16), 3.0, dtype=BF, device=DEV)
    xb = torch.full((M, K + 8), 3.0, dtype=BF, device=DEV)
    p.y(yb[:, :N])
    p.dx(xb[:, :K])
    assert torch.equal(yb[:, :N], ref[0]) and (yb[:, N:] == 3.0).all()
    assert torch.equal(xb[:, :K], ref[1]) and (xb[:, K:] == 3.0).all()
    assert torch.equal(p.dw(), ref[2])


@pytest.mark.parametrize("M,K,N,bm", [(12, 72, 40, 16), (500, 264, 136, 64)])
@pytest.mark.parametrize("per_route", [False, True])
def test_non_finite_stays_where_it_enters(M, K, N, bm, per_route):
    p = Problem(BF, M, 5, K, N, 2, bm, per_route)
    p.ids[0] = torch.tensor([0, -1])
    p.ids[1] = torch.tensor([1, 1])
    p.ids[2] = torch.tensor([-1, 9])             # a token without routes
    p.ids[3:] = torch.where((p.ids[3:] == 0) | (p.ids[3:] == 4), 3, p.ids[3:])
    p.plan = make_plan(p.ids, 5, bm)
    clean = p.y(), p.dx(), p.dw()
    valid = p.valid()
    t0 = torch.zeros(p.R, dtype=torch.bool, device=DEV)
    t0[0] = True                                  # route 0: the only route of expert 0
    p.x[0] = float("nan")                         # the source row of route 0
    p.dy[0] = float("inf")
    p.dy[~valid] = float("nan")                   # masked routes
    p.w[4] = float("nan")                         # an expert without routes
    if per_route:
        p.x[~valid] = float("nan")
    y, dx, dw = p.y(), p.dx(), p.dw()
    assert torch.isnan(y[0]).all()
    assert torch.equal(y[~t0], clean[0][~t0])
    assert not torch.isfinite(dx[0]).any()
    assert torch.equal(dx[1:], clean[1][1:])
    assert torch.isnan(dw[0]).all()
    assert torch.equal(dw[1:], clean[2][1:])
    assert (dw[4] == 0).all()


def test_overflow_rounds_to_infinity():
    p = Problem(HF, 3, 2, 64, 16, 1, 16, routing="one")
    p.x.fill_(60.0)
    p.w.fill_(60.0)                               # 64 * 3600 > 65504
    assert torch.isposinf(p.y()).all()


@pytest.mark.parametrize("M,E,K,N,k,bm", [(2100, 190, 152, 240, 2, 16), (3000, 9, 136, 200, 2, 64),
                                          (5000, 40, 264, 520, 1, 32)])
@pytest.mark.parametrize("dt", [BF, HF])
@pytest.mark.parametrize("accumulate", [False, True])
def test_dw_of_a_crowded_expert(M, E, K, N, k, bm, dt, accumulate):
    """One expert holds most routes (its rows are cut and joined), some a few,
    the first and the last none."""
    p = Problem(dt, M, E, K, N, k, bm)
    g = torch.Generator(device=DEV)
    g.manual_seed(3)
    p.ids = torch.randint(1, E - 1, (M, k), generator=g, device=DEV)
    p.ids[torch.rand((M, k), generator=g, device=DEV) < 0.6] = 3
    p.plan = make_plan(p.ids, E, bm)
    for out in (dt, F32):
        before = torch.randn((E, N, K), generator=g, device=DEV).to(out)
        v, s, n = p.ref_dw()
        ref = (v + before.double(), s + before.double().abs(), n + 1) if accumulate else (v, s, n)
        got = p.dw(out, before.clone(), accumulate)
        check(got, ref, out)
        assert torch.equal(got, p.dw(out, before.clone(), accumulate))


@pytest.mark.parametrize("M,E,K,N,k,bm,crowd", [
    (70001, 3, 8, 16, 1, 16, 0), (9000, 2, 264, 264, 2, 128, 0), (33000, 1, 264, 136, 1, 32, 0),   # cut, 128 squared
    (2100, 190, 152, 240, 2, 16, 0.6), (5000, 40, 264, 520, 1, 32, 0.3), (60000, 9, 136, 200, 2, 64, 0.5),
    (16384, 1, 1032, 2056, 1, 64, 0), (9000, 33, 1032, 1032, 1, 16, 0.4),                          # cut, 256 squared
    (700, 190, 264, 520, 2, 8, 0), (1500, 33, 1032, 1032, 1, 8, 0), (3000, 33, 1032, 1032, 1, 16, 0),
    (20000, 190, 264, 520, 2, 8, 0), (9000, 40, 1032, 2056, 2, 16, 0.2)])                          # many items
@pytest.mark.parametrize("dt", [BF, HF])
def test_dw_of_whole_numbers(M, E, K, N, k, bm, crowd, dt):
    """Every route counts, at any number of rows: with |x| <= 1 and |dy| <= 2
    each sum of at most 2^17 routes is a whole number below 2^24, exact in
    FP32 in any order, so dw equals the sum in 64 bits, rounded once.  A share
    `crowd` of the routes goes to one expert."""
    p = Problem(dt, M, E, K, N, k, bm)
    g = torch.Generator(device=DEV)
    g.manual_seed(M + E)
    p.ids[torch.rand((M, k), generator=g, device=DEV) < crowd] = E - 1
    p.plan = make_plan(p.ids, E, bm)
    draw = lambda shape, n: torch.randint(-n, n + 1, shape, generator=g, device=DEV)
    p.x, p.dy = draw(p.x.shape, 1).to(dt), draw(p.dy.shape, 2).to(dt)
    assert p.R <= 1 << 17
    v = p.ref_dw()[0]
    before = draw(v.shape, 100)
    for out in (F32, dt):
        assert torch.equal(p.dw(out), v.to(out))
        assert torch.equal(p.dw(out, before.to(out), accumulate=True), (v + before).to(out))


@pytest.mark.parametrize("M", [9, 700])
def test_subnormals(M):
    """FP16 subnormals (here the multiples of 2^-24 up to 2^-14) are values
    like any other.  y and dx, with small whole numbers: sums of at most 2^20
    units of 2^-24, exact.  dw: some 466 products of up to 10^6 units of 2^-48
    pass the 2^24 units that FP32 sums hold exactly, so to its tolerance."""
    p = Problem(HF, M, 3, 64, 72, 2, 16)
    g = torch.Generator(device=DEV)
    g.manual_seed(8)
    draw = lambda shape, n: torch.randint(-n, n + 1, shape, generator=g, device=DEV).double()
    p.x, p.dy = (draw(t.shape, 1000).mul(2.0 ** -24).to(HF) for t in (p.x, p.dy))
    p.w = draw(p.w.shape, 4).to(HF)
    valid = p.valid()
    v = p.ref_y()[0][valid]
    assert torch.equal(p.y()[valid], v.to(HF)) and v.abs().max() > 0
    assert torch.equal(p.dx(), p.ref_dx()[0].to(HF))
    check(p.dw(F32), p.ref_dw(), F32)


@pytest.mark.parametrize("M,E,K,N,k,bm", [(40, 6, 64, 48, 2, 16), (333, 3, 40, 24, 2, 32)])
def test_gradients_by_differences(M, E, K, N, k, bm):
    """Small whole numbers: every sum is exact in every type, so the gradients
    equal the central differences of f(x, w) = <dy, y> exactly."""
    p = Problem(BF, M, E, K, N, k, bm)
    g = torch.Generator(device=DEV)
    g.manual_seed(5)

    def ints(shape):
        return (torch.rand(shape, generator=g, device=DEV) < 0.3).float() * \
            torch.randint(-1, 2, shape, generator=g, device=DEV)

    p.x, p.w, p.dy = ints(p.x.shape).to(BF), ints(p.w.shape).to(BF), ints(p.dy.shape).to(BF)
    dirx, dirw = ints(p.x.shape), ints(p.w.shape)

    def f(x, w):
        q = Problem.__new__(Problem)
        q.__dict__.update(p.__dict__)
        q.x, q.w = x.to(BF), w.to(BF)
        return (q.y(torch.zeros((p.R, N), dtype=BF, device=DEV)).double() * p.dy.double()).sum()

    x, w = p.x.float(), p.w.float()
    dx = (f(x + dirx, w) - f(x - dirx, w)) / 2
    dw = (f(x, w + dirw) - f(x, w - dirw)) / 2
    assert (p.dx().double() * dirx.double()).sum() == dx
    assert (p.dw(F32).double() * dirw.double()).sum() == dw


def test_far_offsets():
    """Row offsets past 2^31 elements, weights of more than 2^31 elements."""
    ld = 1 << 26
    p = Problem(BF, 34, 2, 64, 72, 1, 16, routing="full")
    ref = p.y(), p.dx(), p.dw()
    big = torch.empty((34, ld), dtype=BF, device=DEV)
    big[:, :64] = p.x
    far = torch.empty((34, ld), dtype=BF, device=DEV)
    far[:, :72] = p.dy
    yfar = torch.empty((34, ld), dtype=BF, device=DEV)
    p.x, p.dy = big[:, :64], far[:, :72]
    assert torch.equal(p.y(yfar[:, :72]), ref[0])
    assert torch.equal(p.dx(yfar[:, :64]), ref[1])
    assert torch.equal(p.dw(), ref[2])
    del big, far, yfar
    E, N, K = 66, 4096, 8192
    w = torch.zeros((E, N, K), dtype=BF, device=DEV)
    w[E - 1, :, :2] = 1.0
    ids = torch.full((3, 1), E - 1, device=DEV)
    plan = make_plan(ids, E, 16)
    x = torch.ones((3, K), dtype=BF, device=DEV)
    y = torch.empty((3, N), dtype=BF, device=DEV)
    moe.moe_group_mm(x, w, *plan, 1, 16, y, workspace(0, 3, K, N, E, 1, 16, plan[0].numel(), False))
    assert (y == 2.0).all()
    dx = torch.empty((3, K), dtype=BF, device=DEV)
    dy = torch.ones((3, N), dtype=BF, device=DEV)
    moe.moe_group_mm_dx(dy, w, *plan, 1, 16, dx, workspace(1, 3, K, N, E, 1, 16, plan[0].numel(), False))
    assert (dx[:, :2] == 4096.0).all() and (dx[:, 2:] == 0).all()
    moe.moe_group_mm_dw(dy, x, *plan, 1, 16, w, workspace(2, 3, K, N, E, 1, 16, plan[0].numel(), False))
    assert (w[E - 1] == 3.0).all() and not w[:E - 1].any()


def test_deterministic_streams_and_graph():
    """Bit-identical over runs, on a second stream, and captured: the graph's
    replays follow new inputs, workspace contents in between do not matter."""
    p = Problem(BF, 300, 4, 264, 328, 2, 32)
    ref = p.y(), p.dx(), p.dw()
    for a, b in zip(ref, (p.y(), p.dx(), p.dw())):
        assert torch.equal(a, b)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        outs = p.y(), p.dx(), p.dw()
    side.synchronize()
    for a, b in zip(ref, outs):
        assert torch.equal(a, b)

    # one workspace for all three, and for two graphs
    n = max(p.ws(op).numel() for op in range(3))
    ws = torch.full((n,), 0xFF, dtype=torch.uint8, device=DEV)
    y = torch.full((p.R, p.N), 3.0, dtype=BF, device=DEV)
    dx = torch.empty((p.M, p.K), dtype=BF, device=DEV)
    dw = torch.empty((p.E, p.N, p.K), dtype=BF, device=DEV)
    args = (*p.plan, p.k, p.bm)

    def run():
        moe.moe_group_mm(p.x, p.w, *args, y, ws)
        moe.moe_group_mm_dx(p.dy, p.w, *args, dx, ws)
        moe.moe_group_mm_dw(p.dy, p.x, *args, dw, ws)

    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            run()
        graphs.append(g)
    for i in range(4):
        p.x.copy_(torch.randn_like(p.x.float()).to(BF))
        p.dy.copy_(torch.randn_like(p.dy.float()).to(BF))
        want = p.y(), p.dx(), p.dw()
        ws.fill_(i * 85)
        graphs[i & 1].replay()
        torch.cuda.synchronize()
        for a, b in zip(want, (y, dx, dw)):
            assert torch.equal(a, b), i


def test_expert_mlp_and_gradients():
    """The operators as they are used: route, plan, gate/up product, SwiGLU,
    down product, route sum -- and back -- against 64 bits.  Tolerance: the
    forward's and backward's tensors pass through at most four BF16 roundings
    (2^-8 each), each entering the next product as independent relative noise;
    the norms of the differences stay below 4 * 2^-8 of the results' norms."""
    M, E, K, I, k, bm = 96, 12, 256, 128, 4, 16
    g = torch.Generator(device=DEV)
    g.manual_seed(3)
    x = torch.randn((M, K), generator=g, device=DEV).to(BF)
    w13 = (torch.randn((E, 2 * I, K), generator=g, device=DEV) / 16).to(BF)
    w2 = (torch.randn((E, K, I), generator=g, device=DEV) / 11).to(BF)
    logits = torch.randn((M, E), generator=g, device=DEV)
    dout = torch.randn((M, K), generator=g, device=DEV).to(BF)
    sc, bc = moe.moe_plan_capacity(M, k, E, bm)
    ids = torch.empty((M, k), dtype=torch.int32, device=DEV)
    wt = torch.empty((M, k), dtype=F32, device=DEV)
    plan = (torch.empty(sc, dtype=torch.int32, device=DEV), torch.empty(bc, dtype=torch.int32, device=DEV),
            torch.empty(1, dtype=torch.int32, device=DEV))
    moe.moe_route_plan(logits, k, 0, 1.0, bm, ids, wt, *plan)

    def ws(op, K_, N_, pr):
        return workspace(op, M, K_, N_, E, k, bm, sc, pr)

    def silu_parts(h):
        gt, up = h[:, :I].float(), h[:, I:].float()
        s = torch.sigmoid(gt)
        return gt, up, s

    h = torch.empty((M * k, 2 * I), dtype=BF, device=DEV)
    moe.moe_group_mm(x, w13, *plan, k, bm, h, ws(0, K, 2 * I, False))
    gt, up, s = silu_parts(h)
    a = (gt * s * up).to(BF)
    y = torch.empty((M * k, K), dtype=BF, device=DEV)
    moe.moe_group_mm(a, w2, *plan, k, bm, y, ws(0, I, K, True))
    out = (y.view(M, k, K).float() * wt[..., None]).sum(1)

    dy = (dout[:, None].float() * wt[..., None]).reshape(M * k, K).to(BF)
    da = torch.empty((M * k, I), dtype=BF, device=DEV)
    moe.moe_group_mm_dx(dy, w2, *plan, k, bm, da, ws(1, I, K, True))
    dw2 = torch.empty_like(w2)
    moe.moe_group_mm_dw(dy, a, *plan, k, bm, dw2, ws(2, I, K, True))
    daf = da.float()
    dh = torch.cat([daf * up * s * (1 + gt * (1 - s)), daf * gt * s], dim=1).to(BF)
    dx = torch.empty_like(x)
    moe.moe_group_mm_dx(dh, w13, *plan, k, bm, dx, ws(1, K, 2 * I, False))
    dw13 = torch.empty((E, 2 * I, K), dtype=F32, device=DEV)
    moe.moe_group_mm_dw(dh, x, *plan, k, bm, dw13, ws(2, K, 2 * I, False))

    x64, w13_64, w2_64 = (t.cpu().double().requires_grad_() for t in (x, w13, w2))
    idc, wc = ids.cpu().long(), wt.cpu().double()
    ref = 0
    for j in range(k):
        hj = torch.stack([w13_64[idc[t, j]] @ x64[t] for t in range(M)])
        aj = torch.nn.functional.silu(hj[:, :I]) * hj[:, I:]
        ref = ref + wc[:, j:j + 1] * torch.stack([w2_64[idc[t, j]] @ aj[t] for t in range(M)])
    ref.backward(dout.cpu().double())
    for name, got, want in (("out", out, ref.detach()), ("dx", dx, x64.grad), ("dw13", dw13, w13_64.grad),
                            ("dw2", dw2, w2_64.grad)):
        rel = ((got.cpu().double() - want).norm() / want.norm()).item()
        assert rel <= 4 * 2.0 ** -8, (name, rel)
