"""The dense FP8 block-scale product (moe_fp8_linear) against its formula in 64
bits on the same codes and scales.

Tolerance, derived.  One FP8 matrix instruction sums 128 products within a
window 15 bits below the largest: each product is cut by at most 2^-15 of the
block's largest, so a block's sum is off by at most 128 * 2^-15 = 2^-8 of its
largest product, times the block's scales.  Scaling and adding nkb blocks in
FP32 adds (nkb + 4) 2^-23 of the sum of the blocks' magnitudes.  The
activations have slope at most 1.13 (SwiGLU: the product rule) and are
evaluated within 2^-18 of their value and argument; the result is rounded to
BF16 once (2^-8).  The 2-norm of the error is held to 2^-8 of the result's
besides."""

import math

import pytest
import torch

import fp8_block_scale_amd as moe

pytestmark = pytest.mark.gpu

DEV = "cuda"
BF = torch.bfloat16
ACTS = {"none": moe.MOE_ACT_NONE, "silu": moe.MOE_ACT_SILU, "gelu": moe.MOE_ACT_GELU,
        "swiglu": moe.MOE_ACT_SWIGLU}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    torch.cuda.init()


def decode(codes):
    b = codes.long()
    e, m = (b >> 3) & 15, (b & 7).double()
    v = torch.where(e == 0, m * 2.0 ** -9, (8 + m) * torch.exp2(e.double() - 10))
    v = torch.where((b & 127) == 127, torch.full_like(v, math.nan), v)
    return torch.where(b >= 128, -v, v)


class Problem:
    def __init__(self, M, N, K, act="none", bias=True, residual=True, seed=0, spread=1.0):
        g = torch.Generator(device=DEV)
        g.manual_seed(seed + 3 * M + 7 * N + K)
        self.M, self.N, self.K, self.act = M, N, K, act
        self.n_out = N // 2 if act == "swiglu" else N
        nb = (N + 127) // 128
        codes = torch.randn((M + N, K), generator=g, device=DEV) * 100
        codes = codes.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        self.xq, self.w = codes[:M].contiguous(), codes[M:].contiguous()
        self.xs = torch.exp(torch.randn((M, K // 128), generator=g, device=DEV) * spread) * 0.01
        self.ws = torch.exp(torch.randn((nb, K // 128), generator=g, device=DEV) * spread) * 3e-3 / K ** 0.5
        self.bias = torch.randn(N, generator=g, device=DEV) if bias else None
        self.res = torch.randn((M, self.n_out), generator=g, device=DEV).to(BF) if residual else None

    def workspace(self):
        n = moe.moe_fp8_linear_workspace_size(self.M, self.N, self.K, ACTS[self.act])
        return torch.full((max(n, 256),), 0xFF, dtype=torch.uint8, device=DEV)

    def __call__(self, out=None, residual="own"):
        out = torch.full((self.M, self.n_out), 3.0, dtype=BF, device=DEV) if out is None else out
        moe.moe_fp8_linear(self.xq, self.xs, self.w, self.ws, out, self.bias,
                           self.res if isinstance(residual, str) else residual, ACTS[self.act],
                           self.workspace())
        return out

    def ref(self):
        """(result, bound of the error before rounding) in 64 bits."""
        M, N, K = self.M, self.N, self.K
        x, w = decode(self.xq), decode(self.w)
        z = torch.zeros((M, N), dtype=torch.float64, device=DEV)
        mag, win = torch.zeros_like(z), torch.zeros_like(z)
        blk = torch.arange(N, device=DEV) // 128
        for kb in range(K // 128):
            a, b = x[:, kb * 128:kb * 128 + 128], w[:, kb * 128:kb * 128 + 128]
            s = self.xs[:, kb].double()[:, None] * self.ws.double()[blk, kb][None]
            z += s * (a @ b.t())
            mag += s.abs() * (a.abs() @ b.abs().t())
            win += s.abs() * a.abs().amax(1)[:, None] * b.abs().amax(1)[None]
        d = 2.0 ** -8 * win + (K // 128 + 4) * 2.0 ** -23 * mag
        if self.bias is not None:
            z = z + self.bias.double()
            d = d + 2.0 ** -23 * z.abs()
        if self.act == "silu":
            d, z = 1.13 * d + 2.0 ** -18 * z.abs(), z * torch.sigmoid(z)
        elif self.act == "gelu":
            u = math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)
            d, z = 1.13 * d + 2.0 ** -18 * z.abs(), 0.5 * z * (1 + torch.tanh(u))
        elif self.act == "swiglu":
            gt, up, dg, du = z[:, :N // 2], z[:, N // 2:], d[:, :N // 2], d[:, N // 2:]
            dg = 1.13 * dg + 2.0 ** -18 * gt.abs()
            gt = gt * torch.sigmoid(gt)
            d, z = gt.abs() * du + up.abs() * dg + dg * du, gt * up
        if self.res is not None:
            z = z + self.res.double()
            d = d + 2.0 ** -23 * z.abs()
        return z, d


def check(got, ref, norm=True):
    z, d = ref
    tol = 2.0 ** -8 * z.abs() + d * (1 + 2.0 ** -8)
    err = (got.double() - z).abs()
    bad = ~(err <= tol)
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} off, first at {torch.nonzero(bad)[0].tolist()}: " \
        f"err {err[bad][0].item():.3g} tol {tol[bad][0].item():.3g}"
    if norm and z.numel() >= 64:
        assert err.norm() <= 2.0 ** -8 * z.norm(), (err.norm() / z.norm()).item()


SIZES = [(1, 1, 128), (1, 64, 256), (1, 4096, 7168), (2, 130, 384), (7, 257, 1024), (16, 512, 2048),
         (17, 96, 512), (33, 1000, 640), (48, 2048, 4096), (64, 128, 128), (100, 300, 896),
         (129, 2048, 256), (256, 256, 1024), (300, 1026, 512), (1000, 1002, 2048), (513, 4096, 384)]


@pytest.mark.parametrize("act", list(ACTS))
@pytest.mark.parametrize("M,N,K", SIZES)
def test_formula(M, N, K, act):
    if act == "swiglu" and N % 2:
        N += 1
    p = Problem(M, N, K, act, bias=(M + N) % 3 != 0, residual=(M + K // 128) % 2 == 0)
    check(p(), p.ref())


@pytest.mark.parametrize("act", ["gelu", "swiglu"])
@pytest.mark.parametrize("M,N,K", [(2500, 4096, 256), (2501, 4130, 256), (2500, 1026, 384),     # 256 and 128 row tiles
                                   (1100, 264, 384), (1100, 520, 1024),                           # 64 row tiles
                                   (1000, 1024, 2048), (1030, 264, 2432), (70, 200, 4992),        # K splits
                                   (700, 1024, 4096), (4100, 1040, 384), (6000, 1026, 256), (2500, 2048, 2048),
                                   (3000, 1026, 512)])
def test_larger(M, N, K, act):
    p = Problem(M, N, K, act)
    check(p(), p.ref())


WHOLE = [(1, 257, 1024), (3, 1000, 128), (16, 520, 640), (40, 1001, 2048), (100, 520, 4096),     # few rows
         (700, 1024, 4096), (1000, 1001, 2048),                                                    # 64 rows, K split
         (9000, 4097, 128), (5000, 4096, 2048),                                                    # 128 rows
         (9000, 1030, 256), (30000, 4096, 128), (30000, 4100, 256), (20000, 1030, 512)]            # 256 rows


@pytest.mark.parametrize("M,N,K", WHOLE)
@pytest.mark.parametrize("extras", [False, True])
def test_whole_numbers(M, N, K, extras):
    """Codes of whole numbers up to 2, scales 1/2, 1 and 2: every product is a
    multiple of 1/4 of at most 16, the sums of up to 4096 of them are below
    2^24 quarters, and a block's products lie within 4 bits: all exact, with a
    bias and a residual too, so the output equals the value in 64 bits, rounded
    once."""
    p = Problem(M, N, K, "none", bias=extras, residual=extras)
    g = torch.Generator(device=DEV)
    g.manual_seed(M + N)
    draw = lambda shape, n: torch.randint(-n, n + 1, shape, generator=g, device=DEV).float()
    code = lambda shape: draw(shape, 2).to(torch.float8_e4m3fn).view(torch.uint8)
    p.xq, p.w = code((M, K)), code((N, K))
    p.xs, p.ws = torch.exp2(draw(p.xs.shape, 1)), torch.exp2(draw(p.ws.shape, 1))
    if extras:
        p.bias, p.res = draw((N,), 50) / 4, (draw((M, N), 50) / 2).to(BF)
    z = p.ref()[0]
    assert torch.equal(p(), z.to(BF))


@pytest.mark.parametrize("N,K", [(1 << 20, 128), (24, 1 << 20), (300, 1 << 19)])
@pytest.mark.parametrize("M", [1, 20, 300, 1100])
def test_longest_rows(M, N, K):
    """K and N up to 2^20, on codes of whole numbers of at most 1: sums below
    2^24, exact."""
    p = Problem(1, 1, 128, "none", bias=False, residual=False)
    g = torch.Generator(device=DEV)
    g.manual_seed(M)
    one = torch.tensor([0x38, 0x00, 0xB8], dtype=torch.uint8, device=DEV)             # 1, 0, -1
    draw = lambda shape: one[torch.randint(0, 3, shape, generator=g, device=DEV, dtype=torch.int32).long()]
    p.M, p.N, p.K, p.n_out = M, N, K, N
    p.xq, p.w = draw((M, K)), draw((N, K))
    p.xs = torch.ones((M, K // 128), device=DEV)
    p.ws = torch.ones(((N + 127) // 128, K // 128), device=DEV)
    z = torch.zeros((M, N), dtype=torch.float64, device=DEV)
    for k in range(0, K, 1 << 15):
        z += decode(p.xq[:, k:k + (1 << 15)]) @ decode(p.w[:, k:k + (1 << 15)]).t()
    assert torch.equal(p(), z.to(BF))


@pytest.mark.parametrize("M,N,K", [(30000, 264, 128), (50000, 300, 384), (20000, 1030, 512), (30000, 4096, 128),
                                   (30000, 4100, 256)])
def test_many_items(M, N, K):
    """SwiGLU with several tiles of few stages on each workgroup, in every row
    tile form; the same bits twice."""
    p = Problem(M, N, K, "swiglu")
    got = p()
    check(got, p.ref())
    assert torch.equal(got, p())


@pytest.mark.parametrize("act", list(ACTS))
@pytest.mark.parametrize("M,N,K", [(3, 520, 1024), (40, 1002, 2048), (700, 1024, 4096), (5000, 1030, 512),
                                   (9000, 1030, 256)])
def test_before_rounding(M, N, K, act):
    """The value before its rounding to BF16: a residual of minus the rounded
    result leaves the low bits, to the tolerance without the result's own
    2^-8."""
    p = Problem(M, N, K, act, residual=False)
    p.res = -p.ref()[0].to(BF)
    check(p(), p.ref(), norm=False)


def test_no_rows():
    p = Problem(0, 64, 256)
    p()


@pytest.mark.parametrize("M,N,K", [(3, 192, 256), (40, 130, 384), (300, 520, 1024), (1100, 264, 384),
                                   (1030, 264, 2432), (2500, 1026, 384), (2500, 4096, 256)])
@pytest.mark.parametrize("act", ["gelu", "swiglu"])
def test_strides_and_residual_in_place(M, N, K, act):
    p = Problem(M, N, K, act)
    ref = p()
    n = p.n_out
    for extra in (8, 3):
        big = torch.full((M, n + extra), 3.0, dtype=BF, device=DEV)
        rb = torch.full((M, n + 5), float("nan"), dtype=BF, device=DEV)
        rb[:, :n] = p.res
        p(big[:, :n], rb[:, :n])
        assert torch.equal(big[:, :n], ref) and (big[:, n:] == 3.0).all()
        io = torch.full((M, n + extra), 3.0, dtype=BF, device=DEV)
        io[:, :n] = p.res
        p(io[:, :n], io[:, :n])                   # out += act(z)
        assert torch.equal(io[:, :n], ref) and (io[:, n:] == 3.0).all()
    odd = torch.full((M * n + 1,), 3.0, dtype=BF, device=DEV)
    p(odd[1:].view(M, n))                         # an output that is 2-byte aligned only
    assert torch.equal(odd[1:].view(M, n), ref) and odd[0] == 3.0


@pytest.mark.parametrize("M", [4, 5, 200, 1100])
@pytest.mark.parametrize("N", [96, 264])
def test_values_at_the_edges(M, N):
    """NaN codes and infinite scales stay in their rows and columns; all-zero
    rows and zero scales give exactly the bias; large arguments reach the
    activations' limits."""
    K = 256
    p = Problem(M, N, K, "silu", residual=False)
    ref = p()
    p.xq[1, 130] = 0x7F
    p.w[N - 1, 7] = 0xFF
    got = p()
    assert torch.isnan(got[1]).all() and torch.isnan(got[:, N - 1]).all()
    keep = torch.ones((M, N), dtype=torch.bool, device=DEV)
    keep[1] = keep[:, N - 1] = False
    assert torch.equal(got[keep], ref[keep])

    p = Problem(M, N, K, "none", residual=False)
    p.xq[0] = 0
    p.xs[2] = 0.0
    got = p()
    assert torch.equal(got[0], p.bias.to(BF)) and torch.equal(got[2], p.bias.to(BF))
    p.xs[3, 1] = float("inf")
    got = p()
    assert not torch.isfinite(got[3]).any()
    assert torch.isfinite(got[4:]).all() and torch.isfinite(got[:3]).all()

    for act, low in (("silu", 0.0), ("gelu", 0.0)):
        p = Problem(M, N, K, act, residual=False)
        p.xs.zero_()
        p.bias[0], p.bias[1], p.bias[2] = 3e38, -3e38, -200.0
        got = p()
        assert (got[:, 0].float() == torch.tensor(3e38, device=DEV).to(BF).float()).all()
        assert (got[:, 1:3] == low).all()


def test_far_offsets():
    """Codes and outputs past 2^31 bytes."""
    K, N, M = 128, 40, (1 << 24) + 70
    p = Problem(70, N, K, bias=True, residual=False)
    ref = p()
    xq = torch.zeros((M, K), dtype=torch.uint8, device=DEV)
    xs = torch.zeros((M, 1), dtype=torch.float32, device=DEV)
    xq[-70:], xs[-70:] = p.xq, p.xs
    p.xq, p.xs, p.M = xq, xs, M
    out = torch.empty((M, 128), dtype=BF, device=DEV)
    p(out[:, :N])
    assert torch.equal(out[-70:, :N], ref)
    assert torch.equal(out[:70, :N], p.bias.to(BF).expand(70, N))


def test_deterministic_streams_and_graph():
    for M, N, K, act in ((3, 512, 2048, "none"), (150, 1000, 1024, "swiglu"), (1030, 264, 2432, "gelu")):
        p = Problem(M, N, K, act)
        ref = p()
        assert torch.equal(ref, p())
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            o = p()
        side.synchronize()
        assert torch.equal(ref, o)
        ws = p.workspace()
        out = torch.empty_like(ref)
        graphs = []
        for _ in range(2):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                moe.moe_fp8_linear(p.xq, p.xs, p.w, p.ws, out, p.bias, p.res, ACTS[act], ws)
            graphs.append(g)
        for i in range(4):
            p.xs.mul_(1.5)
            p.res.mul_(0.5)
            want = p()
            ws.fill_(i * 85)
            out.fill_(7.0)
            graphs[i & 1].replay()
            torch.cuda.synchronize()
            assert torch.equal(want, out), (M, i)


@pytest.mark.parametrize("M", [3, 130])
def test_shared_expert_beside_the_routed_ones(M):
    """As it is used: the routed experts accumulate into the block's output,
    the shared expert (quantise, gate/up with SwiGLU, quantise, down) is added
    to the same tensor through the residual.  Tolerance: the shared expert's
    hidden row is BF16 (2^-8) and requantised to E4M3 (2^-4 of each value);
    computed here in 64 bits from the very codes the kernels wrote, so only
    the two products' own roundings count (2^-8 of the result's norm)."""
    E, K, I, k, bm = 8, 256, 256, 2, 16
    g = torch.Generator(device=DEV)
    g.manual_seed(11)
    from moe_workloads import make_weights
    w13, w13_s, w2, w2_s = make_weights(E, K, I, 5, False, DEV)
    s13, s13_s, s2, s2_s = (t[0] for t in make_weights(1, K, I, 6, False, DEV))
    x = torch.randn((M, K), generator=g, device=DEV).to(BF)
    wt = torch.rand((M, k), generator=g, device=DEV)
    ids = torch.randint(0, E, (M, k), generator=g, device=DEV).to(torch.int32)
    b = moe.MoeLayerBuffers(M, K, I, E, k, bm)
    out = torch.zeros((M, K), dtype=BF, device=DEV)
    moe.moe_layer(b, x, ids, wt, w13, w13_s, w2, w2_s, out)
    routed = out.clone()

    h = torch.empty((M, I), dtype=BF, device=DEV)
    moe.moe_fp8_linear(b.x_q, b.x_s, s13, s13_s, h, act=moe.MOE_ACT_SWIGLU,
                       workspace=_ws(M, 2 * I, K, moe.MOE_ACT_SWIGLU))
    hq = torch.empty((M, I), dtype=torch.uint8, device=DEV)
    hs = torch.empty((M, I // 128), dtype=torch.float32, device=DEV)
    moe.moe_quant_act(h, hq, hs)
    moe.moe_fp8_linear(hq, hs, s2, s2_s, out, residual=out, workspace=_ws(M, K, I, moe.MOE_ACT_NONE))

    def dense(q, s, w, ws):
        n = w.shape[0]
        xd = decode(q) * s.double().repeat_interleave(128, 1)
        wd = decode(w) * ws.double().repeat_interleave(128, 0)[:n].repeat_interleave(128, 1)
        return xd @ wd.t()

    z = dense(b.x_q, b.x_s, s13, s13_s)
    href = torch.nn.functional.silu(z[:, :I]) * z[:, I:]
    assert (h.double() - href).norm() <= 2.0 ** -8 * href.norm()
    ref = routed.double() + dense(hq, hs, s2, s2_s)
    assert (out.double() - ref).norm() <= 2.0 ** -8 * ref.norm()


def _ws(M, N, K, act):
    n = moe.moe_fp8_linear_workspace_size(M, N, K, act)
    return torch.empty(max(n, 256), dtype=torch.uint8, device=DEV)
