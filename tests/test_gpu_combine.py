"""The weighted sum of a token's routes (moe_combine) and its gradient against
their formulas in 64 bits.

Tolerances, derived.  A sum of k products is k FP32 fused steps, each off by at
most 2^-24 of a partial sum, which the magnitudes bound: (k + 1) 2^-24 of their
sum, then one rounding to the output's type (half a step: 2^-8 BF16, 2^-11 FP16
relative; FP16 steps below its normal numbers are 2^-24).  A weight's gradient
is a sum over K columns: a lane adds K / 512 rounds of 8 columns in 8 chains,
joined in 3 + 6 levels: (K / 512 + 12) 2^-24 of the sum of the magnitudes."""

import pytest
import torch

import fp8_block_scale_amd as moe

pytestmark = pytest.mark.gpu

DEV = "cuda"
DT = {"bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    torch.cuda.init()


def rows(n, K, dtype, g, pad=0):
    return torch.randn((n, K + pad), generator=g, device=DEV).to(DT[dtype])[:, :K]


def half(dtype):
    return torch.finfo(DT[dtype]).eps / 2, (2.0 ** -25 if dtype == "f16" else 2.0 ** -120)


class Problem:
    def __init__(self, M, K, k, dtype, masked=0.0, ids=torch.int32, residual=True, pad=0, seed=0):
        g = torch.Generator(device=DEV)
        g.manual_seed(seed + M + 3 * K + k)
        self.M, self.K, self.k, self.dtype = M, K, k, dtype
        self.y = rows(M * k, K, dtype, g, pad)
        self.w = torch.randn((M, k), generator=g, device=DEV)
        self.E = 10
        e = torch.randint(0, 10, (M, k), generator=g, device=DEV)
        drop = torch.rand((M, k), generator=g, device=DEV) < masked
        e = torch.where(drop, torch.where(e % 2 == 0, torch.full_like(e, -1), e + 10), e)
        self.ids = None if ids is None else e.to(ids)
        self.ok = torch.ones((M, k), dtype=torch.bool, device=DEV) if ids is None else (e >= 0) & (e < 10)
        self.res = rows(M, K, dtype, g, pad) if residual else None
        self.dout = rows(M, K, dtype, g, pad)
        self.pad = pad

    def out(self, n):
        return torch.full((n, self.K + self.pad), 3.0, dtype=DT[self.dtype], device=DEV)

    def forward(self, out=None, residual="own", stream=None):
        full = self.out(self.M)
        o = full[:, :self.K] if out is None else out
        moe.moe_combine(self.y, self.w, o, self.ids, self.E, self.res if isinstance(residual, str) else residual,
                        stream=stream)
        if out is None:
            assert (full[:, self.K:] == 3.0).all()
        return o

    def check_forward(self, got):
        y = torch.where(self.ok[..., None], self.y.double().reshape(self.M, self.k, self.K), 0.0)
        t = torch.where(self.ok, self.w, 0.0).double()[..., None] * y
        z, mag = t.sum(1), t.abs().sum(1)
        if self.res is not None:
            z, mag = z + self.res.double(), mag + self.res.double().abs()
        h, tiny = half(self.dtype)
        assert ((got.double() - z).abs() <= h * z.abs() + (self.k + 1) * 2.0 ** -24 * mag * (1 + h) + tiny).all()

    def backward(self, dy=None, stream=None):
        full = self.out(self.M * self.k)
        dy = full[:, :self.K] if dy is None else dy
        dw = torch.full((self.M, self.k), 9.0, device=DEV)
        moe.moe_combine_bwd(self.dout, self.y, self.w, dy, dw, self.ids, self.E, stream=stream)
        assert (full[:, self.K:] == 3.0).all()
        return dy, dw

    def check_backward(self, dy, dw):
        g = self.dout.double()[:, None]
        h, tiny = half(self.dtype)
        dy = dy.double().reshape(self.M, self.k, self.K)
        assert (dy[~self.ok] == 3.0).all()
        ref = (self.w.double()[..., None] * g)[self.ok]
        # the FP32 product and its rounding
        assert ((dy[self.ok] - ref).abs() <= (h + 2.0 ** -23) * ref.abs() + tiny).all()
        t = torch.where(self.ok[..., None], self.y.double().reshape(self.M, self.k, self.K) * g, 0.0)
        assert ((dw.double() - t.sum(2)).abs() <= (self.K / 512 + 12) * 2.0 ** -24 * t.abs().sum(2)).all()
        assert (dw[~self.ok] == 0).all()


SIZES = [(1, 8, 1), (1, 7168, 9), (3, 16, 2), (4, 256, 2), (17, 520, 3), (64, 4096, 8), (100, 1000, 10),
         (31, 2048, 17), (5, 72, 33), (1, 65544, 3), (700, 512, 4)]


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("M,K,k", SIZES)
def test_formula(M, K, k, dtype):
    p = Problem(M, K, k, dtype, masked=[0.0, 0.3, 0.9][(M + k) % 3], ids=[None, torch.int32, torch.int64][M % 3],
                residual=K % 3 != 0, pad=8 * (M % 2))
    p.check_forward(p.forward())
    p.check_backward(*p.backward())


def test_masked_rows_are_not_read():
    """NaN in the rows of masked routes, a token without routes."""
    p = Problem(9, 64, 4, "bf16", masked=0.5)
    p.ids[3] = -1
    p.ok[3] = False
    p.y[~p.ok.reshape(-1)] = float("nan")
    z = p.forward()
    assert torch.isfinite(z).all() and torch.equal(z[3], p.res[3])
    p.y[~p.ok.reshape(-1)] = 0.0
    p.check_forward(z)
    p.y[~p.ok.reshape(-1)] = float("nan")
    dy, dw = p.backward()
    assert torch.isfinite(dw).all() and (dw[3] == 0).all()
    p.y[~p.ok.reshape(-1)] = 0.0
    p.check_backward(dy, dw)


def test_infinities_stay_in_their_rows():
    p = Problem(4, 64, 2, "bf16", ids=None)
    p.y[2, 5] = float("inf")
    p.dout[3, 1] = float("nan")
    z = p.forward()
    assert not torch.isfinite(z[1, 5]) and torch.isfinite(z).sum() == z.numel() - 1
    dy, dw = p.backward()
    assert torch.isnan(dy[6:8, 1]).all() and torch.isfinite(dy).sum() == dy.numel() - 2
    assert not torch.isfinite(dw[1, 0]) and torch.isnan(dw[3]).all() and torch.isfinite(dw).sum() == 5


def test_out_may_be_the_residual():
    p = Problem(50, 264, 5, "f16", masked=0.2, pad=16)
    ref = p.forward()
    acc = p.res.clone()
    p.forward(acc, acc)
    assert torch.equal(acc, ref)
    none = Problem(50, 264, 5, "f16", masked=0.2, residual=False, pad=16)
    none.check_forward(none.forward())


def test_gradient_by_differences():
    """d of sum(out * c): out is linear in y and in w."""
    p = Problem(3, 16, 2, "f16", residual=False, ids=None)
    dy, dw = p.backward()
    w, y, c = p.w.double(), p.y.double().reshape(3, 2, 16), p.dout.double()

    def loss(w, y):
        return ((w[..., None] * y).sum(1) * c).sum()

    for j in range(2):
        for t in range(3):
            wp = w.clone()
            wp[t, j] += 1.0
            d = loss(wp, y) - loss(w, y)
            assert (d - dw[t, j]).abs() <= 13 * 2.0 ** -24 * (y[t, j] * c[t]).abs().sum() + 1e-12
            yp = y.clone()
            yp[t, j, 3] += 1.0
            d = loss(w, yp) - loss(w, y)
            assert (d - dy[2 * t + j, 3]).abs() <= (2.0 ** -11 + 2.0 ** -23) * d.abs() + 2.0 ** -25 + 1e-12


def test_graph_streams_and_bits():
    p = Problem(300, 1024, 6, "bf16", masked=0.1)
    ref, (rdy, rdw) = p.forward().clone(), p.backward()
    out, dy, dw = p.out(300), p.out(1800), torch.zeros_like(rdw)

    def both(stream=None):
        moe.moe_combine(p.y, p.w, out, p.ids, p.E, p.res, stream=stream)
        moe.moe_combine_bwd(p.dout, p.y, p.w, dy, dw, p.ids, p.E, stream=stream)

    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        both()
    for _ in range(3):
        out.fill_(1)
        dy.fill_(3)
        dw.fill_(3)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, ref) and torch.equal(dy, rdy) and torch.equal(dw, rdw)
    out.fill_(1)
    dw.fill_(3)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    both(s)
    s.synchronize()
    assert torch.equal(out, ref) and torch.equal(dy, rdy) and torch.equal(dw, rdw)


def test_no_tokens():
    p = Problem(0, 64, 2, "bf16", ids=None)
    p.forward()
    p.backward()


def test_more_than_2_to_32_elements():
    """Offsets past 32 bits: the last rows of y lie 4.3e9 elements in."""
    M, K, k = 33000, 16384, 8
    y = torch.zeros((M * k, K), dtype=torch.bfloat16, device=DEV)
    y[-k:] = torch.arange(1, k + 1, device=DEV, dtype=torch.float32)[:, None].to(torch.bfloat16)
    w = torch.ones((M, k), device=DEV)
    out = torch.empty((M, K), dtype=torch.bfloat16, device=DEV)
    moe.moe_combine(y, w, out)
    assert (out[-1] == 36.0).all() and (out[:-1] == 0).all()
    dw = torch.empty((M, k), device=DEV)
    dy = torch.empty_like(y)
    out.fill_(1.0)
    moe.moe_combine_bwd(out, y, w, dy, dw)
    assert torch.equal(dw[-1], K * torch.arange(1, k + 1, device=DEV, dtype=torch.float32)) and (dw[:-1] == 0).all()
    assert (dy[-k:] == 1).all() and (dy[:16] == 1).all()


def test_more_rows_than_a_launch_counts():
    """More workgroups than a launch takes: the kernel goes round (33.6 million
    routes whose rows repeat every 2000)."""
    p = Problem(1000, 8, 2, "bf16", ids=None, residual=False)
    out, (dy, dw) = p.forward(), p.backward()
    n = 16800
    p.y, p.w, p.dout, p.M = p.y.repeat(n, 1), p.w.repeat(n, 1), p.dout.repeat(n, 1), 1000 * n
    assert (p.forward().view(n, -1) == out.reshape(1, -1)).all()
    bdy, bdw = p.backward()
    assert (bdy.view(n, -1) == dy.reshape(1, -1)).all() and (bdw.view(n, -1) == dw.view(1, -1)).all()
