"""Routing by scores, the weighted sum of routes and the 8-bit integer products:
their host checks refuse bad arguments before anything is launched (CPU only),
through the C ABI and through the Python binding."""

import ctypes

import pytest
import torch

import fp8_block_scale_amd as moe

P = [ctypes.c_void_p(0x10000 * (i + 1)) for i in range(8)]      # never dereferenced: validation fails first
BIG = 1 << 40
ODD = ctypes.c_void_p(0x10001)
OFF8 = ctypes.c_void_p(0x10008)


def _err(st):
    return moe.STATUS_NAMES[st]


ROUTE = dict(l=P[0], dt=2, M=4, ld=16, E=16, k=2, score=1, bias=P[1], G=4, tg=2, gt=2, renorm=1, scale=1.0, ns=1,
             ids=P[2], w=P[3])


def _route(**kw):
    a = dict(ROUTE, **kw)
    return _err(moe._c["moe_route_scored"](a["l"], a["dt"], a["M"], a["ld"], a["E"], a["k"], a["score"], a["bias"],
                                           a["G"], a["tg"], a["gt"], a["renorm"], a["scale"], a["ns"], a["ids"],
                                           a["w"], None))


RBWD = dict(l=P[0], dt=2, M=4, ld=16, E=16, slots=3, score=1, renorm=1, scale=1.0, ids=P[1], dw=P[2], dl=P[3],
            ldd=16)


def _rbwd(**kw):
    a = dict(RBWD, **kw)
    return _err(moe._c["moe_route_scored_bwd"](a["l"], a["dt"], a["M"], a["ld"], a["E"], a["slots"], a["score"],
                                               a["renorm"], a["scale"], a["ids"], a["dw"], a["dl"], a["ldd"], None))


@pytest.mark.parametrize("f", [_route, _rbwd])
def test_route_refusals(f):
    assert f(M=-1) == "MOE_ERR_SHAPE"
    assert f(M=1 << 31) == "MOE_ERR_SHAPE"
    assert f(E=0) == "MOE_ERR_SHAPE"
    assert f(E=1025, ld=2000) == "MOE_ERR_SHAPE"
    assert f(dt=3) == "MOE_ERR_SHAPE"
    assert f(dt=-1) == "MOE_ERR_SHAPE"
    assert f(score=2) == "MOE_ERR_SHAPE"
    assert f(ld=15) == "MOE_ERR_SHAPE"
    assert f(ld=(1 << 30) + 1) == "MOE_ERR_UNSUPPORTED"
    for s in (float("nan"), float("inf")):
        assert f(scale=s) == "MOE_ERR_SHAPE"
    assert f(l=None) == "MOE_ERR_NULL"
    assert f(ids=None) == "MOE_ERR_NULL"
    assert f(l=ODD) == "MOE_ERR_ALIGN"
    assert f(l=ctypes.c_void_p(0x10002)) == "MOE_ERR_ALIGN"
    assert f(l=ODD, dt=0) == "MOE_ERR_ALIGN"
    assert f(ids=ODD) == "MOE_ERR_ALIGN"
    assert f(M=0, l=None, ids=None) == "MOE_OK"


def test_route_refusals_of_the_choice():
    assert _route(G=0) == "MOE_ERR_SHAPE"
    assert _route(G=3) == "MOE_ERR_SHAPE"
    assert _route(E=130, ld=130, G=65) == "MOE_ERR_SHAPE"
    assert _route(tg=0) == "MOE_ERR_SHAPE"
    assert _route(tg=5) == "MOE_ERR_SHAPE"
    for gt in (0, 3):
        assert _route(gt=gt) == "MOE_ERR_SHAPE"
    assert _route(k=0) == "MOE_ERR_SHAPE"
    assert _route(k=9) == "MOE_ERR_SHAPE"            # two groups of four experts
    assert _route(k=33, E=64, ld=64, G=1, tg=1) == "MOE_ERR_SHAPE"
    for ns in (-1, 2):
        assert _route(ns=ns) == "MOE_ERR_SHAPE"
    assert _route(E=1024, ld=1024, ns=1) == "MOE_ERR_SHAPE"
    assert _route(w=None) == "MOE_ERR_NULL"
    assert _route(w=ODD) == "MOE_ERR_ALIGN"
    assert _route(bias=ODD) == "MOE_ERR_ALIGN"


def test_route_bwd_refusals():
    for n in (0, 34):
        assert _rbwd(slots=n) == "MOE_ERR_SHAPE"
    assert _rbwd(ldd=15) == "MOE_ERR_SHAPE"
    assert _rbwd(dw=None) == "MOE_ERR_NULL"
    assert _rbwd(dl=None) == "MOE_ERR_NULL"
    assert _rbwd(dl=ODD) == "MOE_ERR_ALIGN"
    assert _rbwd(dw=ODD) == "MOE_ERR_ALIGN"
    for n in ("l", "ids", "dw"):
        assert _rbwd(dl=RBWD[n]) == "MOE_ERR_SHAPE"


COMB = dict(y=P[0], ldy=64, dt=0, w=P[1], ids=P[2], idt=0, E=8, res=P[3], ldr=64, M=4, K=64, k=2, out=P[4], ldo=64)


def _comb(**kw):
    a = dict(COMB, **kw)
    return _err(moe._c["moe_combine"](a["y"], a["ldy"], a["dt"], a["w"], a["ids"], a["idt"], a["E"], a["res"],
                                      a["ldr"], a["M"], a["K"], a["k"], a["out"], a["ldo"], None))


def _cbwd(**kw):
    a = dict(COMB, dy=P[5], ldd=64, dw=P[6])
    a.update(kw)
    return _err(moe._c["moe_combine_bwd"](a["out"], a["ldo"], a["y"], a["ldy"], a["dt"], a["w"], a["ids"], a["idt"],
                                          a["E"], a["M"], a["K"], a["k"], a["dy"], a["ldd"], a["dw"], None))


@pytest.mark.parametrize("f", [_comb, _cbwd])
def test_combine_refusals(f):
    assert f(dt=2) == "MOE_ERR_SHAPE"
    assert f(M=-1) == "MOE_ERR_SHAPE"
    assert f(K=60) == "MOE_ERR_SHAPE"
    assert f(K=0) == "MOE_ERR_SHAPE"
    assert f(K=(1 << 20) + 8) == "MOE_ERR_UNSUPPORTED"
    assert f(k=0) == "MOE_ERR_SHAPE"
    assert f(M=1 << 30, k=2) == "MOE_ERR_SHAPE"
    assert f(idt=2) == "MOE_ERR_SHAPE"
    assert f(E=0) == "MOE_ERR_SHAPE"
    for n, ld in (("y", "ldy"), ("out", "ldo")):
        assert f(**{ld: 56}) == "MOE_ERR_SHAPE"
        assert f(**{ld: 68}) == "MOE_ERR_ALIGN"
        assert f(**{ld: (1 << 30) + 8}) == "MOE_ERR_UNSUPPORTED"
        assert f(**{n: None}) == "MOE_ERR_NULL"
        assert f(**{n: OFF8}) == "MOE_ERR_ALIGN"
    assert f(w=None) == "MOE_ERR_NULL"
    assert f(w=ODD) == "MOE_ERR_ALIGN"
    assert f(ids=ODD) == "MOE_ERR_ALIGN"
    assert f(ids=ctypes.c_void_p(0x10004), idt=1) == "MOE_ERR_ALIGN"
    assert f(M=0, y=None, out=None) == "MOE_OK"


def test_combine_overlaps():
    for n in ("y", "w", "ids"):
        assert _comb(out=COMB[n]) == "MOE_ERR_SHAPE"
    assert _comb(res=COMB["out"], ldr=72) == "MOE_ERR_SHAPE"
    assert _comb(ldr=56) == "MOE_ERR_SHAPE"
    assert _comb(res=OFF8) == "MOE_ERR_ALIGN"
    for n in ("y", "w", "ids", "out"):
        assert _cbwd(dy=COMB[n]) == "MOE_ERR_SHAPE"
        assert _cbwd(dw=COMB[n]) == "MOE_ERR_SHAPE"
    assert _cbwd(dy=P[6]) == "MOE_ERR_SHAPE"
    assert _cbwd(dy=None) == "MOE_ERR_NULL"
    assert _cbwd(dw=None) == "MOE_ERR_NULL"
    assert _cbwd(dw=ODD) == "MOE_ERR_ALIGN"
    assert _cbwd(ldd=56) == "MOE_ERR_SHAPE"


def _quant(**kw):
    a = dict(x=P[0], dt=0, M=4, K=64, ld=64, q=P[1], s=P[2])
    a.update(kw)
    return _err(moe._c["moe_quant_i8"](a["x"], a["dt"], a["M"], a["K"], a["ld"], a["q"], a["s"], None))


def test_quant_refusals():
    assert _quant(dt=2) == "MOE_ERR_SHAPE"
    assert _quant(M=-1) == "MOE_ERR_SHAPE"
    assert _quant(M=1 << 31) == "MOE_ERR_SHAPE"
    assert _quant(K=72, ld=72) == "MOE_ERR_SHAPE"
    assert _quant(K=1 << 17, ld=1 << 17) == "MOE_ERR_UNSUPPORTED"
    assert _quant(ld=56) == "MOE_ERR_SHAPE"
    assert _quant(ld=68) == "MOE_ERR_ALIGN"
    assert _quant(ld=(1 << 30) + 8) == "MOE_ERR_UNSUPPORTED"
    for n in ("x", "q", "s"):
        assert _quant(**{n: None}) == "MOE_ERR_NULL"
        assert _quant(**{n: ctypes.c_void_p(0x10002)}) == "MOE_ERR_ALIGN"
    assert _quant(q=P[0]) == "MOE_ERR_SHAPE"
    assert _quant(s=P[0]) == "MOE_ERR_SHAPE"
    assert _quant(s=P[1]) == "MOE_ERR_SHAPE"


I8 = dict(x=P[0], xs=P[1], w=P[2], ws=P[3], bias=P[4], res=P[5], ldr=32, M=4, N=32, K=64, act=0, out=P[6], dt=0,
          ldo=32, wsp=P[7], wsb=BIG)


def _lin(**kw):
    a = dict(I8, **kw)
    return _err(moe._c["moe_i8_linear"](a["x"], a["xs"], a["w"], a["ws"], a["bias"], a["res"], a["ldr"], a["M"],
                                        a["N"], a["K"], a["act"], a["out"], a["dt"], a["ldo"], a["wsp"], a["wsb"],
                                        None))


def _grp(**kw):
    a = dict(I8, E=8, k=2, bm=16, sc=128, pr=0, s=P[0], e=P[0], n=P[0])
    a.update(kw)
    return _err(moe._c["moe_i8_group_mm"](a["x"], a["xs"], a["pr"], a["w"], a["ws"], a["bias"], a["s"], a["e"],
                                          a["n"], a["M"], a["K"], a["N"], a["E"], a["k"], a["bm"], a["sc"],
                                          a["act"], a["out"], a["dt"], a["ldo"], a["wsp"], a["wsb"], None))


@pytest.mark.parametrize("f", [_lin, _grp])
def test_i8_refusals(f):
    assert f(M=-1) == "MOE_ERR_SHAPE"
    assert f(M=1 << 31) == "MOE_ERR_SHAPE"
    assert f(N=0) == "MOE_ERR_SHAPE"
    assert f(K=0) == "MOE_ERR_SHAPE"
    assert f(K=72) == "MOE_ERR_SHAPE"
    assert f(K=1 << 17) == "MOE_ERR_UNSUPPORTED"
    assert f(N=(1 << 20) + 1, ldo=1 << 21) == "MOE_ERR_UNSUPPORTED"
    assert f(act=4) == "MOE_ERR_SHAPE"
    assert f(act=-1) == "MOE_ERR_SHAPE"
    assert f(act=3, N=31) == "MOE_ERR_SHAPE"
    assert f(dt=2) == "MOE_ERR_SHAPE"
    assert f(ldo=31) == "MOE_ERR_SHAPE"
    assert f(ldo=(1 << 30) + 1) == "MOE_ERR_UNSUPPORTED"
    for n in ("x", "xs", "w", "ws", "out"):
        assert f(**{n: None}) == "MOE_ERR_NULL"
        assert f(**{n: ODD}) == "MOE_ERR_ALIGN"
    for n in ("x", "w"):
        assert f(**{n: OFF8}) == "MOE_ERR_ALIGN"
    assert f(bias=ODD) == "MOE_ERR_ALIGN"
    for n in ("x", "xs", "w", "ws", "bias"):
        assert f(out=I8[n]) == "MOE_ERR_SHAPE"
    assert f(M=1 << 30, k=1, N=1 << 20, ldo=1 << 20, ldr=1 << 20) == "MOE_ERR_UNSUPPORTED"


@pytest.mark.parametrize("f", [_lin, _grp])
def test_i8_tiles_of_64_by_64_are_counted(f):
    """2^43 outputs in tiles of 64 x 64 are 2^31."""
    assert f(M=1 << 24, k=1, N=1 << 19, ldo=1 << 20, ldr=1 << 20) == "MOE_ERR_UNSUPPORTED"


def test_i8_residual():
    assert _lin(res=I8["out"], ldr=40) == "MOE_ERR_SHAPE"
    assert _lin(ldr=31) == "MOE_ERR_SHAPE"
    assert _lin(ldr=(1 << 30) + 1) == "MOE_ERR_UNSUPPORTED"
    assert _lin(res=ODD) == "MOE_ERR_ALIGN"


def test_i8_plan():
    assert _grp(E=0) == "MOE_ERR_SHAPE"
    assert _grp(E=1025) == "MOE_ERR_UNSUPPORTED"
    assert _grp(k=0) == "MOE_ERR_SHAPE"
    assert _grp(bm=24) == "MOE_ERR_UNSUPPORTED"
    assert _grp(sc=120) == "MOE_ERR_SHAPE"
    assert _grp(sc=1 << 31) == "MOE_ERR_SHAPE"
    for n in ("s", "e", "n"):
        assert _grp(**{n: None}) == "MOE_ERR_NULL"
        assert _grp(**{n: ODD}) == "MOE_ERR_ALIGN"
    assert _grp(sc=0, s=None, e=None, n=None, wsp=None, wsb=0) == "MOE_OK"


def test_i8_workspace():
    """A schedule that needs a workspace refuses a missing, small or misaligned one."""
    seen = 0
    for M, N, K in ((4, 32, 64), (700, 1024, 4096), (1000, 1001, 2048), (8192, 4096, 7168)):
        n = moe.moe_i8_linear_workspace_size(M, N, K)
        if n == 0:
            continue
        seen += 1
        a = dict(M=M, N=N, K=K, ldo=N, ldr=N)
        assert _lin(**a, wsp=None) == "MOE_ERR_NULL"
        assert _lin(**a, wsb=n - 1) == "MOE_ERR_CAPACITY"
        assert _lin(**a, wsp=OFF8) == "MOE_ERR_ALIGN"
    a = dict(M=8192, N=2048, K=4096, E=288, k=8, bm=128)
    sc = moe.moe_plan_capacity(8192, 8, 288, 128)[0]
    n = moe.moe_i8_group_mm_workspace_size(8192, 4096, 2048, 288, 8, 128, sc)
    if n:
        seen += 1
        assert _grp(**a, sc=sc, ldo=2048, wsp=None) == "MOE_ERR_NULL"
        assert _grp(**a, sc=sc, ldo=2048, wsb=n - 1) == "MOE_ERR_CAPACITY"
        assert _grp(**a, sc=sc, ldo=2048, wsp=OFF8) == "MOE_ERR_ALIGN"
    assert seen
    assert moe.moe_i8_linear_workspace_size(4, 32, 72) == 0
    assert moe.moe_i8_group_mm_workspace_size(8, 64, 32, 2000, 2, 16, 128) == 0


# ------------------------------------------------------------ the binding --

BF, F32, I32, S8 = torch.bfloat16, torch.float32, torch.int32, torch.int8


def _z(*shape, dtype=F32):
    return torch.zeros(shape, dtype=dtype)


def _refused(f, *a, **kw):
    with pytest.raises(moe.MoeError) as e:
        f(*a, **kw)
    assert e.value.status == moe.MOE_ERR_SHAPE


def test_binding_route():
    l, ids, w = _z(4, 8), _z(4, 2, dtype=I32), _z(4, 2)
    f = moe.moe_route_scored
    _refused(f, l.double(), 2, ids, w)
    _refused(f, l[0], 2, ids, w)
    _refused(f, _z(8, 4).t(), 2, ids, w)
    _refused(f, l, 2, ids.long(), w)
    _refused(f, l, 2, ids[:3], w)
    _refused(f, l, 2, ids, w.half())
    _refused(f, l, 2, _z(4, 4, dtype=I32)[:, :2], w)
    _refused(f, l, 2, ids, w, n_shared=1)
    _refused(f, l, 2, ids, w, bias=_z(7))
    _refused(f, l, 2, ids, w, bias=_z(8).half())
    _refused(f, l, 2, ids, w)                        # on the CPU
    b = moe.moe_route_scored_bwd
    _refused(b, l, ids, w, _z(4, 7))
    _refused(b, l, ids, w, _z(3, 8))
    _refused(b, l, ids, w, _z(4, 8, dtype=BF))
    _refused(b, l, ids[:3], w, _z(4, 8))
    _refused(b, l, ids, _z(4, 3), _z(4, 8))
    _refused(b, l, ids[0], w, _z(4, 8))
    _refused(b, l, ids, w, _z(4, 8))


def test_binding_combine():
    y, w, out, ids = _z(8, 16, dtype=BF), _z(4, 2), _z(4, 16, dtype=BF), _z(4, 2, dtype=I32)
    f = moe.moe_combine
    _refused(f, y.float(), w, out)
    _refused(f, y[:7], w, out)
    _refused(f, y, w.half(), out)
    _refused(f, y, w, out.half())
    _refused(f, y, w, out[:3])
    _refused(f, y, w, out, ids.short(), 8)
    _refused(f, y, w, out, ids)                      # without E
    _refused(f, y, w, out, ids[:3], 8)
    _refused(f, y, w, out, residual=out[:3])
    _refused(f, y, w, out, residual=out.half())
    _refused(f, y, w, out)
    b = moe.moe_combine_bwd
    _refused(b, out, y, w, _z(7, 16, dtype=BF), _z(4, 2))
    _refused(b, out[:3], y, w, _z(8, 16, dtype=BF), _z(4, 2))
    _refused(b, out, y, w, _z(8, 16, dtype=BF), _z(4, 3))
    _refused(b, out, y, w, _z(8, 16, dtype=BF), _z(4, 2))


def test_binding_i8():
    x, q, s = _z(4, 32, dtype=BF), _z(4, 32, dtype=S8), _z(4)
    f = moe.moe_quant_i8
    _refused(f, x.float(), q, s)
    _refused(f, x, q.view(torch.uint8), s)
    _refused(f, x, _z(4, 64, dtype=S8)[:, :32], s)
    _refused(f, x, q, _z(5))
    _refused(f, x, q, s)
    w, ws, out = _z(8, 32, dtype=S8), _z(8), _z(4, 8, dtype=BF)
    f = moe.moe_i8_linear
    _refused(f, q.view(torch.uint8), s, w, ws, out)
    _refused(f, q, s, _z(8, 48, dtype=S8), ws, out)
    _refused(f, q, _z(3), w, ws, out)
    _refused(f, q, s, w, _z(7), out)
    _refused(f, q, s, w, ws, out.float())
    _refused(f, q, s, w, ws, out[:, :7])
    _refused(f, q, s, w, ws, out[:3])
    _refused(f, q, s, w, ws, out, act=moe.MOE_ACT_SWIGLU)
    _refused(f, q, s, w, ws, out, bias=_z(7))
    _refused(f, q, s, w, ws, out, residual=out.half())
    _refused(f, q, s, w, ws, out, residual=out[:3])
    _refused(f, q, s, w, ws, out, workspace=_z(512, dtype=torch.uint8)[::2])
    _refused(f, q, s, w, ws, out)
    E, gw, gs = 3, _z(3, 8, 32, dtype=S8), _z(3, 8)
    srt, eids, n = _z(64, dtype=I32), _z(4, dtype=I32), _z(1, dtype=I32)
    y = _z(8, 8, dtype=BF)
    f = moe.moe_i8_group_mm
    _refused(f, q, s, gw, gs, srt.long(), eids, n, 2, 16, y)
    _refused(f, q, s, gw, gs, srt, eids[:1], n, 2, 16, y)
    _refused(f, q, s, gw, gs, srt, eids, n, 3, 16, y)
    _refused(f, q, s, gw, _z(2, 8), srt, eids, n, 2, 16, y)
    _refused(f, q, s, gw, gs, srt, eids, n, 2, 16, y, bias=_z(8))
    _refused(f, q, s, gw, gs, srt, eids, n, 2, 16, y[:, :4])
    _refused(f, q[:3], s[:3], gw, gs, srt, eids, n, 2, 16, y)
    _refused(f, q, s, gw, gs, srt, eids, n, 2, 16, y)
