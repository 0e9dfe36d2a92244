"""The grouped 16-bit products and the dense FP8 product: their host checks
refuse bad arguments before anything is launched (CPU only), through the C ABI
and through the Python binding."""

import ctypes

import pytest
import torch

import fp8_block_scale_amd as moe

FAKE = ctypes.c_void_p(0x10000)      # never dereferenced: validation fails first
FAKE2, FAKE3 = ctypes.c_void_p(0x20000), ctypes.c_void_p(0x30000)
BIG = 1 << 40


def _err(st):
    return moe.STATUS_NAMES[st]


GMM = dict(M=4, K=64, N=32, E=8, k=2, bm=16, sc=128, dt=0, x=FAKE, w=FAKE2, y=FAKE3, ldx=64, ldy=32, pr=0,
           s=FAKE, e=FAKE, n=FAKE, ws=FAKE, wsb=BIG, dwt=0, acc=0)


def _fwd(**kw):
    a = dict(GMM, **kw)
    return _err(moe._c["moe_group_mm"](a["x"], a["ldx"], a["pr"], a["w"], a["dt"], a["s"], a["e"], a["n"],
                                       a["M"], a["K"], a["N"], a["E"], a["k"], a["bm"], a["sc"], a["y"],
                                       a["ldy"], a["ws"], a["wsb"], None))


def _dx(**kw):
    a = dict(GMM, **kw)
    return _err(moe._c["moe_group_mm_dx"](a["y"], a["ldy"], a["w"], a["dt"], a["s"], a["e"], a["n"], a["M"],
                                          a["K"], a["N"], a["E"], a["k"], a["bm"], a["sc"], a["x"],
                                          a["ldx"], a["pr"], a["ws"], a["wsb"], None))


def _dw(**kw):
    a = dict(GMM, **kw)
    return _err(moe._c["moe_group_mm_dw"](a["y"], a["ldy"], a["x"], a["ldx"], a["pr"], a["dt"], a["s"],
                                          a["e"], a["n"], a["M"], a["K"], a["N"], a["E"], a["k"], a["bm"],
                                          a["sc"], a["w"], a["dwt"], a["acc"], a["ws"], a["wsb"], None))


@pytest.mark.parametrize("f", [_fwd, _dx, _dw])
def test_group_refusals(f):
    assert f(K=60) == "MOE_ERR_SHAPE"
    assert f(N=36) == "MOE_ERR_SHAPE"
    assert f(K=0) == "MOE_ERR_SHAPE"
    assert f(N=-8) == "MOE_ERR_SHAPE"
    assert f(M=-1) == "MOE_ERR_SHAPE"
    assert f(k=0) == "MOE_ERR_SHAPE"
    assert f(E=0) == "MOE_ERR_SHAPE"
    assert f(E=1025) == "MOE_ERR_UNSUPPORTED"
    assert f(K=(1 << 20) + 8) == "MOE_ERR_UNSUPPORTED"
    assert f(bm=24) == "MOE_ERR_UNSUPPORTED"
    assert f(bm=256) == "MOE_ERR_UNSUPPORTED"
    assert f(sc=120) == "MOE_ERR_SHAPE"
    assert f(M=1 << 30, k=2) == "MOE_ERR_SHAPE"
    assert f(sc=1 << 31) == "MOE_ERR_SHAPE"
    assert f(sc=(1 << 31) - 16) == "MOE_ERR_SHAPE"
    assert f(M=(1 << 31) - 1023, k=1) == "MOE_ERR_SHAPE"
    assert f(dt=2) == "MOE_ERR_SHAPE"
    assert f(ldx=56) == "MOE_ERR_SHAPE"
    assert f(ldy=24) == "MOE_ERR_SHAPE"
    assert f(ldx=(1 << 30) + 8) == "MOE_ERR_UNSUPPORTED"
    assert f(ldy=(1 << 30) + 8) == "MOE_ERR_UNSUPPORTED"
    assert f(ldx=68) == "MOE_ERR_ALIGN"
    assert f(ldy=36) == "MOE_ERR_ALIGN"
    for n in ("x", "w", "y"):
        assert f(**{n: None}) == "MOE_ERR_NULL"
        assert f(**{n: ctypes.c_void_p(0x10008)}) == "MOE_ERR_ALIGN"
    # more output tiles than int32 counts
    assert f(M=1 << 30, k=1, K=1 << 20, N=1 << 20, ldx=1 << 20, ldy=1 << 20) == "MOE_ERR_UNSUPPORTED"
    assert f(E=1024, K=1 << 20, N=1 << 20, ldx=1 << 20, ldy=1 << 20) == "MOE_ERR_UNSUPPORTED"
    for n in ("s", "e", "n"):
        assert f(**{n: None}) == "MOE_ERR_NULL"
        assert f(**{n: ctypes.c_void_p(0x10002)}) == "MOE_ERR_ALIGN"


def test_group_tile_limit():
    """Tiles of 32 routes x 256 columns and of 128 x 128 of a weight, below
    2^31 - 2^21 of either: the size query tells by the status it leaves."""
    def size(M, E, K, N):
        moe.moe_group_mm_workspace_size(9, 1, 8, 8, 1, 1, 8, 8)          # leaves another message
        moe.moe_group_mm_workspace_size(moe.MOE_GMM_DX, M, K, N, E, 1, 8, 8)
        return "output tiles" in moe.moe_last_error()

    cols = 1 << 20
    rows = ((1 << 31) - (1 << 21)) // (cols // 256)                       # M / 32 + E of the first refusal
    assert size(32 * (rows - 1), 1, cols, 8) and not size(32 * (rows - 2), 1, cols, 8)
    assert size(32 * (rows - 1), 1, 8, cols) and not size(32 * (rows - 2), 1, 8, cols)
    assert size(8, 32, cols, cols) and not size(8, 31, cols, cols)


def test_group_output_is_no_input():
    assert _fwd(y=FAKE) == _fwd(y=FAKE2) == "MOE_ERR_SHAPE"
    assert _dx(x=FAKE3) == _dx(x=FAKE2) == "MOE_ERR_SHAPE"
    assert _dw(w=FAKE3) == _dw(w=FAKE) == "MOE_ERR_SHAPE"


def test_group_types_and_workspace():
    assert _dw(dwt=1) == "MOE_ERR_SHAPE"                # FP16 dw of BF16 operands
    assert _dw(dt=1, dwt=0) == "MOE_ERR_SHAPE"
    need = moe.moe_group_mm_workspace_size(moe.MOE_GMM_DX, 4, 64, 32, 8, 2, 16, 128)
    assert need > 0
    assert _dx(wsb=need - 1) == "MOE_ERR_CAPACITY"
    assert _dx(ws=None) == "MOE_ERR_NULL"
    assert _dx(ws=ctypes.c_void_p(0x10010)) == "MOE_ERR_ALIGN"
    # the size query rejects what the calls reject
    for bad in (dict(op=3), dict(K=60), dict(E=1025), dict(bm=24), dict(sc=120), dict(M=1 << 30)):
        a = dict(op=1, M=4, K=64, N=32, E=8, k=2, bm=16, sc=128)
        a.update(bad)
        assert moe.moe_group_mm_workspace_size(a["op"], a["M"], a["K"], a["N"], a["E"], a["k"], a["bm"],
                                               a["sc"]) == 0
    # nothing to do: no pointer is needed (dx of tokens without a plan is written, so it is)
    assert _fwd(M=0, x=None, w=None, y=None) == "MOE_OK"
    assert _dx(M=0, x=None, w=None, y=None) == "MOE_OK"
    assert _dw(M=0, acc=1, x=None, w=None, y=None) == "MOE_OK"
    assert _dw(M=0, w=None) == "MOE_ERR_NULL"
    assert _dx(sc=0, x=None) == "MOE_ERR_NULL"


def test_group_empty_plan():
    """A plan without routes needs neither its pointers nor a workspace; dx of
    the tokens is written, so its rows are checked."""
    none = dict(sc=0, s=None, e=None, n=None, ws=None, wsb=0)
    for op in range(3):
        assert moe.moe_group_mm_workspace_size(op, 4, 64, 32, 8, 2, 16, 0) == 0
    assert _fwd(**none) == "MOE_OK"
    assert _dx(pr=1, ldx=64, **none) == "MOE_OK"
    assert _dw(acc=1, **none) == "MOE_OK"
    assert _dx(x=None, **none) == "MOE_ERR_NULL"
    assert _dx(x=ctypes.c_void_p(0x10008), **none) == "MOE_ERR_ALIGN"
    assert _dx(ldx=56, **none) == "MOE_ERR_SHAPE"


LIN = dict(M=4, N=96, K=256, act=0, xq=FAKE, xs=FAKE, w=FAKE, ws=FAKE, b=FAKE, r=None, ldr=0, out=FAKE3,
           ldo=96, wk=FAKE, wkb=BIG)


def _lin(**kw):
    a = dict(LIN, **kw)
    return _err(moe._c["moe_fp8_linear"](a["xq"], a["xs"], a["w"], a["ws"], a["b"], a["r"], a["ldr"], a["M"],
                                         a["N"], a["K"], a["act"], a["out"], a["ldo"], a["wk"], a["wkb"],
                                         None))


def test_linear_refusals():
    assert _lin(K=200) == "MOE_ERR_SHAPE"
    assert _lin(K=0) == "MOE_ERR_SHAPE"
    assert _lin(N=0) == "MOE_ERR_SHAPE"
    assert _lin(M=-1) == "MOE_ERR_SHAPE"
    assert _lin(M=1 << 31) == "MOE_ERR_SHAPE"
    assert _lin(act=4) == "MOE_ERR_SHAPE"
    assert _lin(act=-1) == "MOE_ERR_SHAPE"
    assert _lin(act=3, N=95) == "MOE_ERR_SHAPE"         # SwiGLU of an odd number of rows
    assert _lin(N=(1 << 20) + 1) == "MOE_ERR_UNSUPPORTED"
    assert _lin(ldo=95) == "MOE_ERR_SHAPE"
    assert _lin(r=ctypes.c_void_p(0x20000), ldr=95) == "MOE_ERR_SHAPE"
    assert _lin(r=FAKE3, ldr=104) == "MOE_ERR_SHAPE"     # residual is out, other leading dimension
    assert _lin(out=FAKE) == "MOE_ERR_SHAPE"            # out is x_q or w
    assert _lin(M=1 << 30, N=1 << 20, ldo=1 << 20) == "MOE_ERR_UNSUPPORTED"
    for n in ("xq", "xs", "w", "ws", "out"):
        assert _lin(**{n: None}) == "MOE_ERR_NULL"
    for n, p in (("xq", 0x10008), ("w", 0x10008), ("xs", 0x10002), ("ws", 0x10002), ("b", 0x10002),
                 ("out", 0x10001)):
        assert _lin(**{n: ctypes.c_void_p(p)}) == "MOE_ERR_ALIGN"
    assert _lin(M=0, xq=None, w=None, out=None) == "MOE_OK"
    assert moe.moe_fp8_linear_workspace_size(4, 96, 200) == 0
    assert moe.moe_fp8_linear_workspace_size(4, 95, 256, moe.MOE_ACT_SWIGLU) == 0


def _plan(n=128, blocks=8):
    return (torch.zeros(n, dtype=torch.int32), torch.zeros(blocks, dtype=torch.int32),
            torch.zeros(1, dtype=torch.int32))


def _refused(f, *a, **kw):
    with pytest.raises(moe.MoeError) as ei:
        f(*a, **kw)
    assert ei.value.status == moe.MOE_ERR_SHAPE
    return str(ei.value)


@pytest.mark.parametrize("rows,blocks,want", [(128, 8, 128), (128, 9, 128), (256, 8, 128), (512, 11, 176)])
def test_binding_plan_length(monkeypatch, rows, blocks, want):
    """The kernels read a block's expert wherever the plan's length on the
    device says there is a block: the binding lets them go no further than
    expert_ids reaches, however long sorted_token_ids is."""
    seen = {}
    monkeypatch.setattr(moe, "_launch", lambda where, stream, tensors, *args: seen.update({where: args}))
    bf = torch.bfloat16
    x, w, y = torch.zeros(4, 64, dtype=bf), torch.zeros(8, 32, 64, dtype=bf), torch.zeros(8, 32, dtype=bf)
    plan = _plan(rows, blocks)
    moe.moe_group_mm(x, w, *plan, 2, 16, y)
    moe.moe_group_mm_dx(y, w, *plan, 2, 16, x)
    moe.moe_group_mm_dw(y, x, *plan, 2, 16, w)
    for where, at in (("moe_group_mm", 14), ("moe_group_mm_dx", 13), ("moe_group_mm_dw", 15)):
        assert seen[where][at - 1] == 16 and seen[where][at] == want, where


def test_binding_refusals():
    bf, hf = torch.bfloat16, torch.float16
    x, w, y = torch.zeros(4, 64, dtype=bf), torch.zeros(8, 32, 64, dtype=bf), torch.zeros(8, 32, dtype=bf)
    f = moe.moe_group_mm
    assert "GPU" in _refused(f, x, w, *_plan(), 2, 16, y)               # CPU tensors
    assert "x must be" in _refused(f, x.to(hf), w, *_plan(), 2, 16, y)
    assert "w must be" in _refused(f, x, w.float(), *_plan(), 2, 16, y)
    assert "w must be" in _refused(f, x, w[:, :, :32], *_plan(), 2, 16, y)
    assert "columns" in _refused(f, x[:, :32], w, *_plan(), 2, 16, y)
    assert "unit column stride" in _refused(f, torch.zeros(64, 4, dtype=bf).t(), w, *_plan(), 2, 16, y)
    assert "one row per" in _refused(f, x[:3], w, *_plan(), 2, 16, y)
    assert "no multiple" in _refused(f, x, w, *_plan(), 3, 16, y)
    assert "int32" in _refused(f, x, w, _plan()[0].long(), *_plan()[1:], 2, 16, y)
    assert "shorter" in _refused(f, x, w, *_plan(128, 7), 2, 16, y)
    assert "overlap" in _refused(f, x[:1].expand(4, 64), w, *_plan(), 2, 16, y)
    assert "contiguous" in _refused(f, x, w, *_plan(), 2, 16, y, torch.zeros(4096, dtype=torch.uint8)[::2])
    g = moe.moe_group_mm_dw
    assert "dw must be" in _refused(g, y, x, *_plan(), 2, 16, w.to(hf))
    assert "x must be" in _refused(g, y, x.float(), *_plan(), 2, 16, w)
    h = moe.moe_group_mm_dx
    assert "dx must be" in _refused(h, y, w, *_plan(), 2, 16, x.to(hf))
    assert "one row per" in _refused(h, y, w, *_plan(), 2, 16, x[:2])

    q, s = torch.zeros(4, 256, dtype=torch.uint8), torch.zeros(4, 2)
    lw, ls = torch.zeros(96, 256, dtype=torch.uint8), torch.zeros(1, 2)
    out = torch.zeros(4, 96, dtype=bf)
    lin = moe.moe_fp8_linear
    assert "GPU" in _refused(lin, q, s, lw, ls, out)
    assert "w_s must be" in _refused(lin, q, s, lw, torch.zeros(2, 2), out)
    assert "x_s must be" in _refused(lin, q, torch.zeros(4, 3), lw, ls, out)
    assert "disagree on K" in _refused(lin, q, s, lw[:, :128].contiguous(), ls, out)
    assert "bias" in _refused(lin, q, s, lw, ls, out, bias=torch.zeros(95))
    assert "out must" in _refused(lin, q, s, lw, ls, out, act=moe.MOE_ACT_SWIGLU)
    assert "residual must" in _refused(lin, q, s, lw, ls, out, residual=out.float())
