"""The 8-bit integer products, as far as they can be checked without a GPU: which
bytes of the weights the few-rows kernel loads, which kernel which sizes take, and
the workspaces."""

import ctypes
import os
import shutil
import subprocess

import pytest

import fp8_block_scale_amd as moe
from test_gpu_i8_forms import ALL_GROUP, ALL_LINEAR, GROUP, LINEAR
from test_gpu_i8_mm import ACTS

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "fp8_block_scale_amd", "csrc")

WALK = r"""
#include "i8_index.h"

// Every load of one row of K weights, as the few-rows kernel makes them with `waves`
// waves and `unroll` steps loaded at once: bytes that lie outside the row, and
// values that no load brings, or more than one.
extern "C" int walk(int K, int waves, int unroll, int *outside, int *times) {
    *outside = 0;
    for (int w = 0; w < waves; ++w)
        for (int k0 = w * moe::kI8Step; k0 < K; k0 += waves * unroll * moe::kI8Step)
            for (int u = 0; u < unroll; ++u) {
                const int k = k0 + u * waves * moe::kI8Step;
                if (k >= K) break;
                for (int h = 0; h < 2; ++h)
                    for (int grp = 0; grp < 4; ++grp) {
                        const int at = moe::i8_weights_load(k, h, grp, K);
                        for (int i = at; i < at + 16; ++i) {
                            if (i < 0 || i >= K) ++*outside;
                            else if (moe::i8_weights_count(k, h, grp, K)) ++times[i];
                        }
                    }
            }
    int wrong = 0;
    for (int i = 0; i < K; ++i) wrong += times[i] != 1;
    return wrong;
}
"""


@pytest.fixture(scope="module")
def walk(tmp_path_factory):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("needs a host compiler")
    d = tmp_path_factory.mktemp("i8")
    src, lib = d / "walk.cpp", d / "walk.so"
    src.write_text(WALK)
    subprocess.run([gxx, "-std=c++17", "-O1", "-shared", "-fPIC", "-I", CSRC, str(src), "-o", str(lib)], check=True)
    return ctypes.CDLL(str(lib)).walk


@pytest.mark.parametrize("waves,unroll", [(8, 1), (8, 2)])
def test_weights_loaded_lie_in_their_row(walk, waves, unroll):
    """Whatever K, down to the least: a row may be the last of its allocation."""
    for K in list(range(16, 2320, 16)) + [4096, 7168, 131056]:
        outside, times = ctypes.c_int(), (ctypes.c_int * K)()
        assert walk(K, waves, unroll, ctypes.byref(outside), times) == 0, K
        assert outside.value == 0, K


# ------------------------------------------------------------ the schedule --

def test_forms_are_all_there():
    """Four few-rows passes and five tiles, each without SwiGLU and with it."""
    for sizes in (LINEAR, GROUP):
        assert len(sizes) == 9
        for ps in sizes.values():
            assert [p[-1] == "swiglu" for p in ps] == [False, True]


@pytest.mark.parametrize("form,size", ALL_LINEAR)
def test_dense_form(form, size):
    """The sizes that the GPU tests take for a form take it, some way off as well."""
    M, N, K, act = size
    for f in (0.96, 1.0, 1.04):
        assert moe.moe_debug_i8_schedule(int(M * f), K, N, act=ACTS[act]) == form


@pytest.mark.parametrize("form,size", ALL_GROUP)
def test_grouped_form(form, size):
    M, E, N, K, k, bm, act = size
    for f in (0.96, 1.0, 1.04):
        m = int(M * f)
        cap = moe.moe_plan_capacity(m, k, E, bm)[0]
        assert moe.moe_debug_i8_schedule(m, K, N, E, k, bm, cap, ACTS[act]) == form


def test_schedule_of_nothing_and_refusals():
    assert moe.moe_debug_i8_schedule(0, 64, 32) == (0, 0, 0)
    assert moe.moe_debug_i8_schedule(4, 64, 32, 3, 2, 16, 0) == (0, 0, 0)
    for a in ((4, 72, 32), (-1, 64, 32), (4, 64, 0), (4, 64, 32, -1), (4, 64, 32, 3, 0, 16, 64), (4, 64, 32, 3, 2, 16, 60)):
        with pytest.raises(moe.MoeError) as e:
            moe.moe_debug_i8_schedule(*a)
        assert e.value.status == moe.MOE_ERR_SHAPE
    for a in ((4, 1 << 17, 32), (4, 64, 32, 3, 2, 24, 72)):
        with pytest.raises(moe.MoeError) as e:
            moe.moe_debug_i8_schedule(*a)
        assert e.value.status == moe.MOE_ERR_UNSUPPORTED
    assert moe._c["moe_debug_i8_schedule"](4, 64, 32, 0, 1, 8, 0, 0, None) == moe.MOE_ERR_NULL


# --------------------------------------------------------------- workspaces --

def test_dense_products_have_no_workspace():
    for _, (M, N, K, act) in ALL_LINEAR:
        assert moe.moe_i8_linear_workspace_size(M, N, K, ACTS[act]) == 0


def _grouped(size, workspace, workspace_bytes):
    """The call with pointers that are never dereferenced: it is refused before."""
    M, E, N, K, k, bm, act = size
    p = [ctypes.c_void_p(0x10000 * (i + 1)) for i in range(8)]
    cap = moe.moe_plan_capacity(M, k, E, bm)[0]
    n_out = N // 2 if act == "swiglu" else N
    return moe.STATUS_NAMES[moe._c["moe_i8_group_mm"](p[0], p[1], 0, p[2], p[3], None, p[4], p[5], p[6], M, K, N, E, k, bm,
                                                      cap, ACTS[act], p[7], moe.MOE_DT_BF16, n_out, workspace,
                                                      workspace_bytes, None)]


@pytest.mark.parametrize("form,size", ALL_GROUP)
def test_workspaces_of_grouped_products(form, size):
    """Tiles need the list of them; missing, small or misaligned workspaces are refused."""
    M, E, N, K, k, bm, act = size
    cap = moe.moe_plan_capacity(M, k, E, bm)[0]
    n = moe.moe_i8_group_mm_workspace_size(M, K, N, E, k, bm, cap, ACTS[act])
    assert (n > 0) == (form[0] == 0)
    if n:
        assert _grouped(size, None, 0) == "MOE_ERR_NULL"
        assert _grouped(size, ctypes.c_void_p(0x100000), n - 1) == "MOE_ERR_CAPACITY"
        assert _grouped(size, ctypes.c_void_p(0x100008), n) == "MOE_ERR_ALIGN"
