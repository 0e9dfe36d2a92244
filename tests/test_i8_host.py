"""The 8-bit integer products, as far as they can be checked without a GPU: which
bytes of the weights the few-rows kernel loads."""

import ctypes
import os
import shutil
import subprocess

import pytest

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
