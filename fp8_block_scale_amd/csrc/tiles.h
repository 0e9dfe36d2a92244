// Helpers that the 16-bit grouped products and the FP8 linear product share.
#pragma once
#include "common.h"

namespace moe {

// A value that is the same in every lane, in a scalar register.
__device__ __forceinline__ int uni(int v) { return __builtin_amdgcn_readfirstlane(v); }

// Order of the output tiles of a product: panels of PANEL row tiles, column
// tiles outer and the panel's row tiles inner, so that the tiles that run at
// the same time on an XCD (neighbours in this order) share both operands in
// its L2.  Item i of rows x cols -> its row and column tile.
template <int PANEL>
__device__ __forceinline__ void panel_tile(int i, int rows, int cols, int &row, int &col) {
    const int panel = i / (PANEL * cols);
    const int first = panel * PANEL;
    const int height = rows - first < PANEL ? rows - first : PANEL;
    const int rem = i - first * cols;
    col = rem / height;
    row = first + rem - col * height;
}

}  // namespace moe
