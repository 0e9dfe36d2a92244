// Products of 8-bit integers with row and channel scales (i8_mm.hip): launch
// interface.
#pragma once

#include "group_mm.h"
#include "linear.h"

namespace moe {

struct I8Args {
    const int8_t *xq;        // [rows of x, K]
    const float *xs;         // [rows of x]
    const int8_t *w;         // [N, K], grouped [E, N, K]
    const float *ws;         // [N] or [E, N]
    const float *bias;       // [N] or [E, N], or NULL
    const uint16_t *res;     // [M, ld_res] or NULL (dense)
    uint16_t *out;           // [M or R, ld_out]
    int64_t M, ld_res, ld_out;
    int K, N, n_out;         // n_out = N, or N / 2 with SwiGLU
    int act;
    bool f16;                // FP16 outputs (else BF16)
    bool grouped;
    GroupMmArgs g;           // the plan, E, R, top_k, block_m, per_route; with the tile kernel its
                             // row tiles (grouped)
    // the schedule (i8_workspace)
    int stream_nq;           // few rows: tiles of 16 rows per pass (0: the tile kernel)
    int tile_rows;           // rows of a tile
    int tile_cols;           // its weight rows
};

// Chooses the schedule, lays the workspace out at ws (NULL: sizes only) and
// returns its bytes.
size_t i8_workspace(I8Args &a, void *ws);
hipError_t launch_i8(const I8Args &a, hipStream_t st);

}  // namespace moe
