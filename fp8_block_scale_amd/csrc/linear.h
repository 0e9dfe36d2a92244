// Dense FP8 block-scale product with its epilogue (linear.hip): launch interface.
#pragma once

#include "internal.h"

namespace moe {

enum { kActNone = 0, kActSilu = 1, kActGelu = 2, kActSwiglu = 3 };

enum { kLinStream = 0, kLinTile64, kLinTile128, kLinTile256 };

struct LinearArgs {
    const uint8_t *xq;       // [M, K] E4M3
    const float *xs;         // [M, K / 128]
    const uint8_t *w;        // [N, K] E4M3
    const float *ws;         // [ceil(N / 128), K / 128]
    const float *bias;       // [N] or NULL
    const uint16_t *res;     // [M, ld_res] BF16 or NULL
    uint16_t *out;           // [M, ld_out] BF16
    int64_t M, ld_res, ld_out;
    int K, N, n_out;         // n_out = N, or N / 2 with SwiGLU
    int act;
    // the schedule and the workspace (linear_workspace)
    int form;                // kernel form
    int stream_nq;           // few rows: tiles of 16 rows per workgroup
    int nsplit;              // parts that K is cut into (tile forms)
    float *part;             // FP32 sums of every (tile, split)
};

// Chooses the schedule, lays the workspace out at ws (NULL: sizes only) and
// returns its bytes.
size_t linear_workspace(LinearArgs &a, void *ws);
hipError_t launch_linear(const LinearArgs &a, hipStream_t st);

}  // namespace moe
