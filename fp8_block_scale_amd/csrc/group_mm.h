// Grouped 16-bit matrix products (group_mm.hip): launch interface.
#pragma once

#include "internal.h"

namespace moe {

enum { kGmmFwd = 0, kGmmDx = 1, kGmmDw = 2 };

struct GroupMmArgs {
    int op;                  // kGmmFwd, kGmmDx or kGmmDw
    bool f16;                // FP16 operands (else BF16)
    bool per_route;          // x / dx rows are indexed by route (else by token r / top_k)
    bool out_f32;            // dw in FP32
    bool accumulate;         // dw is added to
    const uint16_t *x;       // [M or R, ld_x]   (forward, dw)
    const uint16_t *dy;      // [R, ld_dy]       (dx, dw)
    const uint16_t *w;       // [E, N, K]        (forward, dx)
    const int32_t *sorted;   // the plan
    const int32_t *eids;
    const int32_t *ntp;
    int64_t M, R, sorted_cap;
    int64_t ld_x, ld_dy, ld_out;
    int K, N, E, top_k, block_m;
    void *out;               // y [R, ld_out], dx [M or R, ld_out] or dw [E, N, K]
    // workspace (group_mm_workspace)
    int32_t *rpos;           // [R] plan row of each route, -1 if masked (dx summed over routes)
    float *part;             // [R, K] FP32 rows of the routes (dx summed over routes)
};

// Lays the workspace out at ws (NULL: sizes only) and returns its bytes.
size_t group_mm_workspace(GroupMmArgs &g, void *ws);
hipError_t launch_group_mm(const GroupMmArgs &g, hipStream_t st);

}  // namespace moe
