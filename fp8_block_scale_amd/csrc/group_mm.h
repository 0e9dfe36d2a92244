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
    // the schedule and the workspace (group_mm_workspace)
    int stream;              // the few-rows kernel (forward): 16-row tiles per pass, 0: the tile kernel
    int tile_rows;           // rows of a tile (forward, dx) or a part (dw)
    int max_tiles;           // most row tiles that any routing gives
    int dw_tile;             // output tile of dw: 128 or 256 squared
    int max_slots;           // dw: most FP32 sums of parts of cut experts (0: none is cut)
    uint32_t div_m;          // r / top_k
    int div_s;
    int32_t *meta;           // [2] row tiles or parts; cut experts (dw)
    int4 *tiles;             // [max_tiles] {first plan row, rows, expert, slot}
    int4 *joins;             // [max_slots] {expert, first slot, slots} of the cut experts (dw)
    int32_t *rpos;           // [R] -1 if the route is masked (dx summed over routes)
    float *part;             // FP32 rows [R, K] (dx summed over routes) or [max_slots, N, K] (dw)

    __host__ __device__ int token_of(int r) const {
        return (int)(((uint64_t)(uint32_t)r * div_m) >> (31 + div_s));
    }
};

// Parts of at most `size` rows that an expert's rows give on average, for routes
// spread evenly over the experts (rows of one: about normal, variance `rows`).
double group_parts(double rows, int size);
// Sets div_m and div_s (token_of) from top_k.
void group_divider(GroupMmArgs &g);
// Lays the workspace out at ws (NULL: sizes only) and returns its bytes.
size_t group_mm_workspace(GroupMmArgs &g, void *ws);
// For another kernel over the plan's row tiles (forward): lays the list of
// tiles of tile_rows rows out at ws and returns its bytes, and lists them.
size_t group_tiles_workspace(GroupMmArgs &g, int tile_rows, void *ws);
hipError_t launch_group_prep(const GroupMmArgs &g, hipStream_t st);
hipError_t launch_group_mm(const GroupMmArgs &g, hipStream_t st);
// dx of tokens without a route (M, K, out and ld_out are read): zeros.
hipError_t launch_group_no_routes(GroupMmArgs g, hipStream_t st);

}  // namespace moe
