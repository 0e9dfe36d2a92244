// Routing by scores and its gradient (router.hip): launch interface.
#pragma once

#include "internal.h"

namespace moe {

enum { kDtBf16 = 0, kDtF16 = 1, kDtF32 = 2 };
enum { kScoreSoftmax = 0, kScoreSigmoid = 1 };

constexpr int kRouteMaxGroups = 64;          // a group has at least one lane of the token's wave

struct ScoreArgs {
    const void *logits;      // [M, ld] of dtype
    int dtype;
    int64_t M, ld;
    int E;                   // routed experts
    int top_k, n_shared;
    int score;               // kScoreSoftmax or kScoreSigmoid
    bool renorm;
    float scale;
    // forward
    const float *bias;       // [E] or NULL
    int n_group, topk_group, group_top;
    int32_t *ids;            // [M, top_k + n_shared] (backward: read)
    float *w;                // [M, top_k + n_shared]
    // backward
    const float *dw;         // [M, slots]
    int slots;               // columns of ids and dw
    void *dl;                // [M, ld_dl] of dtype
    int64_t ld_dl;
};

hipError_t launch_route_scored(const ScoreArgs &a, hipStream_t st);
hipError_t launch_route_scored_bwd(const ScoreArgs &a, hipStream_t st);

}  // namespace moe
