// Row-wise operators around the experts' products (rows.hip): launch interface.
#pragma once

#include "internal.h"

namespace moe {

// 8-bit codes and one scale of every row.
struct QuantI8Args {
    const uint16_t *x;       // [M, ld] BF16 or FP16
    bool f16;
    int64_t M, ld;
    int K;
    int8_t *xq;              // [M, K]
    float *xs;               // [M]
};
hipError_t launch_quant_i8(const QuantI8Args &a, hipStream_t st);

// The weighted sum of a token's routes, and its gradient.
struct CombineArgs {
    bool f16;
    int64_t M;
    int K, top_k, E;
    const float *w;          // [M, top_k]
    const void *ids;         // [M, top_k] int32 or int64, or NULL: every route counts
    bool ids_i64;
    const uint16_t *y;       // [M * top_k, ld_y]
    int64_t ld_y;
    // forward
    const uint16_t *res;     // [M, ld_res] or NULL
    uint16_t *out;           // [M, ld_out]
    int64_t ld_res, ld_out;
    // backward
    const uint16_t *dout;    // [M, ld_out]
    uint16_t *dy;            // [M * top_k, ld_dy]
    int64_t ld_dy;
    float *dw;               // [M, top_k]

    __device__ bool counts(int64_t r) const {
        if (!ids) return true;
        if (ids_i64) {
            const int64_t e = static_cast<const int64_t *>(ids)[r];
            return e >= 0 && e < E;
        }
        const int32_t e = static_cast<const int32_t *>(ids)[r];
        return e >= 0 && e < E;
    }
};
hipError_t launch_combine(const CombineArgs &a, hipStream_t st);
hipError_t launch_combine_bwd(const CombineArgs &a, hipStream_t st);

}  // namespace moe
