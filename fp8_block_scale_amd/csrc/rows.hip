// Row-wise operators around the experts' products: 8-bit codes of rows, and
// the weighted sum of a token's routes with its gradient.  All of them are
// bound by memory: every value is read once (rows to be coded of more than 8192
// values past those twice, the second time from the caches) and written once.
#include <algorithm>

#include "common.h"
#include "rows.h"
#include "tiles.h"

namespace moe {

namespace {

// ----------------------------------------------------------- codes of rows
//   s = max(max |x| / 127, 2^-126),  code = round(x * (1 / s)), ties to even
// with IEEE divisions.  The largest magnitude is found on the bits, where a
// NaN is above infinity above every number: a row that holds one gets a scale
// that is not finite.

// T threads a row, CH chunks of 8 values a thread in registers; longer rows
// (LONG) are read a second time, from the caches.  A wave takes a row of up to 2048
// values, a workgroup longer ones.  Measured: 8192 rows of 4096 in 19.4 us (5.2
// TB/s), of 7168 in 28.7 (6.1, some of it from the caches); 48 rows of 4096 in 3.0.
template <bool F16, int T, int CH, bool LONG>
__global__ void __launch_bounds__(256)
quant_i8_kernel(QuantI8Args a) {
    __shared__ uint32_t part[4];
    const int tid = threadIdx.x % T;
    const int nch = a.K >> 3;
    for (int64_t m0 = (int64_t)blockIdx.x * (256 / T); m0 < a.M; m0 += (int64_t)gridDim.x * (256 / T)) {
        const int64_t m = m0 + threadIdx.x / T;
        const bool there = m < a.M;
        const uint16_t *x = a.x + (there ? m : 0) * a.ld;
        u32x4 r[CH];
        uint32_t top = 0;
        auto largest = [&](const u32x4 &v) {
#pragma unroll
            for (int i = 0; i < 4; ++i) top = max(top, max(v[i] & 0x7fffu, (v[i] >> 16) & 0x7fffu));
        };
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int i = c * T + tid;
            r[c] = i < nch ? *reinterpret_cast<const u32x4 *>(x + (int64_t)i * 8) : u32x4{0u, 0u, 0u, 0u};
        }
#pragma unroll
        for (int c = 0; c < CH; ++c) largest(r[c]);
        if (LONG)
            for (int i = CH * T + tid; i < nch; i += T) largest(*reinterpret_cast<const u32x4 *>(x + (int64_t)i * 8));
#pragma unroll
        for (int d = 32; d >= 1; d >>= 1) top = max(top, (uint32_t)__shfl_xor((int)top, d, 64));
        if constexpr (T > 64) {
            if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = top;
            __syncthreads();
            top = max(max(part[0], part[1]), max(part[2], part[3]));
        }
        if (T > 64) __syncthreads();             // (part is read before the next row writes it)
        if (!there) continue;
        const float amax = widen<F16>(top);
        const float s = amax < INFINITY ? fmaxf(__fdiv_rn(amax, 127.0f), kFltMin) : amax;
        const bool fin = s < INFINITY;               // else the codes are 0
        const float inv = __fdiv_rn(1.0f, s);
        if (tid == 0) a.xs[m] = s;
        auto codes = [&](const u32x4 &v, int i) {
            float f[8];
            widen8<F16>(v, f);
            uint32_t o[2] = {0u, 0u};
#pragma unroll
            for (int j = 0; j < 8; ++j)
                o[j >> 2] |= ((uint32_t)(fin ? (int)rintf(f[j] * inv) : 0) & 0xffu) << (8 * (j & 3));
            *reinterpret_cast<uint2 *>(a.xq + m * a.K + (int64_t)i * 8) = uint2{o[0], o[1]};
        };
#pragma unroll
        for (int c = 0; c < CH; ++c)
            if (c * T + tid < nch) codes(r[c], c * T + tid);
        if (LONG)
            for (int i = CH * T + tid; i < nch; i += T) codes(*reinterpret_cast<const u32x4 *>(x + (int64_t)i * 8), i);
    }
}

// ---------------------------------------------------------------- combine
//   out[t] = residual[t] + sum_j w[t, j] y[t top_k + j]
// in FP32, in route order, rounded once.  A thread takes 8 columns of a token;
// kBatch routes' reads go out together.  Measured: 4096 tokens of 8 routes, K = 4096
// (336 MB), 69 us, 4.8 TB/s; a large copy runs at 5.1.
constexpr int kBatch = 8;

template <bool F16>
__global__ void __launch_bounds__(256)
combine_kernel(CombineArgs a, int64_t chunks) {
    const int nch = a.K >> 3;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < chunks; i += (int64_t)gridDim.x * 256) {
        const int64_t t = i / nch;
        const int c = (int)(i - t * nch) * 8;
        float acc[8];
        if (a.res) widen8<F16>(*reinterpret_cast<const u32x4 *>(a.res + t * a.ld_res + c), acc);
        else {
#pragma unroll
            for (int v = 0; v < 8; ++v) acc[v] = 0.f;
        }
        for (int j0 = 0; j0 < a.top_k; j0 += kBatch) {
            u32x4 y[kBatch];
            float w[kBatch];
            bool ok[kBatch];
#pragma unroll
            for (int j = 0; j < kBatch; ++j) {
                const int64_t r = t * a.top_k + j0 + j;
                ok[j] = j0 + j < a.top_k && a.counts(r);
                if (ok[j]) {
                    y[j] = *reinterpret_cast<const u32x4 *>(a.y + r * a.ld_y + c);
                    w[j] = a.w[r];
                }
            }
#pragma unroll
            for (int j = 0; j < kBatch; ++j) {
                if (!ok[j]) continue;
                float f[8];
                widen8<F16>(y[j], f);
#pragma unroll
                for (int v = 0; v < 8; ++v) acc[v] = fmaf(w[j], f[v], acc[v]);
            }
        }
        *reinterpret_cast<u32x4 *>(a.out + t * a.ld_out + c) = narrow8<F16>(acc);
    }
}

//   dy[r] = w[r] dout[t(r)],  dw[r] = sum_c dout[t(r), c] y[r, c]
// A wave takes a route; a token's routes are neighbours, so its dout row is
// read from memory once.  Measured: 2048 tokens of 10 routes, K = 2048 (175 MB with
// 1% of them masked, dout counted once), 34.5 us from HBM (5.06 TB/s), 30 where some
// of it is in the caches; 4 tokens of 2 routes, K = 256, in 2.5.
template <bool F16>
__global__ void __launch_bounds__(256)
combine_bwd_kernel(CombineArgs a, int64_t R) {
    const int lane = threadIdx.x & 63;
    for (int64_t r = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); r < R; r += (int64_t)gridDim.x * 4) {
        if (!a.counts(r)) {
            if (lane == 0) a.dw[r] = 0.f;
            continue;
        }
        const uint16_t *g = a.dout + r / a.top_k * a.ld_out, *y = a.y + r * a.ld_y;
        uint16_t *dy = a.dy + r * a.ld_dy;
        const float w = a.w[r];
        const int nch = a.K >> 3;
        float s[8];
#pragma unroll
        for (int v = 0; v < 8; ++v) s[v] = 0.f;
        for (int i = lane; i < nch; i += 64) {
            float gf[8], yf[8], d[8];
            widen8<F16>(*reinterpret_cast<const u32x4 *>(g + (int64_t)i * 8), gf);
            widen8<F16>(*reinterpret_cast<const u32x4 *>(y + (int64_t)i * 8), yf);
#pragma unroll
            for (int v = 0; v < 8; ++v) {
                d[v] = w * gf[v];
                s[v] = fmaf(gf[v], yf[v], s[v]);
            }
            *reinterpret_cast<u32x4 *>(dy + (int64_t)i * 8) = narrow8<F16>(d);
        }
        float sum = ((s[0] + s[1]) + (s[2] + s[3])) + ((s[4] + s[5]) + (s[6] + s[7]));
#pragma unroll
        for (int d = 32; d >= 1; d >>= 1) sum += __shfl_xor(sum, d, 64);
        if (lane == 0) a.dw[r] = sum;
    }
}

// Workgroups of a launch: they go round for more than 2^23 (a launch counts its
// threads in 32 bits).
unsigned blocks(int64_t n) { return (unsigned)std::min(n, (int64_t)1 << 23); }

template <bool F16>
hipError_t quant(const QuantI8Args &a, hipStream_t st) {
    if (a.K <= 2048) quant_i8_kernel<F16, 64, 4, false><<<blocks((a.M + 3) / 4), 256, 0, st>>>(a);
    else if (a.K <= 8192) quant_i8_kernel<F16, 256, 4, false><<<blocks(a.M), 256, 0, st>>>(a);
    else quant_i8_kernel<F16, 256, 4, true><<<blocks(a.M), 256, 0, st>>>(a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_quant_i8(const QuantI8Args &a, hipStream_t st) {
    return a.f16 ? quant<true>(a, st) : quant<false>(a, st);
}

hipError_t launch_combine(const CombineArgs &a, hipStream_t st) {
    const int64_t chunks = a.M * (a.K >> 3);
    const unsigned grid = blocks((chunks + 255) / 256);
    if (a.f16) combine_kernel<true><<<grid, 256, 0, st>>>(a, chunks);
    else combine_kernel<false><<<grid, 256, 0, st>>>(a, chunks);
    return hipGetLastError();
}

hipError_t launch_combine_bwd(const CombineArgs &a, hipStream_t st) {
    const int64_t R = a.M * a.top_k;
    const unsigned grid = blocks((R + 3) / 4);
    if (a.f16) combine_bwd_kernel<true><<<grid, 256, 0, st>>>(a, R);
    else combine_bwd_kernel<false><<<grid, 256, 0, st>>>(a, R);
    return hipGetLastError();
}

}  // namespace moe
