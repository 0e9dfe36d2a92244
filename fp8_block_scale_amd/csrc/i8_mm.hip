// Products of 8-bit integers with one scale per row of x and per weight row,
// with their epilogue, dense or grouped by expert over a routing plan:
//   z[r, n]   = x_s[t(r)] w_s[e(r), n] sum_k x_q[t(r), k] w[e(r), n, k] + bias[e(r), n]
//   out[r, n] = act(z)[r, n] + residual[r, n]
// With SwiGLU act(z)[r, j] = silu(z[r, j]) z[r, I + j].
//
// The sums are 32-bit integers, exact for K < 2^17 (2^17 products of at most
// 2^14); scales, bias, activation and residual are FP32, rounded once.
#include <algorithm>

#include "i8_mm.h"
#include "tiles.h"

namespace moe {

namespace {

typedef int v4i __attribute__((ext_vector_type(4)));

__device__ __forceinline__ v4i mfma64(const u32x4 &a, const u32x4 &b, const v4i &c) {
    return __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(v4i, a), __builtin_bit_cast(v4i, b), c, 0, 0, 0);
}

__device__ __forceinline__ float widen16(bool f16, uint32_t v) {
    return f16 ? (float)__builtin_bit_cast(_Float16, (uint16_t)v) : bf16_bits_to_f32(v & 0xffffu);
}
__device__ __forceinline__ uint16_t narrow16(bool f16, float v) {
    return (uint16_t)(f16 ? to16x2<true>(v, 0.f) : to16x2<false>(v, 0.f));
}

// ----------------------------------------------------------------- few rows

// 16 weight rows (with SwiGLU 8 gate and their 8 up rows) x 16 NQ rows of x;
// wave w takes the steps of 128 values of K w, w + NW, ...; the waves' sums
// are added in LDS.  Rows past the end read another row: their results are
// not stored.  Values past the end of K are zeros on the weights' side.
template <int NQ, int NW, bool SW, bool GROUPED>
__global__ void __launch_bounds__(64 * NW)
i8_stream_kernel(I8Args a) {
    __shared__ int sums[NW][16 * NQ * 17];
    const int tid = threadIdx.x, l = tid & 63, w = uni(tid >> 6), i16 = l & 15, grp = l >> 4;
    const int c0 = blockIdx.x * (SW ? 8 : 16);
    int row0 = blockIdx.y * (16 * NQ), rows_end = (int)a.M, e = 0;
    if (GROUPED) {
        int P = *a.g.ntp;
        P = P < a.g.sorted_cap ? P : (int)a.g.sorted_cap;
        row0 = blockIdx.y * a.g.block_m;
        rows_end = row0 + a.g.block_m;
        if (rows_end > P) return;
        e = uni(a.g.eids[blockIdx.y]);
        if (e < 0 || e >= a.g.E) return;
    }
    auto wrow = [&](int i) {                     // weight row of MFMA row i
        const int c = c0 + (SW ? i & 7 : i);
        return (c < a.n_out ? c : a.n_out - 1) + (SW && i >= 8 ? a.n_out : 0);
    };
    const int8_t *we = a.w + (int64_t)e * a.N * a.K;
    const int8_t *ap = we + (int64_t)wrow(i16) * a.K + grp * 16;
    const u32x4 zero = {0u, 0u, 0u, 0u};
    // the output row of row i of the pass (-1: none) and its row of x
    auto out_row = [&](int i) -> int64_t {
        if (!GROUPED) return i < rows_end ? i : -1;
        const int r = i < rows_end ? a.g.sorted[i] : -1;
        return (uint32_t)r < (uint32_t)a.g.R ? r : -1;
    };
    auto x_row = [&](int64_t r) -> int64_t { return GROUPED && !a.g.per_route ? a.g.token_of((int)r) : r; };
    for (; row0 < rows_end; row0 += 16 * NQ) {
        const int64_t r0 = out_row(row0);
        if (r0 < 0) break;                       // sentinels end the segment
        const int8_t *bp[NQ];
#pragma unroll
        for (int n = 0; n < NQ; ++n) {
            const int64_t r = out_row(row0 + 16 * n + i16);
            bp[n] = a.xq + x_row(r < 0 ? r0 : r) * a.K + grp * 16;
        }
        v4i acc[NQ];
#pragma unroll
        for (int n = 0; n < NQ; ++n) acc[n] = v4i{0, 0, 0, 0};
        for (int k = w * 128; k < a.K; k += NW * 128) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const bool ok = k + 64 * h + grp * 16 < a.K;
                const int o = ok ? k + 64 * h : 0;
                const u32x4 av = ok ? *reinterpret_cast<const u32x4 *>(ap + o) : zero;
#pragma unroll
                for (int n = 0; n < NQ; ++n)
                    acc[n] = mfma64(av, ok ? *reinterpret_cast<const u32x4 *>(bp[n] + o) : zero, acc[n]);
            }
        }
#pragma unroll
        for (int n = 0; n < NQ; ++n)
#pragma unroll
            for (int v = 0; v < 4; ++v) sums[w][(n * 16 + i16) * 17 + 4 * grp + v] = acc[n][v];
        __syncthreads();
        constexpr int COLS = SW ? 8 : 16;
        for (int i = tid; i < 16 * NQ * COLS; i += 64 * NW) {
            const int c = i % COLS, q = i / COLS, col = c0 + c;
            const int64_t r = out_row(row0 + q);
            if (r < 0 || col >= a.n_out) continue;
            int s = 0, u = 0;
            for (int k = 0; k < NW; ++k) {
                s += sums[k][q * 17 + c];
                if (SW) u += sums[k][q * 17 + c + 8];
            }
            const float xs = a.xs[x_row(r)];
            const float *ws = a.ws + (int64_t)e * a.N, *bias = a.bias ? a.bias + (int64_t)e * a.N : nullptr;
            float z = (float)s * xs * ws[col] + (bias ? bias[col] : 0.f);
            if (SW) {
                const int cu = col + a.n_out;
                z = silu(z) * ((float)u * xs * ws[cu] + (bias ? bias[cu] : 0.f));
            } else {
                z = act1(z, a.act);
            }
            if (a.res) z += widen16(a.f16, a.res[r * a.ld_res + col]);
            a.out[r * a.ld_out + col] = narrow16(a.f16, z);
        }
        __syncthreads();
        if (!GROUPED) break;
    }
}

template <bool SW, bool GROUPED>
hipError_t launch(const I8Args &a, hipStream_t st) {
    const int64_t rows = GROUPED ? a.g.sorted_cap / a.g.block_m : (a.M + 31) / 32;
    const dim3 grid((a.n_out + (SW ? 7 : 15)) / (SW ? 8 : 16), (unsigned)rows);
    i8_stream_kernel<2, 8, SW, GROUPED><<<grid, 512, 0, st>>>(a);
    return hipGetLastError();
}

}  // namespace

size_t i8_workspace(I8Args &a, void *ws) {
    if (a.grouped) group_divider(a.g);
    return 0;
}

hipError_t launch_i8(const I8Args &a, hipStream_t st) {
    const bool sw = a.act == kActSwiglu;
    if (a.grouped) return sw ? launch<true, true>(a, st) : launch<false, true>(a, st);
    return sw ? launch<true, false>(a, st) : launch<false, false>(a, st);
}

}  // namespace moe
