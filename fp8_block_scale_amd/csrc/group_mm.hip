// Matrix products grouped by expert, ragged, in BF16 or FP16 (FP32 sums):
//   forward   y[r, n]     = sum_k x[t(r), k] w[e(r), n, k]
//   dx        dx[t, k]    = sum_{r: t(r) = t} sum_n dy[r, n] w[e(r), n, k]
//   dw        dw[e, n, k] = sum_{r in e} dy[r, n] x[t(r), k]
// over the routes r that the plan lists for each expert e; t(r) = r / top_k
// (token rows) or r (one row per route).
//
// One 64 x 64 output tile per workgroup, both operands staged through LDS.
#include "common.h"
#include "group_mm.h"

namespace moe {

namespace {

typedef __bf16 v8bf __attribute__((ext_vector_type(8)));

template <bool F16>
__device__ __forceinline__ v4f mfma32(const u32x4 &a, const u32x4 &b, const v4f &c) {
    if constexpr (F16)
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(v8h, a), __builtin_bit_cast(v8h, b), c,
                                                      0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, a),
                                                       __builtin_bit_cast(v8bf, b), c, 0, 0, 0);
}

template <bool F16>
__device__ __forceinline__ uint16_t to16(float v) {
    if constexpr (F16) return __builtin_bit_cast(uint16_t, (_Float16)v);
    else return (uint16_t)f32_to_bf16_bits(v);
}

template <bool F16>
__device__ __forceinline__ float from16(uint16_t v) {
    if constexpr (F16) return (float)__builtin_bit_cast(_Float16, v);
    else return bf16_bits_to_f32(v);
}

// first block in [0, nb) whose expert is >= e (expert ids never decrease)
__device__ __forceinline__ int first_block(const int32_t *eids, int nb, int e) {
    int lo = 0, hi = nb;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (eids[mid] < e) lo = mid + 1;
        else hi = mid;
    }
    return lo;
}

constexpr int kLd = 40;    // LDS row of 32 contraction values, padded

template <bool F16>
__device__ __forceinline__ void tile_step(const uint16_t (*p)[kLd], const uint16_t (*q)[kLd], int wp, int wq,
                                          v4f (&acc)[2][2]) {
    const int l = threadIdx.x & 63;
    u32x4 a[2], b[2];
    for (int i = 0; i < 2; ++i) {
        a[i] = *(const u32x4 *)&p[wp * 32 + i * 16 + (l & 15)][(l >> 4) * 8];
        b[i] = *(const u32x4 *)&q[wq * 32 + i * 16 + (l & 15)][(l >> 4) * 8];
    }
    for (int i = 0; i < 2; ++i)
        for (int j = 0; j < 2; ++j) acc[i][j] = mfma32<F16>(a[i], b[j], acc[i][j]);
}

template <bool F16, int OP>
__global__ void __launch_bounds__(256)
group_mm_kernel(GroupMmArgs g) {
    __shared__ uint16_t p[64][kLd], q[64][kLd];
    __shared__ int rid[64];
    const int tid = threadIdx.x, l = tid & 63, w = tid >> 6, wp = w & 1, wq = w >> 1;
    const int bm = g.block_m;
    int P = g.ntp ? *g.ntp : 0;
    P = P < g.sorted_cap ? P : (int)g.sorted_cap;
    const int nb = P / bm;
    int e, row0 = 0, rows, nred;
    const int p0 = (OP == kGmmDw ? blockIdx.x : blockIdx.y) * 64;
    if (OP == kGmmDw) {
        e = blockIdx.z;
        const int b0 = first_block(g.eids, nb, e), b1 = first_block(g.eids, nb, e + 1);
        row0 = b0 * bm;
        nred = (b1 - b0) * bm;
        rows = 0;
    } else {
        const int b = blockIdx.x;
        if (b >= nb) return;
        e = g.eids[b];
        if (e < 0 || e >= g.E) return;
        row0 = b * bm + blockIdx.z * 64;
        rows = bm - (int)blockIdx.z * 64;
        rows = rows < 64 ? rows : 64;
        nred = OP == kGmmFwd ? g.K : g.N;
        if (tid < 64) rid[tid] = tid < rows ? g.sorted[row0 + tid] : (int)g.R;
        __syncthreads();
    }
    const int np = OP == kGmmFwd ? g.N : g.K;          // output columns
    const uint16_t *we = g.w + (int64_t)e * g.N * g.K;
    v4f acc[2][2] = {};
    for (int k0 = 0; k0 < nred; k0 += 32) {
        __syncthreads();
        for (int i = tid; i < 64 * 32; i += 256) {
            uint16_t vp = 0, vq = 0;
            if (OP == kGmmDw) {
                const int c = i & 63, k = k0 + (i >> 6);
                const int r = k < nred ? g.sorted[row0 + k] : -1;
                if (r >= 0 && r < g.R) {
                    const int64_t xr = g.per_route ? r : r / g.top_k;
                    if (p0 + c < g.K) vp = g.x[xr * g.ld_x + p0 + c];
                    if ((int)blockIdx.y * 64 + c < g.N) vq = g.dy[(int64_t)r * g.ld_dy + blockIdx.y * 64 + c];
                }
                p[c][i >> 6] = vp;
                q[c][i >> 6] = vq;
            } else if (OP == kGmmFwd) {
                const int c = i >> 5, k = k0 + (i & 31);
                const int r = rid[c];
                if (k < nred) {
                    if (p0 + c < np) vp = we[(int64_t)(p0 + c) * g.K + k];
                    if (r >= 0 && r < g.R) vq = g.x[(int64_t)(g.per_route ? r : r / g.top_k) * g.ld_x + k];
                }
                p[c][i & 31] = vp;
                q[c][i & 31] = vq;
            } else {
                const int c = i & 63, k = k0 + (i >> 6);
                if (k < nred && p0 + c < np) vp = we[(int64_t)k * g.K + p0 + c];
                p[c][i >> 6] = vp;
                const int c2 = i >> 5, k2 = k0 + (i & 31);
                const int r = rid[c2];
                if (k2 < nred && r >= 0 && r < g.R) vq = g.dy[(int64_t)r * g.ld_dy + k2];
                q[c2][i & 31] = vq;
            }
        }
        __syncthreads();
        tile_step<F16>(p, q, wp, wq, acc);
    }
    for (int i = 0; i < 2; ++i)
        for (int j = 0; j < 2; ++j)
            for (int v = 0; v < 4; ++v) {
                const int c = p0 + wp * 32 + i * 16 + 4 * (l >> 4) + v;
                const int qr = wq * 32 + j * 16 + (l & 15);
                if (c >= np) continue;
                if (OP == kGmmDw) {
                    const int n = blockIdx.y * 64 + qr;
                    if (n >= g.N) continue;
                    const int64_t o = ((int64_t)e * g.N + n) * g.K + c;
                    float s = acc[i][j][v];
                    if (g.out_f32) {
                        float *d = (float *)g.out + o;
                        *d = g.accumulate ? *d + s : s;
                    } else {
                        uint16_t *d = (uint16_t *)g.out + o;
                        *d = to16<F16>(g.accumulate ? from16<F16>(*d) + s : s);
                    }
                } else {
                    const int r = rid[qr];
                    if (r < 0 || r >= g.R) continue;
                    if (OP == kGmmDx && !g.per_route) g.part[(int64_t)r * g.K + c] = acc[i][j][v];
                    else ((uint16_t *)g.out)[(int64_t)r * g.ld_out + c] = to16<F16>(acc[i][j][v]);
                }
            }
}

__global__ void __launch_bounds__(256)
group_mark_kernel(GroupMmArgs g) {
    int P = *g.ntp;
    P = P < g.sorted_cap ? P : (int)g.sorted_cap;
    for (int i = blockIdx.x * 256 + threadIdx.x; i < P; i += gridDim.x * 256) {
        const int r = g.sorted[i];
        if (r >= 0 && r < g.R) g.rpos[r] = i;
    }
}

template <bool F16>
__global__ void __launch_bounds__(256)
group_sum_kernel(GroupMmArgs g) {
    const int64_t t = blockIdx.x;
    for (int c = threadIdx.x; c < g.K; c += 256) {
        float s = 0.f;
        for (int j = 0; j < g.top_k; ++j) {
            const int64_t r = t * g.top_k + j;
            if (g.rpos[r] >= 0) s += g.part[r * g.K + c];
        }
        ((uint16_t *)g.out)[t * g.ld_out + c] = to16<F16>(s);
    }
}

template <bool F16>
hipError_t launch(const GroupMmArgs &g, hipStream_t st) {
    const unsigned blocks = (unsigned)(g.sorted_cap / g.block_m);
    if (g.op == kGmmDw) {
        dim3 grid((g.K + 63) / 64, (g.N + 63) / 64, g.E);
        group_mm_kernel<F16, kGmmDw><<<grid, 256, 0, st>>>(g);
        return hipGetLastError();
    }
    const int sub = (g.block_m + 63) / 64;
    if (g.op == kGmmFwd) {
        group_mm_kernel<F16, kGmmFwd><<<dim3(blocks, (g.N + 63) / 64, sub), 256, 0, st>>>(g);
        return hipGetLastError();
    }
    if (!g.per_route) {
        hipError_t e = launch_fill((uint32_t *)g.rpos, (size_t)g.R, 0xffffffffu, st);
        if (e != hipSuccess) return e;
        group_mark_kernel<<<256, 256, 0, st>>>(g);
    }
    group_mm_kernel<F16, kGmmDx><<<dim3(blocks, (g.K + 63) / 64, sub), 256, 0, st>>>(g);
    if (!g.per_route) group_sum_kernel<F16><<<(unsigned)g.M, 256, 0, st>>>(g);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_group_mm(const GroupMmArgs &g, hipStream_t st) {
    return g.f16 ? launch<true>(g, st) : launch<false>(g, st);
}

size_t group_mm_workspace(GroupMmArgs &g, void *ws) {
    uint8_t *base = (uint8_t *)ws;
    size_t off = 0;
    if (g.op == kGmmDx && !g.per_route) {
        g.rpos = (int32_t *)(base + off);
        off += ((size_t)g.R * 4 + 255) & ~size_t(255);
        g.part = (float *)(base + off);
        off += ((size_t)g.R * g.K * 4 + 255) & ~size_t(255);
    }
    return off;
}

}  // namespace moe
