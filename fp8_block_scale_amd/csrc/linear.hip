// Dense product of block-scaled E4M3 codes with its epilogue:
//   z[m, n] = sum_kb x_s[m, kb] w_s[n / 128, kb] sum_{k in kb} x_q[m, k] w[n, k] + bias[n]
//   out[m, n] = bf16(act(z)[m, n] + residual[m, n])
// over K-blocks kb of 128.  With SwiGLU act(z)[m, j] = silu(z[m, j]) z[m, I + j].
//
// Two kernels:
//   linear_stream_kernel  few rows: the weights are read once, straight into
//     registers; a workgroup owns 16 weight rows, its waves split K and add up
//     in LDS.
//   linear_tile_kernel    many rows: TQ x TP output tiles from an LDS ring,
//     split over K (FP32 partials, joined by linear_join_kernel) when the
//     tiles alone leave CUs idle.
// In both the weights are the A side of the FP8 MFMA and the rows of x the B
// side, so a lane's results share one row of x (one scale) and run along the
// output's columns.
#include "common.h"
#include "linear.h"

namespace moe {

namespace {

__device__ __forceinline__ int uni(int v) { return __builtin_amdgcn_readfirstlane(v); }

__device__ __forceinline__ v8i join8(const u32x4 &lo, const u32x4 &hi) {
    v8i r;
    r[0] = (int)lo.x; r[1] = (int)lo.y; r[2] = (int)lo.z; r[3] = (int)lo.w;
    r[4] = (int)hi.x; r[5] = (int)hi.y; r[6] = (int)hi.z; r[7] = (int)hi.w;
    return r;
}

__device__ __forceinline__ float silu(float z) {
    return z * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(z * -1.44269504088896340736f));
}
// tanh form: 0.5 z (1 + tanh(u)) = z / (1 + e^-2u), u = sqrt(2 / pi) (z + 0.044715 z^3)
__device__ __forceinline__ float gelu(float z) {
    const float u2 = 1.5957691216057308f * (z + 0.044715f * z * z * z);
    return z * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(u2 * -1.44269504088896340736f));
}
__device__ __forceinline__ float act1(float z, int act) {
    return act == kActSilu ? silu(z) : act == kActGelu ? gelu(z) : z;
}

// ----------------------------------------------------------------- few rows

// 16 weight rows (with SwiGLU 8 gate and their 8 up rows) x 16 NQ rows of x
// per workgroup.  Wave w takes the K-blocks w, w + NW, ...; U of them are
// loaded before the first is multiplied.  NaN codes or scales of rows past
// the end only reach results that are not stored (those lanes read the last
// row instead).
template <int NQ, int NW, int U, bool SW>
__global__ void __launch_bounds__(64 * NW)
linear_stream_kernel(LinearArgs g) {
    __shared__ float red[NW][NQ][16][17];
    const int tid = threadIdx.x, l = tid & 63, w = uni(tid >> 6), i16 = l & 15, grp = l >> 4;
    const int nkb = g.K >> 7;
    const int c0 = blockIdx.x * (SW ? 8 : 16);
    const int64_t m0 = (int64_t)blockIdx.y * (16 * NQ);

    auto wrow = [&](int i) {                     // weight row of MFMA row i
        const int c = c0 + (SW ? i & 7 : i);
        return (c < g.n_out ? c : g.n_out - 1) + (SW && i >= 8 ? g.n_out : 0);
    };
    const uint8_t *ap = g.w + (int64_t)wrow(i16) * g.K + grp * 16;
    const uint8_t *bp[NQ];
    const float *xp[NQ];
    for (int n = 0; n < NQ; ++n) {
        int64_t m = m0 + 16 * n + i16;
        m = m < g.M ? m : g.M - 1;
        bp[n] = g.xq + m * g.K + grp * 16;
        xp[n] = g.xs + m * nkb;
    }
    // a lane's four results are weight rows 4 grp + v; with SwiGLU and an odd
    // number of columns they can straddle a block of 128
    const float *wp[4];
    for (int v = 0; v < 4; ++v) wp[v] = g.ws + (int64_t)(wrow(4 * grp + v) >> 7) * nkb;

    v4f acc[NQ];
    for (int n = 0; n < NQ; ++n) acc[n] = v4f{0.f, 0.f, 0.f, 0.f};
    for (int kb0 = w; kb0 < nkb; kb0 += NW * U) {
        u32x4 a[U][2], b[U][NQ][2];
        float sx[U][NQ], sw[U][SW ? 4 : 1];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int kb = min(kb0 + u * NW, nkb - 1);
            a[u][0] = __builtin_nontemporal_load((const u32x4 *)(ap + (int64_t)kb * 128));
            a[u][1] = __builtin_nontemporal_load((const u32x4 *)(ap + (int64_t)kb * 128 + 64));
#pragma unroll
            for (int n = 0; n < NQ; ++n) {
                b[u][n][0] = *(const u32x4 *)(bp[n] + (int64_t)kb * 128);
                b[u][n][1] = *(const u32x4 *)(bp[n] + (int64_t)kb * 128 + 64);
                sx[u][n] = xp[n][kb];
            }
#pragma unroll
            for (int v = 0; v < (SW ? 4 : 1); ++v) sw[u][v] = wp[v][kb];
        }
        __builtin_amdgcn_sched_barrier(0);       // every load above is issued first
#pragma unroll
        for (int u = 0; u < U; ++u) {
            // past the end the last K-block was read again: its scale is zero
            // (a NaN in it is in the sum already)
            const bool on = kb0 + u * NW < nkb;
            const v8i av = join8(a[u][0], a[u][1]);
#pragma unroll
            for (int n = 0; n < NQ; ++n) {
                const v4f t = mfma16x16x128(av, join8(b[u][n][0], b[u][n][1]));
#pragma unroll
                for (int v = 0; v < 4; ++v) acc[n][v] += t[v] * (on ? sx[u][n] * sw[u][SW ? v : 0] : 0.f);
            }
        }
    }
#pragma unroll
    for (int n = 0; n < NQ; ++n)
#pragma unroll
        for (int v = 0; v < 4; ++v) red[w][n][i16][4 * grp + v] = acc[n][v];
    __syncthreads();
    constexpr int COLS = SW ? 8 : 16;
    for (int i = tid; i < 16 * NQ * COLS; i += 64 * NW) {
        const int c = i % COLS, r = i / COLS;
        const int64_t m = m0 + r;
        const int col = c0 + c;
        if (m >= g.M || col >= g.n_out) continue;
        float z = 0.f, u = 0.f;
        for (int q = 0; q < NW; ++q) {
            z += red[q][r >> 4][r & 15][c];
            if (SW) u += red[q][r >> 4][r & 15][c + 8];
        }
        if (g.bias) {
            z += g.bias[col];
            if (SW) u += g.bias[col + g.n_out];
        }
        z = SW ? silu(z) * u : act1(z, g.act);
        if (g.res) z += bf16_bits_to_f32(g.res[m * g.ld_res + col]);
        g.out[m * g.ld_out + col] = (uint16_t)f32_to_bf16_bits(z);
    }
}

// ---------------------------------------------------------------- many rows

// Weight rows of a tile: LDS row rho of the tile holds weight row
// p0 + rho, or with SwiGLU (per 64 rows: 32 gate rows, then their 32 up rows)
// 32 columns' gate and up rows, so both meet in one wave.
template <int TP, int TQ, int WP, int WQ, int S>
struct LTile {
    static constexpr int NW = WP * WQ;
    static constexpr int PB = TP * 128, QB = TQ * 128, XB = TQ * 4, Stage = PB + QB + XB;
    static constexpr int JP = PB / 1024 / NW, JQ = QB / 1024 / NW;
    static constexpr int XW = TQ / 64;                    // waves that copy 64 scales each
    static constexpr int NP = TP / WP / 16, NQ = TQ / WQ / 16;
    static constexpr size_t Smem = (size_t)S * Stage;
    static_assert(NP % 4 == 0 && JP >= 1 && JQ >= 1 && XW <= NW && Smem <= 160 * 1024, "tile");
};

// The lane's results of a column group: 8 consecutive columns of one row.
struct Store8 {
    const LinearArgs &g;
    bool vec;                                    // 16-byte accesses are aligned
    __device__ __forceinline__ void operator()(int64_t m, int col, float (&z)[8]) const {
        const int n = g.n_out - col;             // valid columns from here
        if (g.res) {
            const uint16_t *r = g.res + m * g.ld_res + col;
            if (vec && n >= 8) {
                const u32x4 o = *reinterpret_cast<const u32x4 *>(r);
#pragma unroll
                for (int v = 0; v < 4; ++v) {
                    z[2 * v] += bf16_bits_to_f32(o[v] & 0xffffu);
                    z[2 * v + 1] += bf16_bits_to_f32(o[v] >> 16);
                }
            } else {
#pragma unroll
                for (int v = 0; v < 8; ++v)
                    if (v < n) z[v] += bf16_bits_to_f32(r[v]);
            }
        }
        uint16_t *d = g.out + m * g.ld_out + col;
        if (vec && n >= 8) {
            u32x4 o;
#pragma unroll
            for (int v = 0; v < 4; ++v) o[v] = f32_to_bf16_bits(z[2 * v]) | (f32_to_bf16_bits(z[2 * v + 1]) << 16);
            *reinterpret_cast<u32x4 *>(d) = o;
        } else {
#pragma unroll
            for (int v = 0; v < 8; ++v)
                if (v < n) d[v] = (uint16_t)f32_to_bf16_bits(z[v]);
        }
    }
};

__device__ __forceinline__ bool vec_ok(const LinearArgs &g) {
    return (((uintptr_t)g.out | (uintptr_t)g.res) & 15u) == 0 && ((g.ld_out | (g.res ? g.ld_res : 0)) & 7) == 0;
}

// GLU: 0 no SwiGLU; 1 SwiGLU; 2 SwiGLU whose up rows in a wave may straddle
// two blocks of 128 weight rows (N / 2 no multiple of 32).
template <int TP, int TQ, int WP, int WQ, int S, int GLU>
__global__ void __launch_bounds__(64 * WP * WQ)
linear_tile_kernel(LinearArgs g) {
    using T = LTile<TP, TQ, WP, WQ, S>;
    constexpr bool SW = GLU != 0;
    constexpr int NW = T::NW, JP = T::JP, JQ = T::JQ, NP = T::NP, NQ = T::NQ;
    constexpr int TC = SW ? TP / 2 : TP;                  // output columns of a tile
    extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
    const int tid = threadIdx.x, l = tid & 63, w = uni(tid >> 6);
    const int wp = w % WP, wq = w / WP, i16 = l & 15, grp = l >> 4;
    const int nkb = g.K >> 7;
    const int nct = (g.n_out + TC - 1) / TC;
    const int n_items = (int)((g.M + TQ - 1) / TQ) * nct * g.nsplit;
    const int xcd = blockIdx.x & 7, step = gridDim.x >> 3;
    const int end = (int)((int64_t)(xcd + 1) * n_items / 8);
    int lit = (int)((int64_t)xcd * n_items / 8) + (blockIdx.x >> 3), cit = lit;
    if (cit >= end) return;
    const int per = (nkb + g.nsplit - 1) / g.nsplit;      // K-blocks per split (none empty)

    // ---- load side
    const uint8_t *pbase = nullptr, *qbase = nullptr;
    const float *xbase = nullptr;
    uint32_t poff[JP], qoff[JQ], xoff = 0;
    int lkb = 0, lkend = 0;
    const int kc_p = (l & 7) ^ (((l >> 3) & 3) | ((w & 1) << 2));
    const int kc_q = (l & 7) ^ (l >> 3);
    auto load_setup = [&]() {
        int i = lit;
        const int sp = i % g.nsplit;
        i /= g.nsplit;
        const int ct = i % nct;
        const int64_t m0 = (int64_t)(i / nct) * TQ;
        lkb = sp * per;
        lkend = min(lkb + per, nkb);
        const int c0 = ct * TC;
        pbase = g.w + (int64_t)c0 * g.K;
#pragma unroll
        for (int j = 0; j < JP; ++j) {
            const int rho = 8 * (j * NW + w) + (l >> 3);
            int c = SW ? (rho >> 6) * 32 + (rho & 31) : rho;
            c = c0 + c < g.n_out ? c : g.n_out - 1 - c0;
            // an up row lies N / 2 rows further: up to 2^39 bytes, so its
            // offset is taken in 16-byte units
            poff[j] = (uint32_t)(((int64_t)(c + (SW && (rho & 32) ? g.n_out : 0)) * g.K) >> 4) + (uint32_t)kc_p;
        }
        qbase = g.xq + m0 * g.K;
        xbase = g.xs + m0 * nkb;
        const int rows = (int)min((int64_t)TQ, g.M - m0);
#pragma unroll
        for (int j = 0; j < JQ; ++j) {
            const int row = 8 * (j * NW + w) + (l >> 3);
            qoff[j] = (uint32_t)(row < rows ? row : rows - 1) * (uint32_t)g.K + (uint32_t)kc_q * 16u;
        }
        const int row = (w % T::XW) * 64 + l;
        xoff = (uint32_t)(row < rows ? row : rows - 1) * (uint32_t)nkb;
    };
    auto issue = [&](int slot) {
        uint8_t *sp = smem + slot * T::Stage, *sq = sp + T::PB, *sx = sq + T::QB;
        const int64_t k0 = (int64_t)lkb * 128;
#pragma unroll
        for (int j = 0; j < JP; ++j) lds_dma16(pbase + k0 + ((uint64_t)poff[j] << 4), sp + (j * NW + w) * 1024);
#pragma unroll
        for (int j = 0; j < JQ; ++j) lds_dma16(qbase + k0 + qoff[j], sq + (j * NW + w) * 1024);
        if (w < T::XW) lds_dma4(xbase + lkb + xoff, sx + w * 256);
        if (++lkb == lkend) {
            lit += step;
            if (lit < end) load_setup();
        }
    };

    // ---- compute side
    v4f acc[NP][NQ];
    auto clear = [&]() {
#pragma unroll
        for (int a = 0; a < NP; ++a)
#pragma unroll
            for (int b = 0; b < NQ; ++b) acc[a][b] = v4f{0.f, 0.f, 0.f, 0.f};
    };
    const int pf = (i16 & 3) | (((i16 >> 2) & 1) << 2);
    const int p_off = (wp * (TP / WP) + 8 * (i16 >> 2) + (i16 & 3)) * 128 + ((grp ^ pf) << 4);
    const int q_off = (wq * (TQ / WQ) + i16) * 128 + ((grp ^ (i16 & 7)) << 4);
    int ckb = 0, ckend = 0, cc0 = 0, csp = 0;
    int64_t cm0 = 0;
    // weight scales: one block of 128 rows per 64-row wave slice (gate and up
    // apart); where its up rows straddle two, rows from `cut` on take the second
    const float *w0 = nullptr, *w1 = nullptr, *w2 = nullptr;
    int cut = 1 << 30;
    auto comp_setup = [&]() {
        int i = cit;
        csp = i % g.nsplit;
        i /= g.nsplit;
        cc0 = (i % nct) * TC;
        cm0 = (int64_t)(i / nct) * TQ;
        ckb = csp * per;
        ckend = min(ckb + per, nkb);
        static_assert(TP / WP == 64, "a wave's columns lie in one block of 128");
        const int c = cc0 + wp * (SW ? 32 : 64);
        const int last = ((SW ? 2 * g.n_out : g.n_out) - 1) >> 7;
        w0 = g.ws + (int64_t)min(c >> 7, last) * nkb;
        if (SW) {
            const int b = (c + g.n_out) >> 7;
            w1 = g.ws + (int64_t)min(b, last) * nkb;
            w2 = g.ws + (int64_t)min(b + 1, last) * nkb;
            cut = ((b + 1) << 7) - (c + g.n_out);       // of the wave's 32 up rows
        }
    };
    auto compute = [&](int slot) {
        const uint8_t *sp = smem + slot * T::Stage, *sq = sp + T::PB;
        const float *sx = reinterpret_cast<const float *>(sq + T::QB);
        const float s0 = w0[ckb], s1 = SW ? w1[ckb] : 0.f, s2 = GLU == 2 ? w2[ckb] : 0.f;
        v8i a[NP];
#pragma unroll
        for (int m = 0; m < NP; ++m) {
            const int o = (m >> 1) * 32 * 128 + (m & 1) * 4 * 128;
            a[m] = join8(lds_read16(sp + p_off + o), lds_read16(sp + (p_off ^ 64) + o));
        }
#pragma unroll
        for (int n = 0; n < NQ; ++n) {
            const v8i b = join8(lds_read16(sq + q_off + n * 2048), lds_read16(sq + (q_off ^ 64) + n * 2048));
            const float x = sx[wq * (TQ / WQ) + n * 16 + i16];
#pragma unroll
            for (int m = 0; m < NP; ++m) {
                const v4f t = mfma16x16x128(a[m], b);
                if (GLU == 2 && m >= 2) {
                    const int r = 8 * grp + 4 * (m & 1);         // the lane's first up row of four
#pragma unroll
                    for (int v = 0; v < 4; ++v) acc[m][n][v] += t[v] * (x * (r + v < cut ? s1 : s2));
                } else {
                    const float s = x * (SW && m >= 2 ? s1 : s0);
#pragma unroll
                    for (int v = 0; v < 4; ++v) acc[m][n][v] += t[v] * s;
                }
            }
        }
    };
    const Store8 store{g, vec_ok(g)};
    auto epilogue = [&]() {
        const int cw = cc0 + wp * (SW ? 32 : 64) + 8 * grp;
#pragma unroll
        for (int n = 0; n < NQ; ++n) {
            const int64_t m = cm0 + wq * (TQ / WQ) + 16 * n + i16;
            if (m >= g.M) continue;
#pragma unroll
            for (int p = 0; p < NP / 2; ++p) {
                const int c = cw + (SW ? 0 : 32 * p);
                if (c >= g.n_out) continue;
                if (g.nsplit > 1) {              // FP32 partial of z, columns as the weight rows
                    float *d = g.part + ((int64_t)csp * g.M + m) * g.ld_part + c + (SW && p ? g.n_out : 0);
#pragma unroll
                    for (int v = 0; v < 8; ++v)
                        if (c + v < g.n_out) d[v] = acc[2 * p + (v >> 2)][n][v & 3];
                    continue;
                }
                if (SW && p) continue;
                float z[8];
#pragma unroll
                for (int v = 0; v < 8; ++v) {
                    z[v] = acc[2 * p + (v >> 2)][n][v & 3];
                    float u = SW ? acc[2 + (v >> 2)][n][v & 3] : 0.f;
                    if (g.bias && c + v < g.n_out) {
                        z[v] += g.bias[c + v];
                        if (SW) u += g.bias[c + v + g.n_out];
                    }
                    z[v] = SW ? silu(z[v]) * u : act1(z[v], g.act);
                }
                store(m, c, z);
            }
        }
    };

    load_setup();
    comp_setup();
    clear();
    int issued = 0, done = 0;
    auto issue_next = [&]() {
        if (lit >= end) return;
        issue(issued % S);
        ++issued;
    };
    for (int s = 0; s < S - 1; ++s) issue_next();
    while (true) {
        // the stage's copies have landed for this wave, then for all; every
        // read of the slot the next copies overwrite is complete
        constexpr int ahead = (S - 2) * (JP + JQ);
        if (S > 2 && issued - done == S - 1) wait_vmcnt<(ahead < 63 ? ahead : 63)>();
        else wait_vmcnt<0>();
        __builtin_amdgcn_s_waitcnt(0xC07F);               // lgkmcnt(0)
        stage_barrier();
        issue_next();
        compute(done % S);
        ++done;
        if (++ckb == ckend) {
            epilogue();
            cit += step;
            if (cit >= end) break;
            comp_setup();
            clear();
        }
    }
}

// Adds the splits of z in order, then the epilogue; 8 columns per thread.
__global__ void __launch_bounds__(256)
linear_join_kernel(LinearArgs g) {
    const int per = (g.n_out + 7) / 8;
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= g.M * per) return;
    const int64_t m = i / per;
    const int c = (int)(i - m * per) * 8;
    const bool sw = g.act == kActSwiglu;
    float z[8], u[8];
    for (int v = 0; v < 8; ++v) z[v] = u[v] = 0.f;
    for (int s = 0; s < g.nsplit; ++s) {
        const float *p = g.part + ((int64_t)s * g.M + m) * g.ld_part + c;
        for (int v = 0; v < 8; ++v)
            if (c + v < g.n_out) {
                z[v] += p[v];
                if (sw) u[v] += p[v + g.n_out];
            }
    }
    for (int v = 0; v < 8; ++v) {
        if (g.bias && c + v < g.n_out) {
            z[v] += g.bias[c + v];
            if (sw) u[v] += g.bias[c + v + g.n_out];
        }
        z[v] = sw ? silu(z[v]) * u[v] : act1(z[v], g.act);
    }
    Store8{g, vec_ok(g)}(m, c, z);
}

// ----------------------------------------------------------------- launch

template <int TP, int TQ, int WP, int WQ, int S, int GLU>
hipError_t launch_tile(const LinearArgs &g, hipStream_t st) {
    using T = LTile<TP, TQ, WP, WQ, S>;
    static std::atomic<uint64_t> done{0};
    auto fn = linear_tile_kernel<TP, TQ, WP, WQ, S, GLU>;
    hipError_t e = raise_lds_limit(done, (const void *)fn, (int)T::Smem);
    if (e != hipSuccess) return e;
    const int tc = GLU ? TP / 2 : TP;
    const int64_t items = ((g.M + TQ - 1) / TQ) * ((g.n_out + tc - 1) / tc) * g.nsplit;
    int64_t grid = (int64_t)device_cu_count() * (2 * T::Smem <= 160 * 1024 ? 2 : 1);
    if (grid > items) grid = items;
    grid = (grid + 7) / 8 * 8;
    fn<<<(unsigned)grid, 64 * WP * WQ, T::Smem, st>>>(g);
    e = hipGetLastError();
    if (e != hipSuccess || g.nsplit == 1) return e;
    const int64_t n = g.M * ((g.n_out + 7) / 8);
    linear_join_kernel<<<(unsigned)((n + 255) / 256), 256, 0, st>>>(g);
    return hipGetLastError();
}

template <int GLU>
hipError_t launch(const LinearArgs &g, hipStream_t st) {
    constexpr bool SW = GLU != 0;
    switch (g.form) {
        case kLinStream1:
        case kLinStream2:
        case kLinStream4: {
            const int nq = g.form == kLinStream1 ? 1 : g.form == kLinStream2 ? 2 : 4;
            const dim3 grid((g.n_out + (SW ? 7 : 15)) / (SW ? 8 : 16), (unsigned)((g.M + 16 * nq - 1) / (16 * nq)));
            if (nq == 1) linear_stream_kernel<1, 8, 7, SW><<<grid, 512, 0, st>>>(g);
            else if (nq == 2) linear_stream_kernel<2, 8, 4, SW><<<grid, 512, 0, st>>>(g);
            else linear_stream_kernel<4, 8, 2, SW><<<grid, 512, 0, st>>>(g);
            return hipGetLastError();
        }
        case kLinTile256:
            if constexpr (GLU < 2) return launch_tile<256, 256, 4, 2, 2, GLU>(g, st);
            [[fallthrough]];
        case kLinTile128: return launch_tile<256, 128, 4, 2, 3, GLU>(g, st);
        default: return launch_tile<128, 64, 2, 2, 3, GLU>(g, st);
    }
}

}  // namespace

size_t linear_workspace(LinearArgs &a, void *ws) {
    const int n = a.act == kActSwiglu ? 2 * a.n_out : a.n_out;     // weight rows
    const int nkb = a.K / 128;
    auto items = [&](int tp, int tq) { return ((a.M + tq - 1) / tq) * ((n + tp - 1) / tp); };
    a.nsplit = 1;
    a.part = nullptr;
    if (a.M <= 64) {
        a.form = a.M <= 16 ? kLinStream1 : a.M <= 32 ? kLinStream2 : kLinStream4;
        return 0;
    }
    if (items(256, 256) >= 200) a.form = kLinTile256;
    else if (items(256, 128) >= 200) a.form = kLinTile128;
    else {
        a.form = kLinTile64;
        int64_t s = 512 / items(128, 64);
        if (s > nkb / 4) s = nkb / 4;
        if (s > 1) {
            const int per = (int)((nkb + s - 1) / s);
            a.nsplit = (nkb + per - 1) / per;                      // none empty
        }
    }
    a.ld_part = (n + 3) / 4 * 4;
    if (a.nsplit == 1) return 0;
    a.part = (float *)ws;
    return (size_t)a.nsplit * a.M * a.ld_part * 4;
}

hipError_t launch_linear(const LinearArgs &a, hipStream_t st) {
    if (a.act != kActSwiglu) return launch<0>(a, st);
    return a.n_out % 32 == 0 ? launch<1>(a, st) : launch<2>(a, st);
}

}  // namespace moe
