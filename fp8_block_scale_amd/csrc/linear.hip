// Dense product of block-scaled E4M3 codes with its epilogue:
//   z[m, n] = sum_kb x_s[m, kb] w_s[n / 128, kb] sum_{k in kb} x_q[m, k] w[n, k] + bias[n]
//   out[m, n] = bf16(act(z)[m, n] + residual[m, n])
// over K-blocks kb of 128.  With SwiGLU act(z)[m, j] = silu(z[m, j]) z[m, I + j].
//
// Two kernels:
//   linear_stream_kernel  few rows (up to 1024, by size): weights straight into
//     registers; a workgroup owns 16 weight rows, for 16 to 64 rows of x; its
//     waves split K and add up in LDS.
//   linear_tile_kernel    many rows: TQ x TP output tiles from an LDS ring,
//     split over K (FP32 partials, joined by linear_join_kernel) when the
//     tiles alone leave CUs idle.
// In both the weights are the A side of the FP8 MFMA and the rows of x the B
// side, so a lane's results share one row of x (one scale) and run along the
// output's columns.  The MFMA adds to nothing: each K-block's sum is scaled
// and added to the FP32 accumulators by the vector unit, beside the MFMAs of
// the next.
//
// Fewer bits than FP32, and why.  The FP8 MFMA sums its 128 products in fixed
// point, cut some 15 bits below the largest; everything after it (scales, sum
// over K-blocks, bias, activation, residual) is FP32.  Widened to FP16 the
// products would be exact, but the FP16 MFMA has half the rate, before the
// conversions.  Measured on random codes of K = 2048 to 7168 the value before
// the last rounding is off by 5.5e-6 of the result's norm (7.5e-6 with
// SwiGLU), 1/300 of the rounding to BF16 that follows (1.7e-3).  SiLU and GELU
// take the hardware's reciprocal and exp2, one unit in the last place each.
//
// Measured: 8192 x 4096 x 7168 with bias, SiLU and residual 0.242 ms, 1.99
// PFLOP/s, with its operands in the last-level cache, 0.267 ms from HBM (a
// plain FP8 library product without block scales reaches 3.0 at 8192 cubed):
// the matrix cores are busy 40% of the time and the scaling's vector
// instructions as long again, at 2.0 GHz on random codes; zeros, at 2.3 GHz,
// are 13% faster.  1000 x 1001 x 2048: 15.9 us, bound by latency: 12 us for 8
// steps of a three-stage ring, alone on its CU, 4 us for the join's launch.
#include <algorithm>

#include "linear.h"
#include "tiles.h"

namespace moe {

namespace {

__device__ __forceinline__ v8i join8(const u32x4 &lo, const u32x4 &hi) {
    v8i r;
    r[0] = (int)lo.x; r[1] = (int)lo.y; r[2] = (int)lo.z; r[3] = (int)lo.w;
    r[4] = (int)hi.x; r[5] = (int)hi.y; r[6] = (int)hi.z; r[7] = (int)hi.w;
    return r;
}

// ----------------------------------------------------------------- few rows

// 16 weight rows (with SwiGLU 8 gate and their 8 up rows) x 16 NQ rows of x
// per workgroup.  Wave w takes the K-blocks w, w + NW, ...; U of them are
// loaded before the first is multiplied, and the waves' sums are added in
// order.  Rows past the end read the last row: their results are not stored.
//
// Bound by the reads of x and w from the L2 (each workgroup reads all of its
// rows of both).  Weights go straight into registers.  Rows of x that differ
// (XL) are copied to the wave's share of LDS, 8 whole rows of 128 bytes an
// instruction, and read from there: register loads in the operand's layout
// touch 16 rows, 64 bytes each, and ran at some 13 bytes a clock and CU.
// Measured (us, registers -> LDS), K = 4096, N = 2048: 16 rows 6.5 -> 5.4, 32
// rows 12.6 -> 6.7, 48 rows 12.1 -> 8.3, 64 rows 15.3 -> 9.8; one row, whose
// 16 copies are one line, 4.3 -> 4.7, so up to 4 rows stay in registers.
// One row at K = 7168, N = 4096 takes 8.5 us (29 MB, 3.5 TB/s with the launch).

// Bytes of LDS of nw waves: their rows of x, then their sums.
constexpr int stream_lds(int nq, int nw, int u, bool xl) {
    const int sums = (nq * 16 * 17 * 4 + 15) / 16 * 16, x = xl ? u * nq * 2048 : 0;
    return nw * (x > sums ? x : sums);
}

template <int NQ, int NW, int U, bool SW, bool XL>
__global__ void __launch_bounds__(64 * NW)
linear_stream_kernel(LinearArgs g) {
    // a wave's share of LDS: its rows of x (XL), then its sums [NQ][16][17]
    constexpr int kWave = stream_lds(NQ, 1, U, XL);
    extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
    const int tid = threadIdx.x, l = tid & 63, w = uni(tid >> 6), i16 = l & 15, grp = l >> 4;
    const int nkb = g.K >> 7;
    const int c0 = blockIdx.x * (SW ? 8 : 16), m0 = blockIdx.y * (16 * NQ);

    auto wrow = [&](int i) {                     // weight row of MFMA row i
        const int c = c0 + (SW ? i & 7 : i);
        return (c < g.n_out ? c : g.n_out - 1) + (SW && i >= 8 ? g.n_out : 0);
    };
    const uint8_t *ap = g.w + (int64_t)wrow(i16) * g.K + grp * 16;
    uint8_t *const lds = smem + w * kWave;
    const uint8_t *bp[XL ? 2 * NQ : NQ];
    const float *xp[NQ];
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
        const int64_t m = min(m0 + 16 * n + i16, (int)g.M - 1);
        if (!XL) bp[n] = g.xq + m * g.K + grp * 16;
        xp[n] = g.xs + m * nkb;
    }
    if (XL) {
        // copies of 8 rows x 128 bytes; chunk c of row r lies at c ^ (r & 7)
#pragma unroll
        for (int j = 0; j < 2 * NQ; ++j) {
            const int64_t m = min(m0 + 8 * j + (l >> 3), (int)g.M - 1);
            bp[j] = g.xq + m * g.K + ((l & 7) ^ (l >> 3)) * 16;
        }
    }
    const int x_off = i16 * 128 + ((grp ^ (i16 & 7)) << 4);
    // a lane's four results are weight rows 4 grp + v; with SwiGLU and an odd
    // number of columns they can straddle a block of 128
    const float *wp[4];
    for (int v = 0; v < 4; ++v) wp[v] = g.ws + (int64_t)(wrow(4 * grp + v) >> 7) * nkb;

    v4f acc[NQ];
#pragma unroll
    for (int n = 0; n < NQ; ++n) acc[n] = v4f{0.f, 0.f, 0.f, 0.f};
    for (int kb0 = w; kb0 < nkb; kb0 += NW * U) {
        u32x4 a[U][2], b[U][NQ][2];
        float sx[U][NQ], sw[U][SW ? 4 : 1];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int kb = kb0 + u * NW;
            if (kb >= nkb) break;
            a[u][0] = __builtin_nontemporal_load((const u32x4 *)(ap + (int64_t)kb * 128));
            a[u][1] = __builtin_nontemporal_load((const u32x4 *)(ap + (int64_t)kb * 128 + 64));
#pragma unroll
            for (int n = 0; n < NQ; ++n) {
                if (XL) {
                    lds_dma16(bp[2 * n] + (int64_t)kb * 128, lds + (u * NQ + n) * 2048);
                    lds_dma16(bp[2 * n + 1] + (int64_t)kb * 128, lds + (u * NQ + n) * 2048 + 1024);
                } else {
                    b[u][n][0] = *(const u32x4 *)(bp[n] + (int64_t)kb * 128);
                    b[u][n][1] = *(const u32x4 *)(bp[n] + (int64_t)kb * 128 + 64);
                }
                sx[u][n] = xp[n][kb];
            }
#pragma unroll
            for (int v = 0; v < (SW ? 4 : 1); ++v) sw[u][v] = wp[v][kb];
        }
        __builtin_amdgcn_sched_barrier(0);       // every load above is issued first
        if (XL) {
            asm volatile("s_waitcnt vmcnt(0)" ::: "memory");       // the wave's own copies
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int n = 0; n < NQ; ++n) {
                    if (kb0 + u * NW >= nkb) break;
                    b[u][n][0] = lds_read16(lds + (u * NQ + n) * 2048 + x_off);
                    b[u][n][1] = lds_read16(lds + (u * NQ + n) * 2048 + (x_off ^ 64));
                }
            // read before the next round's copies write there
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (kb0 + u * NW >= nkb) break;
            const v8i av = join8(a[u][0], a[u][1]);
#pragma unroll
            for (int n = 0; n < NQ; ++n) {
                const v4f t = mfma16x16x128(av, join8(b[u][n][0], b[u][n][1]));
#pragma unroll
                for (int v = 0; v < 4; ++v) acc[n][v] += t[v] * (sx[u][n] * sw[u][SW ? v : 0]);
            }
        }
    }
#pragma unroll
    for (int n = 0; n < NQ; ++n)
#pragma unroll
        for (int v = 0; v < 4; ++v)
            reinterpret_cast<float *>(lds)[(n * 16 + i16) * 17 + 4 * grp + v] = acc[n][v];
    __syncthreads();
    constexpr int COLS = SW ? 8 : 16;
    for (int i = tid; i < 16 * NQ * COLS; i += 64 * NW) {
        const int c = i % COLS, r = i / COLS;
        const int64_t m = m0 + r;
        const int col = c0 + c;
        if (m >= g.M || col >= g.n_out) continue;
        float z = 0.f, u = 0.f;
        for (int q = 0; q < NW; ++q) {
            const float *d = reinterpret_cast<const float *>(smem + q * kWave) + r * 17 + c;
            z += d[0];
            if (SW) u += d[8];
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
    static constexpr int PB = TP * 128, QB = TQ * 128, XB = TQ * 4, WB = 256, Stage = PB + QB + XB + WB;
    static constexpr int JP = PB / 1024 / NW, JQ = QB / 1024 / NW;
    static constexpr int XW = TQ / 64;                    // waves that copy 64 scales of x each; the last wave
                                                          // copies the weights'
    static constexpr int NP = TP / WP / 16, NQ = TQ / WQ / 16;
    static constexpr size_t Smem = (size_t)S * Stage;
    static_assert(NP % 4 == 0 && JP >= 1 && JQ >= 1 && XW < NW && Smem <= 160 * 1024, "tile");
};

// A lane's results of a column group are 8 consecutive columns of one row.
// Rows of an odd number of columns are 2-byte aligned only: global memory
// takes 16-byte accesses at any alignment.
typedef u32x4 u32x4_any __attribute__((aligned(2)));
typedef v4f v4f_any __attribute__((aligned(4)));

// b[0, 8) = bias[c, c + 8), 0 past n (and without a bias)
__device__ __forceinline__ void load_bias8(const float *bias, int c, int n, float (&b)[8]) {
#pragma unroll
    for (int v = 0; v < 8; ++v) b[v] = 0.f;
    if (!bias) return;
    if (c + 8 <= n) {
        const v4f lo = *reinterpret_cast<const v4f_any *>(bias + c), hi = *reinterpret_cast<const v4f_any *>(bias + c + 4);
#pragma unroll
        for (int v = 0; v < 4; ++v) {
            b[v] = lo[v];
            b[4 + v] = hi[v];
        }
    } else {
#pragma unroll
        for (int v = 0; v < 8; ++v)
            if (c + v < n) b[v] = bias[c + v];
    }
}

__device__ __forceinline__ void act8(float (&z)[8], int act) {
    if (act == kActSilu) {
#pragma unroll
        for (int v = 0; v < 8; ++v) z[v] = silu(z[v]);
    } else if (act == kActGelu) {
#pragma unroll
        for (int v = 0; v < 8; ++v) z[v] = gelu(z[v]);
    }
}

// z += residual, out = bf16(z) at row m, columns [col, col + 8); `res` holds
// the residual's 8 values where all 8 columns exist.
__device__ __forceinline__ void store8(const LinearArgs &g, int64_t m, int col, float (&z)[8], const u32x4 &res) {
    uint16_t *d = g.out + m * g.ld_out + col;
    if (col + 8 <= g.n_out) {
        u32x4 o;
#pragma unroll
        for (int v = 0; v < 4; ++v) {
            if (g.res) {
                z[2 * v] += bf16_bits_to_f32(res[v] & 0xffffu);
                z[2 * v + 1] += bf16_bits_to_f32(res[v] >> 16);
            }
            o[v] = f32_to_bf16_bits(z[2 * v]) | (f32_to_bf16_bits(z[2 * v + 1]) << 16);
        }
        *reinterpret_cast<u32x4_any *>(d) = o;
    } else {
#pragma unroll
        for (int v = 0; v < 8; ++v)
            if (col + v < g.n_out) {
                if (g.res) z[v] += bf16_bits_to_f32(g.res[m * g.ld_res + col + v]);
                d[v] = (uint16_t)f32_to_bf16_bits(z[v]);
            }
    }
}

// GLU: 0 no SwiGLU; 1 SwiGLU; 2 SwiGLU whose up rows in a wave may straddle
// two blocks of 128 weight rows (N / 2 no multiple of 32).
// SPLIT: the K-blocks of a tile may be cut over several items.
template <int TP, int TQ, int WP, int WQ, int S, int GLU, bool SPLIT>
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
    const int nrt = (int)((g.M + TQ - 1) / TQ);
    const int n_items = nrt * nct * (SPLIT ? g.nsplit : 1);
    const int xcd = blockIdx.x & 7, step = gridDim.x >> 3;
    const int end = (int)((int64_t)(xcd + 1) * n_items / 8);
    int lit = (int)((int64_t)xcd * n_items / 8) + (blockIdx.x >> 3), cit = lit;
    if (cit >= end) return;
    const int nsp = SPLIT ? g.nsplit : 1;
    const int per = (nkb + nsp - 1) / nsp;                // K-blocks per split (none empty)

    // ---- load side.  A 16-byte copy instruction of a wave fills 8 rows of a
    // tile (8 lanes a row): its first row is uniform, so an address is a
    // scalar base, stepped from copy to copy, and one lane offset, which all
    // copies share; only tiles that reach past the last row clamp row by row.
    const uint8_t *pbase = nullptr, *qbase = nullptr;     // the wave's first copy, K-block lkb
    const float *xbase = nullptr;
    uint32_t xoff = 0;                                    // of x's or the weights' scales
    int lkb = 0, lkend = 0, pleft = 0, qleft = 0;         // pleft, qleft: the tile's rows that exist
    const int lrow = l >> 3;
    const uint32_t poff = (uint32_t)lrow * (uint32_t)g.K + (uint32_t)((l & 7) ^ ((lrow & 3) | ((w & 1) << 2))) * 16u;
    const uint32_t qoff = (uint32_t)lrow * (uint32_t)g.K + (uint32_t)((l & 7) ^ lrow) * 16u;
    // LDS row 8 (j NW + w) of the weights' tile: its column within the tile
    // and whether it is an up row; scalar steps from copy to copy
    auto pcol = [&](int j) {
        const int rho = 8 * (j * NW + w);
        return SW ? (rho >> 6) * 32 + (rho & 31) : rho;
    };
    const int64_t up = SW ? (int64_t)g.n_out * g.K : 0;
    static_assert(NW == 8 || NW == 4, "the steps below");
    const int64_t pstep0 = !SW ? (int64_t)(8 * NW) * g.K : NW == 8 ? (int64_t)32 * g.K : up;
    const int64_t pstep1 = SW && NW == 4 ? (int64_t)32 * g.K - up : pstep0;
    const int64_t qstep = (int64_t)(8 * NW) * g.K;
    auto load_setup = [&]() {
        int i = lit;
        const int sp = i % nsp;
        i /= nsp;
        int rt, ct;
        panel_tile<8>(i, nrt, nct, rt, ct);
        const int64_t m0 = (int64_t)rt * TQ;
        lkb = sp * per;
        lkend = min(lkb + per, nkb);
        const int c0 = ct * TC;
        pbase = g.w + (int64_t)(c0 + pcol(0)) * g.K + (NW == 8 && w >= 4 ? up : 0) + (int64_t)lkb * 128;
        pleft = min(TC, g.n_out - c0);
        qbase = g.xq + (m0 + 8 * w) * g.K + (int64_t)lkb * 128;
        qleft = (int)min((int64_t)TQ, g.M - m0);
        if (w < T::XW) {
            xbase = g.xs + m0 * nkb + lkb;
            xoff = (uint32_t)min(w * 64 + l, qleft - 1) * (uint32_t)nkb;
        } else {
            // the weights' scales, from the tile's first block on; with SwiGLU
            // lanes 32.. take the up rows' blocks
            const int first = (SW && l >= 32 ? c0 + g.n_out : c0) >> 7;
            const int last = ((SW ? 2 * g.n_out : g.n_out) - 1) >> 7;
            xbase = g.ws + lkb;
            xoff = (uint32_t)min(first + (SW ? l & 31 : l), last) * (uint32_t)nkb;
        }
    };
    // Copy c of a stage (JP of the weights, JQ of x, one of scales) into slot.
    // Rows past the last read the last one: the copy's first row r moves back
    // to it (uniform), then each lane by what its own row exceeds it, at most
    // lrow (24-bit products: below 2^8 times K <= 2^20), so that the lane
    // offset never goes below zero.
    constexpr int kCopies = JP + JQ + 1;
    auto copy8 = [&](const uint8_t *base, int r, int last, uint32_t off, uint8_t *dst) {
        const int back = max(r - last, 0);
        const int over = max(r - back + lrow - last, 0);
        lds_dma16(base - (int64_t)(back * g.K) + (off - __umul24(over, g.K)), dst);
    };
    auto issue_copy = [&](int c, int slot) {
        uint8_t *sp = smem + slot * T::Stage;
        if (c < JP) {
            const int64_t st = (int64_t)((c + 1) / 2) * pstep0 + (int64_t)(c / 2) * pstep1;
            copy8(pbase + st, pcol(c), pleft - 1, poff, sp + (c * NW + w) * 1024);
        } else if (c < JP + JQ) {
            const int j = c - JP;
            copy8(qbase + j * qstep, 8 * (j * NW + w), qleft - 1, qoff, sp + T::PB + (j * NW + w) * 1024);
        } else if (w < T::XW) {
            lds_dma4(xbase + xoff, sp + T::PB + T::QB + w * 256);
        } else if (w == NW - 1) {
            lds_dma4(xbase + xoff, sp + T::PB + T::QB + T::XB);
        }
    };
    auto stage_issued = [&]() {
        pbase += 128;
        qbase += 128;
        xbase += 1;
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
    // weight scales: one block of 128 rows per 64-row wave slice (gate and up
    // apart: b0, b1, counted from the tile's first); where its up rows
    // straddle two, rows from `cut` on take the second
    struct Item {
        int c0, kb, kend, b0, b1, cut;
        int64_t m0;
    };
    auto item_of = [&](int i) {
        Item it;
        const int csp = i % nsp;
        i /= nsp;
        int rt, ct;
        panel_tile<8>(i, nrt, nct, rt, ct);
        it.c0 = ct * TC;
        it.m0 = (int64_t)rt * TQ;
        it.kb = csp * per;
        it.kend = min(it.kb + per, nkb);
        static_assert(TP / WP == 64, "a wave's columns lie in one block of 128");
        const int c = it.c0 + wp * (SW ? 32 : 64);
        it.b0 = (c >> 7) - (it.c0 >> 7);
        it.b1 = it.cut = 0;
        if (SW) {
            const int b = (c + g.n_out) >> 7;
            it.b1 = 32 + b - ((it.c0 + g.n_out) >> 7);
            it.cut = ((b + 1) << 7) - (c + g.n_out);      // of the wave's 32 up rows
        }
        return it;
    };
    // Operands of a step in registers: all of the weights' (a), x's in a ring
    // of three (b), read from LDS two row tiles ahead of the MFMAs; a row
    // tile's products (t) are scaled and added while the next one's are formed.
    v8i a[NP], b[3];
    float x[3], s0 = 0.f, s1 = 0.f, s2 = 0.f;
    v4f t[2][NP];
    auto read_b = [&](int slot, int n) {
        const uint8_t *sq = smem + slot * T::Stage + T::PB;
        b[n % 3] = join8(lds_read16(sq + q_off + n * 2048), lds_read16(sq + (q_off ^ 64) + n * 2048));
        x[n % 3] = reinterpret_cast<const float *>(sq + T::QB)[wq * (TQ / WQ) + n * 16 + i16];
    };
    auto read_head = [&](int slot, const Item &it) {
        const uint8_t *sp = smem + slot * T::Stage;
        const float *sw = reinterpret_cast<const float *>(sp + T::PB + T::QB + T::XB);
#pragma unroll
        for (int m = 0; m < NP; ++m) {
            const int o = (m >> 1) * 32 * 128 + (m & 1) * 4 * 128;
            a[m] = join8(lds_read16(sp + p_off + o), lds_read16(sp + (p_off ^ 64) + o));
        }
        read_b(slot, 0);
        read_b(slot, 1);
        s0 = sw[it.b0];
        if (SW) s1 = sw[it.b1];
        if (GLU == 2) s2 = sw[it.b1 + 1];
    };
    auto add = [&](int n, float xn, float f0, float f1, float f2, int cut) {
#pragma unroll
        for (int m = 0; m < NP; ++m) {
            if (GLU == 2 && m >= 2) {
                const int r = 8 * grp + 4 * (m & 1);      // the lane's first up row of four
#pragma unroll
                for (int v = 0; v < 4; ++v) acc[m][n][v] += t[n & 1][m][v] * (xn * (r + v < cut ? f1 : f2));
            } else {
                const float f = xn * (SW && m >= 2 ? f1 : f0);
#pragma unroll
                for (int v = 0; v < 4; ++v) acc[m][n][v] += t[n & 1][m][v] * f;
            }
            // keeps the additions here: the compiler would gather them behind
            // the last MFMA and spill the products until then
            asm volatile("" : "+v"(acc[m][n]));
        }
    };
    auto epilogue = [&](const Item &it) {
        if (SPLIT && g.nsplit > 1) {             // FP32 sums, 1 KB per wave and MFMA tile
            float *d = g.part + ((int64_t)cit * NW + w) * (NP * NQ * 256) + l * 4;
#pragma unroll
            for (int m = 0; m < NP; ++m)
#pragma unroll
                for (int n = 0; n < NQ; ++n) *reinterpret_cast<v4f *>(d + (m * NQ + n) * 256) = acc[m][n];
            return;
        }
        // The residual's reads of NB row tiles go out together: one wait for
        // memory per NB tiles instead of one per tile.
        constexpr int NB = NQ < 4 ? NQ : 4;
#pragma unroll
        for (int p = 0; p < (SW ? 1 : NP / 2); ++p) {
            const int c = it.c0 + wp * (SW ? 32 : 64) + 8 * grp + 32 * p;
            if (c >= g.n_out) continue;
            float bz[8], bu[8];
            load_bias8(g.bias, c, g.n_out, bz);
            if (SW) load_bias8(g.bias ? g.bias + g.n_out : nullptr, c, g.n_out, bu);
#pragma unroll
            for (int n0 = 0; n0 < NQ; n0 += NB) {
                u32x4 r[NB];
#pragma unroll
                for (int n = 0; n < NB; ++n) {
                    r[n] = u32x4{0u, 0u, 0u, 0u};
                    const int64_t m = it.m0 + wq * (TQ / WQ) + 16 * (n0 + n) + i16;
                    if (g.res && c + 8 <= g.n_out && m < g.M)
                        r[n] = *reinterpret_cast<const u32x4_any *>(g.res + m * g.ld_res + c);
                }
#pragma unroll
                for (int n = 0; n < NB; ++n) {
                    const int64_t m = it.m0 + wq * (TQ / WQ) + 16 * (n0 + n) + i16;
                    if (m >= g.M) continue;
                    float z[8];
#pragma unroll
                    for (int v = 0; v < 8; ++v) z[v] = acc[2 * p + (v >> 2)][n0 + n][v & 3] + bz[v];
                    if (SW) {
#pragma unroll
                        for (int v = 0; v < 8; ++v) z[v] = silu(z[v]) * (acc[2 + (v >> 2)][n0 + n][v & 3] + bu[v]);
                    } else {
                        act8(z, g.act);
                    }
                    store8(g, m, c, z, r[n]);
                }
            }
        }
    };

    load_setup();
    Item cur = item_of(cit);
    int ckb = cur.kb;
    clear();
    int issued = 0, done = 0, islot = 0, slot = 0;        // stages issued and multiplied, their slots
    // The stage's copies have landed for this wave, then for all; every read
    // of the slot that the next copies overwrite is complete.
    auto next_stage = [&]() {
        constexpr int ahead = (S - 2) * (JP + JQ);
        if (S > 2 && issued - done == S - 1) wait_vmcnt<(ahead < 63 ? ahead : 63)>();
        else wait_vmcnt<0>();
        __builtin_amdgcn_s_waitcnt(0xC07F);               // lgkmcnt(0)
        stage_barrier();
    };
    for (int s = 0; s < S - 1 && lit < end; ++s) {
#pragma unroll
        for (int c = 0; c < kCopies; ++c) issue_copy(c, islot);
        stage_issued();
        ++issued;
        islot = islot + 1 == S ? 0 : islot + 1;
    }
    next_stage();
    while (true) {
        // The products of this step, and beside them the copies of the stage
        // S - 1 steps ahead, a few per row tile: copies all issued at once
        // would hold every wave up before its first MFMA.
        read_head(slot, cur);
        const bool load = lit < end;
        constexpr int kPer = (2 * kCopies + NQ - 1) / NQ;
        float xp = 0.f;
#pragma unroll
        for (int n = 0; n < NQ; ++n) {
            if (n + 2 < NQ) read_b(slot, n + 2);
            if (load) {
#pragma unroll
                for (int c = n * kPer; c < (n + 1) * kPer && c < kCopies; ++c) issue_copy(c, islot);
            }
#pragma unroll
            for (int m = 0; m < NP; ++m) t[n & 1][m] = mfma16x16x128(a[m], b[n % 3]);
            if (n > 0) add(n - 1, xp, s0, s1, s2, cur.cut);
            xp = x[n % 3];
            // reads ahead, then each MFMA beside a quarter of the previous row
            // tile's additions
            __builtin_amdgcn_sched_group_barrier(0x100, 3, 0);
#pragma unroll
            for (int m = 0; m < NP; ++m) {
                __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
                __builtin_amdgcn_sched_group_barrier(0x002, 5, 0);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
        add(NQ - 1, xp, s0, s1, s2, cur.cut);
        if (load) {
            stage_issued();
            ++issued;
            islot = islot + 1 == S ? 0 : islot + 1;
        }
        ++done;
        slot = slot + 1 == S ? 0 : slot + 1;
        if (issued > done) next_stage();
        if (++ckb == cur.kend) {
            epilogue(cur);
            cit += step;
            if (cit >= end) break;
            clear();
            cur = item_of(cit);
            ckb = cur.kb;
        }
    }
}

// Adds the splits' sums in order, then the epilogue: a thread takes the 8
// columns of one row that a lane of the tile kernel held.
template <int TP, int TQ, int WP, int WQ, int GLU>
__global__ void __launch_bounds__(256)
linear_join_kernel(LinearArgs g) {
    constexpr int NW = WP * WQ, NP = TP / WP / 16, NQ = TQ / WQ / 16, TC = GLU ? TP / 2 : TP;
    constexpr int NG = GLU ? 1 : NP / 2;                  // column groups of a wave
    const int l = threadIdx.x & 63;
    int i = (int)(((int64_t)blockIdx.x * 256 + threadIdx.x) >> 6);
    const int n = i % NQ;
    i /= NQ;
    const int p = i % NG;
    i /= NG;
    const int w = i % NW, tile = i / NW;
    const int nct = (g.n_out + TC - 1) / TC;
    const int wp = w % WP, wq = w / WP;
    int rt, ct;
    panel_tile<8>(tile, (int)((g.M + TQ - 1) / TQ), nct, rt, ct);
    const int64_t m = (int64_t)rt * TQ + wq * (TQ / WQ) + 16 * n + (l & 15);
    const int c = ct * TC + wp * (GLU ? 32 : 64) + 32 * p + 8 * (l >> 4);
    if (m >= g.M || c >= g.n_out) return;
    v4f z[2], u[2];
    for (int h = 0; h < 2; ++h) z[h] = u[h] = v4f{0.f, 0.f, 0.f, 0.f};
    for (int s = 0; s < g.nsplit; ++s) {
        const float *d = g.part + (((int64_t)tile * g.nsplit + s) * NW + w) * (NP * NQ * 256) + l * 4;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            z[h] += *reinterpret_cast<const v4f *>(d + ((2 * p + h) * NQ + n) * 256);
            if (GLU) u[h] += *reinterpret_cast<const v4f *>(d + ((2 + h) * NQ + n) * 256);
        }
    }
    float o[8], bz[8], bu[8];
    u32x4 r = {0u, 0u, 0u, 0u};
    load_bias8(g.bias, c, g.n_out, bz);
    if (GLU) load_bias8(g.bias ? g.bias + g.n_out : nullptr, c, g.n_out, bu);
    if (g.res && c + 8 <= g.n_out) r = *reinterpret_cast<const u32x4_any *>(g.res + m * g.ld_res + c);
#pragma unroll
    for (int v = 0; v < 8; ++v) {
        o[v] = z[v >> 2][v & 3] + bz[v];
        if (GLU) o[v] = silu(o[v]) * (u[v >> 2][v & 3] + bu[v]);
    }
    if (!GLU) act8(o, g.act);
    store8(g, m, c, o, r);
}

// ----------------------------------------------------------------- launch

template <int TP, int TQ, int WP, int WQ, int S, int GLU, bool SPLIT>
hipError_t launch_tile(const LinearArgs &g, hipStream_t st) {
    using T = LTile<TP, TQ, WP, WQ, S>;
    static std::atomic<uint64_t> done{0};
    auto fn = linear_tile_kernel<TP, TQ, WP, WQ, S, GLU, SPLIT>;
    hipError_t e = raise_lds_limit(done, (const void *)fn, (int)T::Smem);
    if (e != hipSuccess) return e;
    const int tc = GLU ? TP / 2 : TP;
    const int64_t items = ((g.M + TQ - 1) / TQ) * ((g.n_out + tc - 1) / tc) * g.nsplit;
    int64_t grid = (int64_t)device_cu_count() * (2 * T::Smem <= 160 * 1024 ? 2 : 1);
    if (grid > items) grid = items;
    grid = (grid + 7) / 8 * 8;
    fn<<<(unsigned)grid, 64 * WP * WQ, T::Smem, st>>>(g);
    e = hipGetLastError();
    if constexpr (SPLIT)
        if (e == hipSuccess && g.nsplit > 1) {
            const int64_t waves = items / g.nsplit * (WP * WQ) * (GLU ? 1 : T::NP / 2) * T::NQ;
            linear_join_kernel<TP, TQ, WP, WQ, GLU><<<(unsigned)((waves + 3) / 4), 256, 0, st>>>(g);
            e = hipGetLastError();
        }
    return e;
}

template <int NQ, int NW, int U, bool SW, bool XL>
hipError_t launch_stream(const LinearArgs &g, hipStream_t st) {
    const dim3 grid((g.n_out + (SW ? 7 : 15)) / (SW ? 8 : 16), (unsigned)((g.M + 16 * NQ - 1) / (16 * NQ)));
    constexpr int smem = stream_lds(NQ, NW, U, XL);
    static_assert(smem <= 160 * 1024, "LDS");
    static std::atomic<uint64_t> done{0};
    auto fn = linear_stream_kernel<NQ, NW, U, SW, XL>;
    hipError_t e = raise_lds_limit(done, (const void *)fn, smem);
    if (e != hipSuccess) return e;
    fn<<<grid, 64 * NW, smem, st>>>(g);
    return hipGetLastError();
}

template <int GLU>
hipError_t launch(const LinearArgs &g, hipStream_t st) {
    constexpr bool SW = GLU != 0;
    switch (g.form) {
        case kLinStream: {
            if (g.stream_nq == 4) return launch_stream<4, 8, 1, SW, true>(g, st);
            if (g.stream_nq == 3) return launch_stream<3, 8, 1, SW, true>(g, st);
            if (g.stream_nq == 2) return launch_stream<2, 8, 1, SW, true>(g, st);
            if (g.M > 4) return launch_stream<1, 8, 2, SW, true>(g, st);
            return launch_stream<1, 8, 2, SW, false>(g, st);
        }
        case kLinTile256:
            if constexpr (GLU < 2) return launch_tile<256, 256, 4, 2, 2, GLU, false>(g, st);
            [[fallthrough]];
        case kLinTile128: return launch_tile<256, 128, 4, 2, 3, GLU, false>(g, st);
        default: return launch_tile<128, 64, 2, 2, 3, GLU, true>(g, st);
    }
}

}  // namespace

size_t linear_workspace(LinearArgs &a, void *ws) {
    const int n = a.act == kActSwiglu ? 2 * a.n_out : a.n_out;     // weight rows
    const int nkb = a.K / 128;
    auto items = [&](int tp, int tq) { return ((a.M + tq - 1) / tq) * ((n + tp - 1) / tp); };
    a.nsplit = 1;
    a.part = nullptr;
    // Tile form by estimated time: rounds of tiles over the CUs, each nkb
    // steps and a fill and store of the tile.  Per step and per tile, measured
    // with every CU busy: 256 x 256 2.0 and 10 us, 256 x 128 1.1 and 6 us,
    // 128 x 64, alone on its CU, 0.8 and 3 us.  (The larger tile does the most per step, the
    // smaller ones lose less to a last, partly filled round.)
    const int64_t cus = 256;
    // Few rows by estimated time: a workgroup of 16 NQ rows takes (0.075 +
    // 0.055 NQ) us per K-block; small NQ fills the CUs, large NQ reads the
    // weights less often.  Against the tiles, which also pay some 3 us more
    // for their ring's first stages.  Measured (us, few rows / tiles): K = N =
    // 1024, 64 / 256 / 1000 rows 3.2 / 9.8, 4.6 / 10.0, 10.8 / 10.2; K = 4096,
    // N = 2048, 64 / 128 / 192 rows 6.8 / 11.6, 10.1 / 13.8, 17.3 / 14.7; K =
    // 4096, N = 8192, 16 / 33 / 64 rows 10.3 / 14.0, 14.5 / 14.6, 19.8 / 14.8.
    double t_few = 1e300;
    for (int nq = 1; nq <= 4 && a.M <= 1024; ++nq) {
        const int64_t wgs = ((n + 15) / 16) * ((a.M + 16 * nq - 1) / (16 * nq));
        const double t = 2.5 + (wgs > cus ? wgs / 256.0 : 1.0) * nkb * (0.075 + 0.055 * nq);
        if (t < t_few) {
            t_few = t;
            a.stream_nq = nq;
        }
    }
    auto est = [&](int64_t it, int steps, double step, double tile) {
        return (double)((it + cus - 1) / cus) * (steps * step + tile);
    };
    const double t256 = est(items(256, 256), nkb, 2.0, 10.0), t128 = est(items(256, 128), nkb, 1.1, 6.0);
    // The small tile has a ring of three stages, so that two fit a CU and hide
    // each other's waits: 0.97 us a step and 3.5 a tile for both (K = 4096, N =
    // 1024, 4000 rows 46 us with six stages and one tile a CU, 36 so).  It may
    // split K over idle CUs (at least 4 steps each); joining the parts costs
    // about 4 us and their way through memory.  Measured, K = 4096, N = 1024
    // (us, parts): 512 rows 15.6 (4), 18.1 (8); 700 rows 18.8 (2), 16.5 (5);
    // 1500 rows 26.9 (1), 23.8 (2).
    const int64_t it64 = items(128, 64);
    auto est64 = [&](int64_t it, int steps) {
        return it <= cus ? steps * 0.8 + 3.0 : (double)((it + 2 * cus - 1) / (2 * cus)) * (steps * 0.97 + 3.5);
    };
    double t64 = est64(it64, nkb);
    for (int64_t fit = cus; fit <= 2 * cus; fit += cus) {
        int64_t sp = std::min(fit / it64, (int64_t)nkb / 4);
        if (sp < 2) continue;
        const int per = (int)((nkb + sp - 1) / sp);
        sp = (nkb + per - 1) / per;                                // none empty
        const double t = est64(it64 * sp, per) + 4.0 + (double)sp * a.M * n * 1.1e-6;
        if (t < t64) {
            t64 = t;
            a.nsplit = (int)sp;
        }
    }
    // SwiGLU with straddling blocks has no 256 x 256 form (registers)
    const bool no256 = a.act == kActSwiglu && a.n_out % 32 != 0;
    a.form = kLinTile64;
    if (t128 < t64) a.form = kLinTile128;
    if (!no256 && t256 < (t128 < t64 ? t128 : t64)) a.form = kLinTile256;
    const double t_tile = a.form == kLinTile64 ? t64 : a.form == kLinTile128 ? t128 : t256;
    if (t_few < t_tile + 3) a.form = kLinStream;
    if (a.form != kLinTile64) a.nsplit = 1;
    if (a.nsplit == 1) return 0;
    a.part = (float *)ws;
    return (size_t)a.nsplit * items(128, 64) * (128 * 64 * 4);
}

hipError_t launch_linear(const LinearArgs &a, hipStream_t st) {
    if (a.act != kActSwiglu) return launch<0>(a, st);
    return a.n_out % 32 == 0 ? launch<1>(a, st) : launch<2>(a, st);
}

}  // namespace moe
