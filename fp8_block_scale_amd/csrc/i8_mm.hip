// Products of 8-bit integers with one scale per row of x and per weight row,
// with their epilogue, dense or grouped by expert over a routing plan:
//   z[r, n]   = x_s[t(r)] w_s[e(r), n] sum_k x_q[t(r), k] w[e(r), n, k] + bias[e(r), n]
//   out[r, n] = act(z)[r, n] + residual[r, n]
// With SwiGLU act(z)[r, j] = silu(z[r, j]) z[r, I + j].
//
// The sums are 32-bit integers, exact for K < 2^17 (2^17 products of at most
// 2^14); scales, bias, activation and residual are FP32, rounded once.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "i8_index.h"
#include "i8_mm.h"
#include "tiles.h"

namespace moe {

namespace {

typedef int v4i __attribute__((ext_vector_type(4)));

__device__ __forceinline__ v4i mfma64(const u32x4 &a, const u32x4 &b, const v4i &c) {
    return __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(v4i, a), __builtin_bit_cast(v4i, b), c, 0, 0, 0);
}

__device__ __attribute__((aligned(16))) const uint32_t kZeros[4] = {0u, 0u, 0u, 0u};

// ----------------------------------------------------------------- few rows

// 16 weight rows (with SwiGLU 8 gate and their 8 up rows) x 16 NQ rows of x a
// workgroup; grouped, a plan block's rows, 16 NQ at a time.  Wave w takes the
// steps of 128 values of K w, w + NW, ...; U of them are loaded, straight into
// registers, before the first is multiplied, and the waves' sums are added in
// LDS.  Rows of x go through the wave's share of LDS, 8 whole rows of 128 bytes a
// copy: register loads touch 16 rows, 64 bytes of each.
// Rows past the end read another row: their results are not stored.  Values past
// the end of K are zeros on one side at least.
// Bound by the weights from HBM where they are many (4 tokens of 9 routes, 257
// experts, K = 7168, N = 512: 125 MB in 29 us, 4.3 TB/s), by its latency else (48
// rows, K = 4096, N = 2048, SwiGLU: 5.5 us, 8.4 MB).
template <int NQ, int NW, int U, bool F16, bool SW, bool GROUPED>
__global__ void __launch_bounds__(64 * NW)
i8_stream_kernel(I8Args a) {
    // a wave's share of LDS: its rows of x, then its sums [16 NQ][17]
    constexpr int kSums = (NQ * 16 * 17 * 4 + 15) / 16 * 16, kRows = U * NQ * 2048;
    constexpr int kWave = kRows > kSums ? kRows : kSums;
    __shared__ __attribute__((aligned(16))) uint8_t smem[NW * kWave];
    const int tid = threadIdx.x, l = tid & 63, w = uni(tid >> 6), i16 = l & 15, grp = l >> 4;
    uint8_t *const lds = smem + w * kWave;
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
    const int8_t *ap = a.w + ((int64_t)e * a.N + wrow(i16)) * a.K;
    const u32x4 zero = {0u, 0u, 0u, 0u};
    // the output row of row i (-1: none) and its row of x
    auto out_row = [&](int i) -> int64_t {
        if (!GROUPED) return i < rows_end ? i : -1;
        const int r = i < rows_end ? a.g.sorted[i] : -1;
        return (uint32_t)r < (uint32_t)a.g.R ? r : -1;
    };
    auto x_row = [&](int64_t r) -> int64_t { return GROUPED && !a.g.per_route ? a.g.token_of((int)r) : r; };
    constexpr int NR = 2 * NQ;                   // the lane's rows of x
    const int x_off = i16 * 128 + ((grp ^ (i16 & 7)) << 4);
    for (; row0 < rows_end; row0 += 16 * NQ) {
        const int64_t r0 = out_row(row0);
        if (r0 < 0) break;                       // sentinels end the segment
        const int8_t *bp[NR];
#pragma unroll
        for (int n = 0; n < NR; ++n) {
            const int64_t r = out_row(row0 + 8 * n + (l >> 3));
            // (chunk c of row r lies at c ^ (r & 7) in LDS)
            bp[n] = a.xq + x_row(r < 0 ? r0 : r) * a.K + ((l & 7) ^ (l >> 3)) * 16;
        }
        v4i acc[NQ];
#pragma unroll
        for (int n = 0; n < NQ; ++n) acc[n] = v4i{0, 0, 0, 0};
        for (int k0 = w * kI8Step; k0 < a.K; k0 += NW * U * kI8Step) {
            u32x4 av[U][2], x[U][NQ][2];
            bool ok[U][2];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int k = k0 + u * NW * kI8Step;
                if (k >= a.K) break;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    ok[u][h] = i8_weights_count(k, h, grp, a.K);
                    av[u][h] = __builtin_nontemporal_load(
                        reinterpret_cast<const u32x4 *>(ap + i8_weights_load(k, h, grp, a.K)));
                }
                const bool in = k + ((l & 7) ^ (l >> 3)) * 16 < a.K;
#pragma unroll
                for (int n = 0; n < NR; ++n)
                    lds_dma16(in ? (const void *)(bp[n] + k) : (const void *)kZeros, lds + (u * NR + n) * 1024);
            }
            __builtin_amdgcn_sched_barrier(0);   // every load above is issued first
            asm volatile("s_waitcnt vmcnt(0)" ::: "memory");       // the wave's own copies
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (k0 + u * NW * kI8Step >= a.K) break;
#pragma unroll
                for (int n = 0; n < NQ; ++n) {
                    x[u][n][0] = lds_read16(lds + (u * NQ + n) * 2048 + x_off);
                    x[u][n][1] = lds_read16(lds + (u * NQ + n) * 2048 + (x_off ^ 64));
                }
            }
            // read before the next steps' copies write there
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (k0 + u * NW * kI8Step >= a.K) break;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const u32x4 v = ok[u][h] ? av[u][h] : zero;
#pragma unroll
                    for (int n = 0; n < NQ; ++n) acc[n] = mfma64(v, x[u][n][h], acc[n]);
                }
            }
        }
#pragma unroll
        for (int n = 0; n < NQ; ++n)
#pragma unroll
            for (int v = 0; v < 4; ++v) reinterpret_cast<int *>(lds)[(n * 16 + i16) * 17 + 4 * grp + v] = acc[n][v];
        __syncthreads();
        constexpr int COLS = SW ? 8 : 16;
        for (int i = tid; i < 16 * NQ * COLS; i += 64 * NW) {
            const int c = i % COLS, q = i / COLS, col = c0 + c;
            const int64_t r = out_row(row0 + q);
            if (r < 0 || col >= a.n_out) continue;
            const float xs = a.xs[x_row(r)];
            const float *ws = a.ws + (int64_t)e * a.N, *bias = a.bias ? a.bias + (int64_t)e * a.N : nullptr;
            const float sc = ws[col], scu = SW ? ws[col + a.n_out] : 0.f;
            const float b = bias ? bias[col] : 0.f, bu = SW && bias ? bias[col + a.n_out] : 0.f;
            int s = 0, u = 0;
#pragma unroll
            for (int k = 0; k < NW; ++k) {
                const int *d = reinterpret_cast<const int *>(smem + k * kWave) + q * 17 + c;
                s += d[0];
                if (SW) u += d[8];
            }
            float z = (float)s * xs * sc + b;
            z = SW ? silu(z) * ((float)u * xs * scu + bu) : act1(z, a.act);
            if (a.res) z += widen<F16>(a.res[r * a.ld_res + col]);
            a.out[r * a.ld_out + col] = (uint16_t)to16x2<F16>(z, 0.f);
        }
        __syncthreads();
        if (!GROUPED) break;
    }
}

// ---------------------------------------------------------------- many rows

// An item is a TQ x TP tile: TQ rows of x (B side of the MFMA) and TP weight
// rows (A side), so that a lane's results are 8 consecutive columns of one
// row: row i of MFMA tile 2 t + h is weight row 32 t + 8 (i / 4) + 4 h + i % 4.
// With SwiGLU the tile holds, per 64 rows, 32 gate rows and then their 32 up
// rows: both meet in one wave.
//
// A stage is 128 values of K of both operands, in rings of SP slots (weights) and
// SQ slots (rows of x) in LDS, filled by 16-byte global -> LDS copies, rows
// gathered by the plan on the way.  The MFMAs of one half of a stage (64 values
// of K) run beside the LDS reads of the next half, into the other register set.
// A slot is free once every wave has read its second half, in the middle of its
// own stage: the copies of the stages SQ and SP further on go out then, beside the
// second half's MFMAs.  Weights, which come from HBM, are given the more time
// where the LDS does not hold another slot of both.
//
// Four waves of 128 x 128 sums each (256 x 256): a stage's LDS reads take half the
// time of its MFMAs, with eight waves of 64 x 128 three quarters.  A stage takes
// 1.02 us on zeros and 1.36 on random values, where the card's power limits the
// matrix cores (56% busy at 2.03 GHz, 8192 x 4096 x 7168 in 200 us: 2.4 PFLOP/s; a
// library's 8-bit product reaches 2.1), the epilogue 9.5: some twenty vector
// instructions for each of 256 results a lane, and no other wave's MFMAs beside
// them.  Over a plan with few rows an expert weights from HBM are the bound (8192
// tokens of 8 routes, 288 experts, K = 4096, N = 2048: 640 us, 3.3 GB, 5.1 TB/s).
// Smaller tiles, down to 64 x 64, two workgroups to a CU, are for what gives the
// CUs too few large ones.
template <int TP, int TQ, int WP, int WQ, int SP, int SQ>
struct I8Tile {
    static constexpr int NW = WP * WQ;
    static constexpr int PB = TP * 128, QB = TQ * 128;
    static constexpr int JP = PB / 1024 / NW, JQ = QB / 1024 / NW, J = JP + JQ;
    static constexpr int NP = TP / WP / 16, NQ = TQ / WQ / 16;
    static constexpr size_t Smem = (size_t)SP * PB + (size_t)SQ * QB;
    static constexpr bool Ragged = TP * TQ < 256 * 256;      // output columns no multiple of 8
    static_assert(NP % 4 == 0 && NW == 4 && JP % 2 == 0 && JQ >= 1 && Smem <= 160 * 1024 && SP >= SQ && SQ >= 2, "tile");
};

// SiLU (g1 = -log2 e, g3 = 0) and GELU (g1 = -2 sqrt(2 / pi) log2 e, g3 = 0.044715 g1)
// in one form, z / (1 + 2^(g1 z + g3 z^3)): one copy of the epilogue's code.  (z^2
// is kept finite, so that it counts for nothing where g3 = 0.)
__device__ __forceinline__ float gated(float z, float g1, float g3) {
    const float e = z * fmaf(fminf(z * z, 3.402823466e38f), g3, g1);
    return z * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(e));
}

// f(0), f(1), ... f(N - 1) with constants
template <int N, typename F, int I = 0>
__device__ __forceinline__ void static_for(F &&f) {
    if constexpr (I < N) {
        f(std::integral_constant<int, I>());
        static_for<N, F, I + 1>(static_cast<F &&>(f));
    }
}

typedef u32x4 u32x4_any __attribute__((aligned(2)));
typedef v4f v4f_any __attribute__((aligned(4)));

// f[0, 8) = p[c, c + 8), 0 past n
__device__ __forceinline__ void load8(const float *p, int c, int n, float (&f)[8]) {
    if (c + 8 <= n) {
        const v4f lo = *reinterpret_cast<const v4f_any *>(p + c), hi = *reinterpret_cast<const v4f_any *>(p + c + 4);
#pragma unroll
        for (int v = 0; v < 4; ++v) {
            f[v] = lo[v];
            f[4 + v] = hi[v];
        }
    } else {
#pragma unroll
        for (int v = 0; v < 8; ++v) f[v] = c + v < n ? p[c + v] : 0.f;
    }
}

template <int TP, int TQ, int WP, int WQ, int SP, int SQ, bool F16, bool SW, bool GROUPED>
__global__ void __launch_bounds__(64 * WP * WQ, 1)
i8_tile_kernel(I8Args a) {
    using T = I8Tile<TP, TQ, WP, WQ, SP, SQ>;
    constexpr int NW = T::NW, JP = T::JP, JQ = T::JQ, NP = T::NP, NQ = T::NQ;
    constexpr int TC = SW ? TP / 2 : TP;                      // output columns of a tile
    extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
    const int tid = threadIdx.x, l = tid & 63, w = uni(tid >> 6);
    const int wp = w % WP, wq = w / WP, i16 = l & 15, grp = l >> 4;
    const int nct = (a.n_out + TC - 1) / TC;
    const int nrt = GROUPED ? min(uni(a.g.meta[0]), a.g.max_tiles) : (int)((a.M + TQ - 1) / TQ);
    const int n_items = nrt * nct;
    const int xcd = blockIdx.x & 7, step = gridDim.x >> 3;
    const int end = (int)((int64_t)(xcd + 1) * n_items / 8);
    const int lit = (int)((int64_t)xcd * n_items / 8) + (blockIdx.x >> 3);
    int cit = lit;
    if (cit >= end) return;
    const int nst = (a.K + 127) >> 7;                         // stages of an item

    struct Item {
        int e, c0, row0, rows;       // expert, first column, first row (of the plan), rows
    };
    auto item_of = [&](int i) {
        Item it;
        int rt, ct;
        panel_tile<8>(i, nrt, nct, rt, ct);
        it.c0 = ct * TC;
        if (GROUPED) {
            const int4 t = a.g.tiles[rt];
            it.row0 = uni(t.x);
            it.rows = uni(t.y);
            it.e = uni(t.z);
        } else {
            it.row0 = rt * TQ;
            it.rows = (int)min((int64_t)TQ, a.M - it.row0);
            it.e = 0;
        }
        return it;
    };
    // the output row of a tile's row, -1 if none
    auto out_row = [&](const Item &it, int row) {
        if (row >= it.rows) return -1;
        if (!GROUPED) return it.row0 + row;
        const int r = a.g.sorted[it.row0 + row];
        return (uint32_t)r < (uint32_t)a.g.R ? r : -1;
    };
    auto x_row = [&](int r) { return GROUPED && !a.g.per_route ? a.g.token_of(r) : r; };

    // ---- load side: a copy of a wave fills 8 rows of 128 bytes.  An address of
    // weights is a uniform base, stepped from stage to stage, and a lane offset
    // that holds the row (past the last: the last one); one of x the row's own.
    const int lrow = l >> 3;
    const int kc_p = (l & 7) ^ ((lrow & 3) | ((w & 1) << 2)), kc_q = (l & 7) ^ lrow;      // chunks of the rows
    const int8_t *pbase = nullptr;           // the tile's first weight row, the stage's values of K
    const int64_t up = SW ? (int64_t)a.n_out * a.K : 0;       // from a gate row to its up row
    uint32_t poff[JP];
    const int8_t *qptr[JQ];
    int pit = lit, qit = lit, pkt = 0, qkt = 0;               // items of the copies, their stages
    auto setup_p = [&]() {
        const Item it = item_of(pit);
        pkt = 0;
        pbase = a.w + ((int64_t)it.e * a.N + it.c0) * a.K;
        const int last = min(TC, a.n_out - it.c0) - 1;
#pragma unroll
        for (int j = 0; j < JP; ++j) {
            const int c = (SW ? (j >> 1) * 32 + 8 * w : 8 * (j * NW + w)) + lrow;
            poff[j] = (uint32_t)min(c, last) * (uint32_t)a.K + (uint32_t)kc_p * 16u;
        }
    };
    auto setup_q = [&]() {
        const Item it = item_of(qit);
        qkt = 0;
#pragma unroll
        for (int j = 0; j < JQ; ++j) {
            // a row that has no route reads row 0 of x, one past the last row
            // that: their results are not stored
            int r = out_row(it, 8 * (j * NW + w) + lrow);
            if (r < 0) r = GROUPED ? 0 : it.row0 + it.rows - 1;
            qptr[j] = a.xq + (int64_t)x_row(r) * a.K + kc_q * 16;
        }
    };
    // Copy j of the next stage of weights or rows of x to its slot.  `any`: the stage
    // may reach past the end of K or lie past the last item: zeros there.
    auto copy_p = [&](auto any, int j, uint8_t *slot) __attribute__((always_inline)) {
        const void *p = pbase + (SW && (j & 1) ? up : 0) + poff[j];
        if (decltype(any)::value && kc_p * 16 >= a.K - pkt * 128) p = kZeros;
        lds_dma16(p, slot + (j * NW + w) * 1024);
    };
    auto copy_q = [&](auto any, int j, uint8_t *slot) __attribute__((always_inline)) {
        const void *p = qptr[j];
        if (decltype(any)::value && kc_q * 16 >= a.K - qkt * 128) p = kZeros;
        lds_dma16(p, slot + (j * NW + w) * 1024);
    };
    auto next_p = [&]() {
        ++pkt;
        pbase += 128;
    };
    auto next_q = [&]() {
        ++qkt;
#pragma unroll
        for (int j = 0; j < JQ; ++j) qptr[j] += 128;
    };
    auto issued_p = [&]() {
        next_p();
        if (pkt == nst) {
            pit += step;
            if (pit < end) setup_p();
        }
    };
    auto issued_q = [&]() {
        next_q();
        if (qkt == nst) {
            qit += step;
            if (qit < end) setup_q();
        }
    };

    // ---- compute side
    v4i acc[NP][NQ];
    auto clear = [&]() {
#pragma unroll
        for (int m = 0; m < NP; ++m)
#pragma unroll
            for (int n = 0; n < NQ; ++n) acc[m][n] = v4i{0, 0, 0, 0};
    };
    // (emits nothing: tells the compiler that the sums stay in accumulation
    // registers, which it would copy to vector registers and back every stage)
    auto keep = [&]() {
#pragma unroll
        for (int m = 0; m < NP; ++m)
#pragma unroll
            for (int n = 0; n < NQ; ++n) asm volatile("" : "+a"(acc[m][n]));
    };
    const int pf = (i16 & 3) | (((i16 >> 2) & 1) << 2);
    const int p_off = (wp * (TP / WP) + 8 * (i16 >> 2) + (i16 & 3)) * 128 + ((grp ^ pf) << 4);
    const int q_off = (wq * (TQ / WQ) + i16) * 128 + ((grp ^ (i16 & 7)) << 4);
    u32x4 pa[2][NP], qb[2][NQ];
    auto read_op = [&](const uint8_t *ps, const uint8_t *qs, int h, int i) {      // operand i of half h: weights, then x
        if (i < NP) pa[h][i] = lds_read16(ps + (p_off ^ (h << 6)) + (i >> 1) * 32 * 128 + (i & 1) * 4 * 128);
        else qb[h][i - NP] = lds_read16(qs + (q_off ^ (h << 6)) + (i - NP) * 16 * 128);
    };
    // The products of a stage in two halves of K, beside them the reads of the
    // next half (the second half's from ps and qs, then the next stage's first from
    // pn and qn) and in the second half the copies, into the same ps and qs:
    // `arrive` lies between.  Rows of x go first: they have less time.
    auto multiply = [&](auto any, uint8_t *ps, uint8_t *qs, const uint8_t *pn, const uint8_t *qn, auto arrive)
                        __attribute__((always_inline)) {
        constexpr int kReads = NP + NQ, kPer = (4 * kReads + 3 * NQ - 1) / (3 * NQ);      // in three quarters of the units
        constexpr int kCopy = (T::J + NQ - 1) / NQ;
        __builtin_amdgcn_s_waitcnt(0xC07F);                   // lgkmcnt(0): the first half's operands
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            if (h == 1) arrive();
#pragma unroll
            for (int n = 0; n < NQ; ++n) {
#pragma unroll
                for (int i = n * kPer; i < (n + 1) * kPer && i < kReads; ++i)
                    read_op(h ? pn : ps, h ? qn : qs, h ^ 1, i);
                if (h == 1) {
#pragma unroll
                    for (int c = n * kCopy; c < (n + 1) * kCopy && c < T::J; ++c) {
                        if (c < JQ) copy_q(any, c, qs);
                        else copy_p(any, c - JQ, ps);
                    }
                }
#pragma unroll
                for (int m = 0; m < NP; ++m) acc[m][n] = mfma64(pa[h][m], qb[h][n], acc[m][n]);
                __builtin_amdgcn_sched_barrier(0);
            }
        }
    };
    // (emits no more than the wait for a load: one that some path leaves pending
    // would be waited for in the loop over the stages, together with all copies)
    auto arrived = [](float v) { asm volatile("" : : "v"(v)); };
    const float g1 = a.act == kActGelu ? -2.30220818f : -1.44269504f, g3 = a.act == kActGelu ? -0.10294324f : 0.f;
    // Everything is read before the first store, the residual in batches of NB
    // rows: loads and stores are counted together, so a wait for a load waits for
    // every store before it.  The code is unrolled (registers have no index) and
    // kept small: beyond the instruction cache it costs its misses on every tile
    // (with both output types and ragged ends 80 KB, 17 us a tile of 256 x 256).
    constexpr int NT = NP / (SW ? 4 : 2), NB = NQ == 1 ? 1 : NQ < 4 || NT > 2 ? 2 : 4;     // column groups of 32; rows of a batch
    auto epilogue = [&](const Item &it) __attribute__((always_inline)) {
        const float *ws = a.ws + (int64_t)it.e * a.N, *bias = a.bias ? a.bias + (int64_t)it.e * a.N : nullptr;
        const int c0 = it.c0 + wp * (TC / WP) + 8 * grp;      // the lane's columns: c0 + 32 t + [0, 8)
        int rr[NQ];
        float xs[NQ], s[NT][8], b[NT][8], su[SW ? NT : 1][8], bu[SW ? NT : 1][8];
#pragma unroll
        for (int n = 0; n < NQ; ++n) rr[n] = out_row(it, wq * (TQ / WQ) + 16 * n + i16);
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            load8(ws, c0 + 32 * t, a.n_out, s[t]);
            if (SW) load8(ws + a.n_out, c0 + 32 * t, a.n_out, su[t]);
#pragma unroll
            for (int v = 0; v < 8; ++v) {
                b[t][v] = 0.f;
                if (SW) bu[t][v] = 0.f;
            }
            if (bias) {
                load8(bias, c0 + 32 * t, a.n_out, b[t]);
                if (SW) load8(bias + a.n_out, c0 + 32 * t, a.n_out, bu[t]);
            }
        }
#pragma unroll
        for (int n = 0; n < NQ; ++n) xs[n] = rr[n] < 0 ? 0.f : a.xs[x_row(rr[n])];
#pragma unroll
        for (int n = 0; n < NQ; ++n) arrived(xs[n]);
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int v = 0; v < 8; ++v) {
                arrived(s[t][v]);
                arrived(b[t][v]);
                if (SW) arrived(su[t][v]);
                if (SW) arrived(bu[t][v]);
            }
        static_for<NQ / NB>([&](auto nc) __attribute__((always_inline)) {
            constexpr int n0 = decltype(nc)::value * NB;
            u32x4 q[NB][NT];
#pragma unroll
            for (int n = 0; n < NB; ++n)
#pragma unroll
                for (int t = 0; t < NT; ++t) q[n][t] = u32x4{0u, 0u, 0u, 0u};
            if (a.res) {
#pragma unroll
                for (int n = 0; n < NB; ++n) {
                    const uint16_t *res = a.res + (int64_t)rr[n0 + n] * a.ld_res + c0;
#pragma unroll
                    for (int t = 0; t < NT; ++t)
                        if (rr[n0 + n] >= 0 && c0 + 32 * t + 8 <= a.n_out)
                            q[n][t] = *reinterpret_cast<const u32x4_any *>(res + 32 * t);
                }
            }
#pragma unroll
            for (int n = 0; n < NB; ++n) {
                __builtin_amdgcn_sched_barrier(0);
                // (emits nothing: not moved to vector registers before)
#pragma unroll
                for (int m = 0; m < NP; ++m) asm volatile("" : "+a"(acc[m][n0 + n]));
                uint16_t *d = a.out + (int64_t)rr[n0 + n] * a.ld_out + c0;
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    const int c = c0 + 32 * t;
                    float z[8], r[8];
#pragma unroll
                    for (int v = 0; v < 8; ++v) {
                        const int m = (SW ? 4 : 2) * t + (v >> 2);
                        z[v] = (float)acc[m][n0 + n][v & 3] * xs[n0 + n] * s[t][v] + b[t][v];
                        if (SW) z[v] = silu(z[v]) * ((float)acc[m + (SW ? 2 : 0)][n0 + n][v & 3] * xs[n0 + n] *
                                                         su[SW ? t : 0][v] + bu[SW ? t : 0][v]);
                    }
                    if (!SW && a.act != kActNone) {
#pragma unroll
                        for (int v = 0; v < 8; ++v) z[v] = gated(z[v], g1, g3);
                    }
                    if (a.res) {
                        widen8<F16>(q[n][t], r);
#pragma unroll
                        for (int v = 0; v < 8; ++v) z[v] += r[v];
                    }
                    if (rr[n0 + n] < 0) continue;
                    if (c + 8 <= a.n_out) {
                        *reinterpret_cast<u32x4_any *>(d + 32 * t) = narrow8<F16>(z);
                    } else if (T::Ragged) {
                        const uint16_t *res = a.res ? a.res + (int64_t)rr[n0 + n] * a.ld_res + c : nullptr;
#pragma unroll
                        for (int v = 0; v < 8; ++v)
                            if (c + v < a.n_out)
                                d[32 * t + v] = (uint16_t)to16x2<F16>(res ? z[v] + widen<F16>(res[v]) : z[v], 0.f);
                    }
                }
            }
        });
    };

    // ---- the pipeline: SP stages of weights and SQ of rows of x are in flight or
    // being multiplied at any time (past the last they are copies of zeros: the
    // count of copies to wait for stays the same, and no branch comes between the
    // MFMAs).  In each stage the copies of x go out before those of weights, so
    // that those of weights alone may stay in flight beyond the next stage's.
    uint8_t *const pring = smem, *const qring = smem + SP * T::PB;
    setup_p();
    setup_q();
#pragma unroll 1
    for (int s = 0; s < SP; ++s) {
#pragma unroll
        for (int j = 0; j < JP; ++j) copy_p(std::true_type(), j, pring + s * T::PB);
        issued_p();
        if (s < SQ) {
#pragma unroll
            for (int j = 0; j < JQ; ++j) copy_q(std::true_type(), j, qring + s * T::QB);
            issued_q();
        }
    }
    // the next stage's copies have landed for this wave, then for all; every
    // wave has read the slots that the next copies overwrite
    auto arrive = [&](auto ahead) {          // `ahead` stages may stay in flight
        constexpr int n = decltype(ahead)::value * T::J + (SP - SQ) * JP;
        wait_vmcnt<(n < 63 ? n : 63)>();
        __builtin_amdgcn_s_waitcnt(0xC07F);                   // lgkmcnt(0)
        stage_barrier();
    };
    int pslot = 0, qslot = 0;                // of the stage that is being multiplied
    arrive(std::integral_constant<int, SQ - 1>());
#pragma unroll
    for (int i = 0; i < NP + NQ; ++i) read_op(pring, qring, 0, i);
    auto stage = [&](auto any) __attribute__((always_inline)) {
        uint8_t *const ps = pring + pslot * T::PB, *const qs = qring + qslot * T::QB;
        pslot = pslot + 1 == SP ? 0 : pslot + 1;
        qslot = qslot + 1 == SQ ? 0 : qslot + 1;
        multiply(any, ps, qs, pring + pslot * T::PB, qring + qslot * T::QB, [&]() __attribute__((always_inline)) {
            arrive(std::integral_constant<int, SQ - 2>());
        });
        keep();
    };
    const int nsame = max(0, nst - SP - 1);
    for (; cit < end; cit += step) {
        clear();
        keep();
        // stages beside which a whole stage of the same item is copied that is
        // not its last, then the rest
        for (int k = 0; k < nsame; ++k) {
            stage(std::false_type());
            next_p();
            next_q();
        }
        for (int k = nsame; k < nst; ++k) {
            stage(std::true_type());
            issued_q();
            issued_p();
        }
        epilogue(item_of(cit));
    }
    wait_vmcnt<0>();                         // no copy into LDS outlives the workgroup
}

template <int TP, int TQ, int WP, int WQ, int SP, int SQ, bool F16, bool SW, bool GROUPED>
hipError_t launch_tile(const I8Args &a, hipStream_t st) {
    using T = I8Tile<TP, TQ, WP, WQ, SP, SQ>;
    static std::atomic<uint64_t> done{0};
    auto fn = i8_tile_kernel<TP, TQ, WP, WQ, SP, SQ, F16, SW, GROUPED>;
    hipError_t e = raise_lds_limit(done, (const void *)fn, (int)T::Smem);
    if (e != hipSuccess) return e;
    constexpr int TC = SW ? TP / 2 : TP;
    const int64_t rows = GROUPED ? a.g.max_tiles : (a.M + TQ - 1) / TQ;
    const int64_t items = rows * ((a.n_out + TC - 1) / TC);
    int64_t grid = (int64_t)device_cu_count() * (2 * T::Smem <= 160 * 1024 ? 2 : 1);
    if (grid > items) grid = items;
    grid = (grid + 7) / 8 * 8;
    fn<<<(unsigned)grid, 64 * WP * WQ, T::Smem, st>>>(a);
    return hipGetLastError();
}

template <bool F16, bool SW, bool GROUPED>
hipError_t launch(const I8Args &a, hipStream_t st) {
    if (a.stream_nq) {
        const int64_t rows = GROUPED ? a.g.sorted_cap / a.g.block_m : (a.M + 16 * a.stream_nq - 1) / (16 * a.stream_nq);
        const dim3 grid((a.n_out + (SW ? 7 : 15)) / (SW ? 8 : 16), (unsigned)rows);
        switch (a.stream_nq) {
            case 1: i8_stream_kernel<1, 8, 2, F16, SW, GROUPED><<<grid, 512, 0, st>>>(a); break;
            case 2: i8_stream_kernel<2, 8, 2, F16, SW, GROUPED><<<grid, 512, 0, st>>>(a); break;
            case 3: i8_stream_kernel<3, 8, 1, F16, SW, GROUPED><<<grid, 512, 0, st>>>(a); break;
            default: i8_stream_kernel<4, 8, 1, F16, SW, GROUPED><<<grid, 512, 0, st>>>(a);
        }
        return hipGetLastError();
    }
    if (GROUPED) {
        hipError_t e = launch_group_prep(a.g, st);
        if (e != hipSuccess) return e;
    }
    if (a.tile_rows == 256) return launch_tile<256, 256, 2, 2, 3, 2, F16, SW, GROUPED>(a, st);
    if (a.tile_cols == 256) return launch_tile<256, 128, 2, 2, 3, 3, F16, SW, GROUPED>(a, st);
    if (a.tile_rows == 128) return launch_tile<128, 128, 2, 2, 3, 2, F16, SW, GROUPED>(a, st);
    if (a.tile_cols == 128) return launch_tile<128, 64, 2, 2, 3, 3, F16, SW, GROUPED>(a, st);
    return launch_tile<64, 64, 1, 4, 5, 5, F16, SW, GROUPED>(a, st);
}

template <bool F16>
hipError_t launch_type(const I8Args &a, hipStream_t st) {
    const bool sw = a.act == kActSwiglu;
    if (a.grouped) return sw ? launch<F16, true, true>(a, st) : launch<F16, false, true>(a, st);
    return sw ? launch<F16, true, false>(a, st) : launch<F16, false, false>(a, st);
}

}  // namespace

size_t i8_workspace(I8Args &a, void *ws) {
    // The form by estimated time (us), the smallest first.  All constants are
    // measured with weights from HBM where there are more than the caches hold.
    const double steps = (a.K + 127) / 128;
    const bool sw = a.act == kActSwiglu;
    const double R = (double)(a.grouped ? a.g.R : a.M), E = a.grouped ? a.g.E : 1;
    const double hit = E > 1 ? E * -std::expm1(R * std::log1p(-1.0 / E)) : 1;         // experts with a route
    const double rows = R / hit, wbytes = hit * (double)a.N * (double)a.K;
    auto parts = [&](int size) {                          // of at most `size` rows, of an expert
        return a.grouped ? group_parts(rows, size) : std::ceil(rows / size);
    };
    // Few rows: a workgroup takes about 0.10, 0.13, 0.16 or 0.18 us for a step and 16,
    // 32, 48 or 64 rows, 0.7 to 2.0 at least (a wave's loads, the sum over waves) and
    // over a plan 0.4 to 1.6 more (it reads which expert and rows are its own before
    // it begins); start and end of the launch take 3.3.
    // Measured (us, by rows of a pass): K = 4096, N = 2048, 16 / 64 / 256 rows 6.2, 6.5,
    // 7.2, 7.5 / 9.4, 7.4, 8.0, 9.8 / 29, 20, 19, 16; K = 1024, N = 8192, 64 rows 10.3,
    // 8.9, 9.4, 6.9; K = 352, N = 5830, 173 rows 14.7, 14.7, 11.5, 13.3; E = 14, K = 832,
    // N = 392, 364 rows an expert 53, 42, 37, 35.
    static const double few[4] = {0.10, 0.13, 0.16, 0.18}, least[4] = {0.7, 1.2, 1.5, 2.0},
                        begin[4] = {0.4, 0.8, 1.2, 1.6};
    auto whole = [](double rounds) { return rounds < 4 ? std::ceil(rounds) : rounds; };
    double best = 1e300;
    a.stream_nq = 0;
    const int64_t blocks = a.grouped ? a.g.sorted_cap / a.g.block_m : 0;
    for (int nq = 1; nq <= 4; ++nq) {
        if (a.grouped ? blocks > 65535 : a.M > 1024) break;
        const double wgs = hit * parts(a.grouped ? std::min(a.g.block_m, 16 * nq) : 16 * nq) *
                           ((a.n_out + (sw ? 7 : 15)) / (sw ? 8 : 16));
        const double each = std::max(steps * few[nq - 1], least[nq - 1]) + (a.grouped ? begin[nq - 1] : 0);
        const double t = 3.3 + std::max(whole(wgs / 256) * each, wbytes / 4.3e6);
        if (t < best) {
            best = t;
            a.stream_nq = nq;
        }
    }
    // Tiles: launch and first copies take about 3.5 us, over a plan the set-up launch
    // before 5 (in a graph 3.9 for 4 or 8 experts, 6.0 to 6.5 for 288, 8.0 for 512; an
    // empty launch 2.1); a step of 128 of K `idle` alone and `busy` with a tile on every CU, a
    // tile's end `ends`.  HBM gives 5.4 TB/s of the weights, which a row tile finds in
    // the caches in part where another one has read them; `mix` of the shorter of both
    // times adds to the longer.
    // Measured (us; rows x columns 64 x 64 / 64 x 128 / 128 x 128 / 128 x 256 / 256 x 256):
    //   K = 2048, N = 1000, 1000 rows    8.6,  9.8, 13.2, 18.3, 27.9
    //   K = 4096, N = 2048, 1000 rows   19.1, 15.0, 20.2, 27.4, 44.8
    //                       4096 rows   64.3, 52.3, 41.0, 37.7, 54.0
    //   K = 7168, N = 4096, 512 rows    33.4, 29.4, 36.4, 51.7, 71.7
    //                       2048 rows    107, 87.6, 61.2, 57.8, 85.0
    //                       4096 rows    204,  170,  119,  111, 95.3
    //   E = 288, K = 4096, N = 2048, SwiGLU, by rows an expert
    //                       14           457,  434,  448,  438,  564
    //                       57           596,  515,  480,  467,  574
    //                       114          887,  692,  585,  539,  592
    //                       228         1450, 1095,  848,  766,  668
    // (32 and 64 rows x 256 columns measured no faster anywhere.)
    struct Form {
        int rows, cols;
        double idle, busy, ends, mix;
    };
    static const Form forms[5] = {{64, 64, 0.21, 0.22, 0.9, 0.3},
                                  {64, 128, 0.28, 0.35, 1.4, 0.15},
                                  {128, 128, 0.42, 0.48, 2.2, 0.17},
                                  {128, 256, 0.60, 0.84, 6.3, 0.1},
                                  {256, 256, 1.04, 1.36, 9.5, 0.1}};
    a.tile_rows = 0;
    for (const Form &f : forms) {
        if (f.rows == 256 && a.n_out % 8 != 0) continue;      // (no code for ragged ends)
        const double per = parts(f.rows), items = hit * per * ((a.N + f.cols - 1) / f.cols);
        const double step = f.idle + (f.busy - f.idle) * std::min(items / 256, 1.0), rounds = items / 256;
        const double busy = (rounds < 4 ? std::ceil(rounds) : rounds + 0.5) * (steps * step + f.ends);
        const double mem = (1 + (per - 1) * (a.grouped ? 0.35 : 0.1)) * wbytes / 5.4e6;
        const double t = 3.5 + std::max(busy, mem) + f.mix * std::min(busy, mem) + (a.grouped ? 5 : 0);
        if (t < best) {
            best = t;
            a.tile_rows = f.rows;
            a.tile_cols = f.cols;
        }
    }
    if (a.tile_rows) a.stream_nq = 0;
    if (!a.grouped) return 0;
    group_divider(a.g);
    return a.stream_nq ? 0 : group_tiles_workspace(a.g, a.tile_rows, ws);
}

hipError_t launch_i8(const I8Args &a, hipStream_t st) { return a.f16 ? launch_type<true>(a, st) : launch_type<false>(a, st); }

}  // namespace moe
