// Matrix products grouped by expert, ragged, in BF16 or FP16 (FP32 sums):
//   forward   y[r, n]     = sum_k x[t(r), k] w[e(r), n, k]
//   dx        dx[t, k]    = sum_{r: t(r) = t} sum_n dy[r, n] w[e(r), n, k]
//   dw        dw[e, n, k] = sum_{r in e} dy[r, n] x[t(r), k]
// over the routes r that the plan lists for each expert e; t(r) = r / top_k
// (token rows) or r (one row per route).
//
// One kernel form serves all three.  A work item is a TQ x TP output tile:
// TP output columns (contiguous in memory: n, k, k) from operand P, the A
// side of the MFMA, and TQ output rows (routes, routes, n) from operand Q,
// the B side.  A stage holds 64 of the contraction for both operands, 128
// bytes per row, in LDS; it is filled by 16-byte global -> LDS copies, S - 1
// stages ahead of the MFMAs.  An operand whose memory runs along the
// contraction (x, dy in dx, w in forward) is staged as [row][64] and read by
// 16-byte LDS reads; one whose memory runs along the output (w in dx, x and
// dy in dw) as [64][columns] and read by the transposing LDS read
// (ds_read_b64_tr_b16), so no operand is ever re-laid out in memory and rows
// are gathered by the plan on the way in.
//
// The kernel is persistent: a workgroup walks its items, and the copies for
// the next item's first stages are in flight while the current item's last
// stages are multiplied and its tile is stored (weight gradients have only a
// few stages per tile).  Neighbouring items, which share rows or weights, run
// on one XCD at the same time (panel_tile).
//
// What bounds it, measured (counters on random values, and on zeros, where the
// clock is higher).  Experts of two hundred rows: neither side alone.  E =
// 288, K = 4096, N = 2048, 8192 tokens of 8 routes in BF16 take 1.44 ms, 766
// TFLOP/s of routes (the padding of each expert's last tile comes on top): the
// matrix cores are busy 46% of the time at 1.7 GHz, HBM moves 6.1 GB at 4.1
// TB/s and the waves wait 35% of their time for the two-stage ring; zeros, at
// 2.3 GHz, are 11% faster.  Experts of some tens of rows: the weights (E =
// 512, K = 2048, N = 1024, 40 routes an expert: 0.45 ms, 2.4 GB at 5.3 TB/s).
// dx summed over a token's routes: HBM too, with the FP32 rows' way through
// memory (4096 tokens at the first sizes: 1.25 ms, 440 TFLOP/s; the tile
// kernel moves 6.5 GB at 5.7 TB/s, zeros are 1% faster).  dw with a few stages
// per tile: the tile's store, some 3.5 us, that the next tile's products do
// not cover as they wait for it (36 experts of 227 rows: 0.25 ms for 0.6 GB
// out, matrix cores busy 25%).  Small calls: the set-up launch (4 us) and the
// latency of a tile's first copies.
#include <algorithm>
#include <cmath>

#include "group_mm.h"
#include "tiles.h"

namespace moe {

namespace {

typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef short v4s __attribute__((ext_vector_type(4)));

template <bool F16>
__device__ __forceinline__ v4f mfma32(const u32x4 &a, const u32x4 &b, const v4f &c) {
    if constexpr (F16)
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(v8h, a), __builtin_bit_cast(v8h, b), c,
                                                      0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, a),
                                                       __builtin_bit_cast(v8bf, b), c, 0, 0, 0);
}

// Two values at once (one packed conversion, round to nearest even).
template <bool F16>
__device__ __forceinline__ uint32_t to16x2(float lo, float hi) {
    typedef float v2f __attribute__((ext_vector_type(2)));
    typedef __bf16 v2bf __attribute__((ext_vector_type(2)));
    const v2f v = {lo, hi};
    if constexpr (F16) return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, v2h));
    else return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, v2bf));
}

template <bool F16>
__device__ __forceinline__ float from16(uint32_t v) {
    if constexpr (F16) return (float)__builtin_bit_cast(_Float16, (uint16_t)v);
    else return bf16_bits_to_f32(v & 0xffffu);
}

// What the copies of contraction values past the end read: zeros on both
// operands (0 * garbage could be NaN).
__device__ __attribute__((aligned(16))) const uint32_t kZeros[4] = {0u, 0u, 0u, 0u};

// ------------------------------------------------------------ set-up launch

// Workgroup 0 finds every expert's rows in the plan (its sentinels are all at
// the end of its last block) and cuts them into row tiles of tile_rows, listed
// as {first row, rows, expert, slot} with their count in meta[0].  For dw an
// expert without rows has one empty tile (none if dw is added to: it stays as
// it is), the tiles of an expert with several have slots one after the other
// (else -1), and those experts, meta[1] of them, are listed as joins =
// {expert, first slot, slots}.  The other workgroups set rpos[0, R) = -1 for
// the sum over a token's routes.
constexpr int kPrepThreads = 1024;

__global__ void __launch_bounds__(kPrepThreads)
group_prep_kernel(GroupMmArgs g, int tile_rows) {
    const int tid = threadIdx.x;
    if (blockIdx.x > 0) {
        const int64_t stride = (int64_t)(gridDim.x - 1) * kPrepThreads;
        for (int64_t i = (int64_t)(blockIdx.x - 1) * kPrepThreads + tid; i < g.R; i += stride) g.rpos[i] = -1;
        return;
    }
    __shared__ int first[1024], last[1024], pre[1025], slot[1024], wsum[16];
    int P = *g.ntp;
    P = P < g.sorted_cap ? P : (int)g.sorted_cap;
    const int bm = g.block_m, nb = P > 0 ? P / bm : 0;
    first[tid] = last[tid] = 0;
    __syncthreads();
    for (int b = tid; b < nb; b += kPrepThreads) {
        const int e = g.eids[b], before = g.eids[b > 0 ? b - 1 : 0], after = g.eids[b < nb - 1 ? b + 1 : b];
        if (e < 0 || e >= g.E) continue;
        if (b == 0 || before != e) first[e] = b;
        if (b == nb - 1 || after != e) last[e] = b + 1;
    }
    __syncthreads();
    int rows = 0;
    if (last[tid] > first[tid]) {
        // the valid rows of the last block: in eighths, then in the eighth
        // that they end in (two rounds of loads, where halving takes up to 7)
        const int *blk = g.sorted + (last[tid] - 1) * bm;
        auto valid = [&](int i) { return (uint32_t)blk[i] < (uint32_t)g.R; };
        const int step = bm >> 3;                    // 1 to 16
        int pos = 0;
#pragma unroll
        for (int k = 1; k <= 8; ++k) pos += valid(k * step - 1) ? step : 0;
        int more = 0;
        if (pos < bm) {
#pragma unroll
            for (int k = 0; k < 15; ++k) more += (int)valid(min(pos + k, bm - 1)) & (int)(k < step - 1);
        }
        rows = (last[tid] - 1 - first[tid]) * bm + pos + more;
    }
    int cnt = rows / tile_rows + (rows % tile_rows != 0);
    if (g.op == kGmmDw && !g.accumulate && tid < g.E && cnt == 0) cnt = 1;
    const int waves = (g.E + 63) >> 6;          // with experts (the others add nothing)
    auto scan = [&](int v) {                    // inclusive sum over the threads
        for (int d = 1; d < 64; d <<= 1) {
            const int o = __shfl_up(v, d, 64);
            if ((tid & 63) >= d) v += o;
        }
        __syncthreads();
        if ((tid & 63) == 63) wsum[tid >> 6] = v;
        __syncthreads();
        for (int q = 0; q < (tid >> 6) && q < waves; ++q) v += wsum[q];
        return v;
    };
    pre[tid + 1] = scan(cnt);
    if (tid == 0) pre[0] = 0;
    slot[tid] = -1;
    if (g.max_slots > 0) {
        const int end = scan(cnt > 1 ? cnt : 0);
        const bool cut = cnt > 1 && end <= g.max_slots;        // (no more in a plan that lists a route once)
        const int j = scan(cut ? 1 : 0);
        if (cut) {
            slot[tid] = end - cnt;
            g.joins[j - 1] = make_int4(tid, end - cnt, cnt, 0);
        }
        if (tid == kPrepThreads - 1) g.meta[1] = j;
    }
    __syncthreads();
    const int n = pre[1024];
    if (tid == 0) g.meta[0] = n;
    last[tid] = rows;
    __syncthreads();
    for (int i = tid; i < n && i < g.max_tiles; i += kPrepThreads) {
        int lo = 0, hi = g.E - 1;               // the expert e with pre[e] <= i < pre[e + 1]
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (pre[mid + 1] <= i) lo = mid + 1;
            else hi = mid;
        }
        const int off = (i - pre[lo]) * tile_rows;
        const int rem = last[lo] - off;
        g.tiles[i] = make_int4(first[lo] * bm + off, rem < tile_rows ? rem : tile_rows, lo,
                               slot[lo] >= 0 ? slot[lo] + i - pre[lo] : -1);
    }
}

// ------------------------------------------------------------- tile kernel

// The routes of an item's rows (forward, dx) stay in LDS from the step that
// sets its copies up to the one that stores its tile, in a ring of slots.
// Steps count the stages multiplied, k per item, with the copies S - 1 ahead:
// item i's routes are written in step i k - S, before that step's barrier
// (right after the copies of item i - 1's last stage), and read by its
// epilogue in step (i + 1) k - 1, after that step's barrier.  The item that
// takes the slot over may be written two steps after that and no sooner: only
// then is the next step's barrier between a slow wave's read and a fast wave's
// write.  A contraction of one stage needs S + 2 slots, longer ones fewer.
constexpr bool route_ring_holds(int slots, int S) {
    for (int k = 1; k <= S + 2; ++k) {
        const int read = k - 1, overwritten = slots * k - S;         // of item 0's slot
        if (overwritten < read + 2) return false;
    }
    return true;
}

// Columns of MFMA tile pair t: row i of tile 2 t + h is column
// 32 t + 8 (i / 4) + 4 h + i % 4, so that a lane's results of the pair
// (rows 4 (l / 16) + v of either) are 8 consecutive columns.
template <bool F16, int OP, int TP, int TQ, int WP, int WQ, int S>
struct Tile {
    static constexpr int NW = WP * WQ;
    static constexpr bool PKS = OP != kGmmFwd;      // operand memory runs along the output
    static constexpr bool QKS = OP == kGmmDw;
    static constexpr int PB = TP * 128, QB = TQ * 128, Stage = PB + QB;
    static constexpr int JP = PB / 1024 / NW;       // 1-KB copies per wave and stage
    static constexpr int JQ = (QB / 1024 + NW - 1) / NW;
    static constexpr int Ahead = (S - 2) * (JP + QB / 1024 / NW);   // copies that may be in flight
    static constexpr int NP = TP / WP / 16, NQ = TQ / WQ / 16;
    // behind the stages: the ring of the routes of items' rows (forward, dx),
    // or the routes of a stage's rows (two) and the list of parts (dw)
    static constexpr int Ring = S + 2;
    static_assert(route_ring_holds(Ring, S), "a slot is overwritten before its item is stored");
    static constexpr int Tail = QKS ? 2 * 256 : Ring * TQ * 4;
    static constexpr size_t Smem = (size_t)S * Stage + Tail;
    static_assert(NP % 2 == 0 && JP >= 1 && NW % 2 == 0 && Smem <= 160 * 1024, "tile");
    static_assert(!QKS || (TP == TQ && NQ % 2 == 0 && S == 2), "dw tile");
};

__device__ __forceinline__ u32x4 lds_read_tr(const uint8_t *p, int second) {
    typedef __attribute__((address_space(3))) v4s *lp;
    const v4s a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lp)p);
    const v4s b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lp)(p + second));
    const uint2 x = __builtin_bit_cast(uint2, a), y = __builtin_bit_cast(uint2, b);
    return u32x4{x.x, x.y, y.x, y.y};
}

template <bool F16, int OP, int TP, int TQ, int WP, int WQ, int S>
__global__ void __launch_bounds__(64 * WP * WQ)
group_tile_kernel(GroupMmArgs g) {
    using T = Tile<F16, OP, TP, TQ, WP, WQ, S>;
    constexpr int NW = T::NW, JP = T::JP, JQ = T::JQ, NP = T::NP, NQ = T::NQ;
    constexpr bool DW = OP == kGmmDw;
    extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
    int *rids = reinterpret_cast<int *>(smem + (size_t)S * T::Stage);          // [Ring][TQ] (forward, dx)
    int *sids = rids;                                                          // [2][64] (dw)
    int4 *parts = reinterpret_cast<int4 *>(smem + (size_t)S * T::Stage + 512); // [max_tiles] (dw)

    const int tid = threadIdx.x, l = tid & 63, w = uni(tid >> 6);
    const int wp = w % WP, wq = w / WP;
    const int np = OP == kGmmFwd ? g.N : g.K;                 // output columns
    const int nct = (np + TP - 1) / TP;

    // ---- the items of this workgroup: a contiguous range per XCD
    const int ntiles = min(uni(g.meta[0]), g.max_tiles);
    const int qtiles = DW ? (g.N + TQ - 1) / TQ : 1;
    const int n_items = ntiles * nct * qtiles;
    const int xcd = blockIdx.x & 7, step = gridDim.x >> 3;
    const int end = (int)((int64_t)(xcd + 1) * n_items / 8);
    int lit = (int)((int64_t)xcd * n_items / 8) + (blockIdx.x >> 3);     // load cursor
    int cit = lit;                                                        // compute cursor
    if (cit >= end) return;
    if (DW) {
        for (int i = tid; i < ntiles; i += 64 * NW) parts[i] = g.tiles[i];
        __syncthreads();
    }

    struct Item {
        int e, ct, qt, slot;         // expert, column tile; row tile and slot of the FP32 sums (dw)
        int row0, rows;              // its plan rows
    };
    auto item_of = [&](int i) {
        Item it = {};
        if (DW) {
            const int per = qtiles * nct, j = i / per;
            panel_tile<4>(i - j * per, qtiles, nct, it.qt, it.ct);
            const int4 t = parts[j];
            it.row0 = uni(t.x);
            it.rows = uni(t.y);
            it.e = uni(t.z);
            it.slot = uni(t.w);
        } else {
            int rt;
            panel_tile<4>(i, ntiles, nct, rt, it.ct);
            const int4 t = g.tiles[rt];
            it.row0 = uni(t.x);
            it.rows = uni(t.y);
            it.e = uni(t.z);
        }
        return it;
    };
    const int nred = OP == kGmmFwd ? g.K : g.N;               // the contraction (forward, dx)
    auto stages_of = [&](const Item &it) {
        return DW ? (it.rows > 0 ? (it.rows + 63) / 64 : 1) : (nred + 63) / 64;
    };

    // ---- load side.  A copy instruction of a wave fills 1 KB of a tile: 8
    // rows of 128 bytes, or 2 (TP = 256) or 4 rows of the output's columns.
    constexpr int RPI = 1024 / (TP * 2);                     // KS rows per copy
    const int lrow = l >> 3;
    const int kc_p = (l & 7) ^ ((lrow & 3) | ((w & 1) << 2));           // KC: global chunk (P swizzle)
    const int kc_q = (l & 7) ^ lrow;                                    // KC: global chunk (Q swizzle)
    const int ks_l = l / (TP / 8);                                      // KS: row in the copy
    const int ks_chunk = (l % (TP / 8)) ^ (((w * RPI + ks_l) & 3) << 2);   // (NW RPI is a multiple of 4)
    static_assert(!T::PKS || (NW * RPI) % 4 == 0, "the swizzle is the same for all copies");
    const uint8_t *pbase = nullptr;          // P, uniform: the wave's first copy of the stage
    uint32_t poff = 0;                       // its lane offset
    int plast = 0;                           // KC: last row of the tile that exists
    const uint8_t *qptr[JQ];                 // Q (forward, dx): each copy's row, gathered
    const uint8_t *xcol = nullptr, *dycol = nullptr;         // dw: the lane's columns
    const int64_t pstep = T::PKS ? (int64_t)(NW * RPI) * g.K * 2 : (int64_t)(8 * NW) * g.K * 2;
    const int64_t padv = T::PKS ? (int64_t)64 * g.K * 2 : 128;          // stage to stage
    Item ld = item_of(lit), ld_next = ld;
    int lkt = 0, lnk = 0, lord = 0;          // stage in the item, its stages, its ordinal

    auto load_setup = [&]() {
        lkt = 0;
        lnk = stages_of(ld);
        if (DW) {
            const int pc = ld.ct * TP + ks_chunk * 8, qc = ld.qt * TQ + ks_chunk * 8;
            xcol = reinterpret_cast<const uint8_t *>(g.x + (pc < g.K ? pc : 0));
            dycol = reinterpret_cast<const uint8_t *>(g.dy + (qc < g.N ? qc : 0));
            if (lit + step < end) ld_next = item_of(lit + step);
            return;
        }
        const int p0 = ld.ct * TP;
        const uint8_t *we = reinterpret_cast<const uint8_t *>(g.w + (int64_t)ld.e * g.N * g.K);
        if (T::PKS) {
            pbase = we + ((int64_t)(w * RPI) * g.K + p0) * 2;
            const int c = p0 + ks_chunk * 8 < g.K ? ks_chunk * 8 : 0;
            poff = ((uint32_t)ks_l * (uint32_t)g.K + (uint32_t)c) * 2u;
        } else {
            pbase = we + (int64_t)(p0 + 8 * w) * g.K * 2;
            poff = (uint32_t)lrow * (uint32_t)g.K * 2u + (uint32_t)kc_p * 16u;
            plast = min(TP, g.N - p0) - 1;
        }
        const uint16_t *src = OP == kGmmFwd ? g.x : g.dy;
        const int64_t ldq = OP == kGmmFwd ? g.ld_x : g.ld_dy;
#pragma unroll
        for (int j = 0; j < JQ; ++j) {
            const int row = 8 * (j * NW + w) + lrow;
            int r = row < ld.rows ? g.sorted[ld.row0 + row] : -1;
            if (r >= g.R) r = -1;
            if (row < TQ && (l & 7) == 0) rids[(lord % T::Ring) * TQ + row] = r;
            const int64_t xr = OP == kGmmFwd && !g.per_route ? g.token_of(r) : r;
            qptr[j] = r < 0 ? nullptr : reinterpret_cast<const uint8_t *>(src + xr * ldq) + kc_q * 16;
        }
    };

    // dw: the routes of stage kt of item it, 64 of them, into ids
    auto fetch_ids = [&](const Item &it, int kt, int *ids) {
        if (w != 0) return;
        const int last = it.rows > 0 ? it.rows - 1 : 0;
        const int i = kt * 64 + l < last ? kt * 64 + l : last;
        lds_dma4(g.sorted + it.row0 + i, ids);
    };

    // Copy c of the next stage into the slot at sp: P's JP copies, then Q's
    // JQ; in dw P's and Q's c-th together, as they share their rows (whose
    // routes are at ids).  `tail`: the stage reaches past the end of the
    // contraction, where both operands are read as zeros.
    constexpr int kCopies = DW ? JP : JP + JQ;
    const bool by_route = g.per_route || g.top_k == 1;
    const uint32_t ldx2 = (uint32_t)g.ld_x * 2u, ldy2 = (uint32_t)g.ld_dy * 2u;
    int rid[JP];                             // dw: routes of the lane's rows in the stage being copied
    auto issue_copy = [&](int c, uint8_t *sp, const int *ids, bool tail) {
        uint8_t *sq = sp + T::PB;
        const void *zero = kZeros;
        if (DW) {
            // (32-bit factors: each row address is one multiply-add)
            const int kr = (c * NW + w) * RPI + ks_l;
            const uint32_t r = (uint32_t)(tail ? ids[kr] : rid[c]);
            const bool ok = r < (uint32_t)g.R && kr < ld.rows - lkt * 64;
            const uint32_t xr = by_route ? r : __umulhi(r, g.div_m) >> (g.div_s - 1);
            const void *px = xcol + (uint64_t)xr * ldx2, *py = dycol + (uint64_t)r * ldy2;
            lds_dma16(ok ? px : zero, sp + (c * NW + w) * 1024);
            lds_dma16(ok ? py : zero, sq + (c * NW + w) * 1024);
        } else if (c < JP) {
            const int left = nred - lkt * 64;              // of the contraction
            const uint8_t *base = pbase + c * pstep;
            if (T::PKS) {
                const void *p = base + poff;
                if (tail && (c * NW + w) * RPI + ks_l >= left) p = zero;
                lds_dma16(p, sp + (c * NW + w) * 1024);
            } else {
                // rows past the last read the last one: first the copy's
                // first row moves back (uniform), then each lane by what its
                // own row exceeds it (at most lrow: the offset stays >= 0)
                const int r = 8 * (c * NW + w), back = max(r - plast, 0);
                const int over = max(r - back + lrow - plast, 0);
                const void *p = base - (int64_t)back * g.K * 2 + (poff - __umul24(over, 2 * g.K));
                if (tail && kc_p * 8 >= left) p = zero;
                lds_dma16(p, sp + (c * NW + w) * 1024);
            }
        } else {
            const int j = c - JP;
            if ((j + 1) * NW > T::QB / 1024 && j * NW + w >= T::QB / 1024) return;
            // rows without a route are zeros: multiplying them costs least power
            const void *p = qptr[j] ? (const void *)(qptr[j] + (int64_t)lkt * 128) : zero;
            if (tail && kc_q * 8 >= nred - lkt * 64) p = zero;
            lds_dma16(p, sq + (j * NW + w) * 1024);
        }
    };
    auto stage_issued = [&]() {
        pbase += padv;
        if (++lkt == lnk) {
            lit += step;
            ++lord;
            if (lit < end) {
                ld = DW ? ld_next : item_of(lit);
                load_setup();
            }
        }
    };

    // ---- compute side
    const int i16 = l & 15, grp = l >> 4;
    v4f acc[NP][NQ];
    auto clear = [&]() {
#pragma unroll
        for (int a = 0; a < NP; ++a)
#pragma unroll
            for (int b = 0; b < NQ; ++b) acc[a][b] = v4f{0.f, 0.f, 0.f, 0.f};
    };
    // LDS offsets of this lane's operand reads
    const int pf = (i16 & 3) | (((i16 >> 2) & 1) << 2);
    const int p_kc = (wp * (TP / WP) + 8 * (i16 >> 2) + (i16 & 3)) * 128 + ((grp ^ pf) << 4);
    const int q_kc = (wq * (TQ / WQ) + i16) * 128 + ((grp ^ (i16 & 7)) << 4);
    const int ks_row = 8 * grp + (i16 >> 2);
    const int ks_x = ((i16 >> 2) & 3) << 2;

    // A step is 2 NQ units, (contraction half kk, row tile n) in turn.  The
    // columns' operand (a) of a half and the rows' operand (b) of the units
    // ahead are read from LDS while earlier units are multiplied; the first
    // reads of a stage go out before the last kLast units of the stage before,
    // whose operands are in registers by then, so that neither the barrier
    // between the stages nor the reads' latency leaves the MFMAs idle.
    constexpr int kUnits = 2 * NQ, kAhead = NQ < 3 ? NQ : 3, kLast = kAhead;   // (the last units: second half)
    u32x4 a[2][NP], b[kUnits], head[kAhead];
    auto read_a = [&](const uint8_t *sp, int kk) {
#pragma unroll
        for (int n = 0; n < NP; ++n) {
            if constexpr (T::PKS) {
                const int ch = (wp * (TP / WP) / 8 + 4 * (n >> 1) + (i16 & 3)) ^ ks_x;
                a[kk][n] = lds_read_tr(sp + (kk * 32 + ks_row) * (TP * 2) + ch * 16 + (n & 1) * 8, 4 * TP * 2);
            } else {
                a[kk][n] = lds_read16(sp + (p_kc ^ (kk << 6)) + (n >> 1) * 32 * 128 + (n & 1) * 4 * 128);
            }
        }
    };
    auto read_b = [&](const uint8_t *sp, int u, u32x4 &bu) {
        const uint8_t *sq = sp + T::PB;
        const int kk = u / NQ, n = u % NQ;
        if constexpr (T::QKS) {
            const int ch = (wq * (TQ / WQ) / 8 + 4 * (n >> 1) + (i16 & 3)) ^ ks_x;
            bu = lds_read_tr(sq + (kk * 32 + ks_row) * (TQ * 2) + ch * 16 + (n & 1) * 8, 4 * TQ * 2);
        } else {
            bu = lds_read16(sq + (q_kc ^ (kk << 6)) + n * 16 * 128);
        }
    };

    auto store8 = [&](uint16_t *d, const v4f &x, const v4f &y) {
        u32x4 o;
        o.x = to16x2<F16>(x[0], x[1]);
        o.y = to16x2<F16>(x[2], x[3]);
        o.z = to16x2<F16>(y[0], y[1]);
        o.w = to16x2<F16>(y[2], y[3]);
        *reinterpret_cast<u32x4 *>(d) = o;
    };

    auto epilogue = [&](const Item &it, int ord) {
        const int c0 = it.ct * TP + wp * (TP / WP) + 8 * grp;
#pragma unroll
        for (int n = 0; n < NQ; ++n) {
            const int q = wq * (TQ / WQ) + (T::QKS ? 32 * (n >> 1) + 8 * (i16 >> 2) + 4 * (n & 1) + (i16 & 3)
                                                   : 16 * n + i16);
            if (DW) {
                const int row = it.qt * TQ + q;
                if (row >= g.N) continue;
                const int64_t o = ((int64_t)it.e * g.N + row) * g.K;
#pragma unroll
                for (int m = 0; m < NP / 2; ++m) {
                    const int c = c0 + 32 * m;
                    if (c >= g.K) continue;
                    v4f x = acc[2 * m][n], y = acc[2 * m + 1][n];
                    if (it.slot >= 0) {
                        float *d = g.part + ((int64_t)it.slot * g.N + row) * g.K + c;
                        *reinterpret_cast<v4f *>(d) = x;
                        *reinterpret_cast<v4f *>(d + 4) = y;
                    } else if (g.out_f32) {
                        float *d = (float *)g.out + o + c;
                        if (g.accumulate) {
                            x += *reinterpret_cast<v4f *>(d);
                            y += *reinterpret_cast<v4f *>(d + 4);
                        }
                        *reinterpret_cast<v4f *>(d) = x;
                        *reinterpret_cast<v4f *>(d + 4) = y;
                    } else {
                        uint16_t *d = (uint16_t *)g.out + o + c;
                        if (g.accumulate) {
                            const u32x4 old = *reinterpret_cast<const u32x4 *>(d);
#pragma unroll
                            for (int v = 0; v < 2; ++v) {
                                x[2 * v] += from16<F16>(old[v]);
                                x[2 * v + 1] += from16<F16>(old[v] >> 16);
                                y[2 * v] += from16<F16>(old[2 + v]);
                                y[2 * v + 1] += from16<F16>(old[2 + v] >> 16);
                            }
                        }
                        store8(d, x, y);
                    }
                }
            } else {
                const int r = rids[(ord % T::Ring) * TQ + q];
                if (r < 0) continue;
                if (OP == kGmmDx && !g.per_route) {
                    if (it.ct == 0 && wp == 0 && grp == 0) g.rpos[r] = 0;
                    float *d = g.part + (int64_t)r * g.K + c0;
#pragma unroll
                    for (int m = 0; m < NP / 2; ++m) {
                        if (c0 + 32 * m >= np) continue;
                        *reinterpret_cast<v4f *>(d + 32 * m) = acc[2 * m][n];
                        *reinterpret_cast<v4f *>(d + 32 * m + 4) = acc[2 * m + 1][n];
                    }
                } else {
                    uint16_t *d = (uint16_t *)g.out + (int64_t)r * g.ld_out + c0;
#pragma unroll
                    for (int m = 0; m < NP / 2; ++m)
                        if (c0 + 32 * m < np) store8(d + 32 * m, acc[2 * m][n], acc[2 * m + 1][n]);
                }
            }
        }
    };

    // ---- the pipeline
    int issued = 0, done = 0, islot = 0, slot = 0;       // stages issued and multiplied, their slots
    // This wave's copies of the stage have landed, then everyone's; all reads
    // of the slot that the next copies overwrite are complete.
    auto next_stage = [&]() {
        if (S > 2 && issued - done == S - 1) wait_vmcnt<(T::Ahead < 63 ? T::Ahead : 63)>();
        else wait_vmcnt<0>();
        __builtin_amdgcn_s_waitcnt(0xC07F);              // lgkmcnt(0)
        stage_barrier();
    };
    // dw: what follows stage lkt of ld, to fetch its routes along
    auto fetch_next = [&](int *ids) {
        if (lkt + 1 < lnk) fetch_ids(ld, lkt + 1, ids);
        else if (lit + step < end) fetch_ids(ld_next, 0, ids);
    };
    auto advance = [&]() {
        stage_issued();
        ++issued;
        islot = islot + 1 == S ? 0 : islot + 1;
    };
    // The products of the stage at rd but for the last units, and beside the
    // first units' the copies of the stage S - 1 steps ahead into wr (all at
    // once they would hold every wave up).  The pointers do not alias: rd, wr
    // are different slots, idr, idw different halves of sids; without that the
    // compiler would wait for all copies in flight before each transposing read.
    auto products = [&](int u) {
#pragma unroll
        for (int m = 0; m < NP; ++m) acc[m][u % NQ] = mfma32<F16>(a[u / NQ][m], b[u], acc[m][u % NQ]);
        __builtin_amdgcn_sched_barrier(0);
    };
    auto multiply = [&](const uint8_t *__restrict__ rd, uint8_t *__restrict__ wr, const int *__restrict__ idr,
                        int *__restrict__ idw, bool load) __attribute__((always_inline)) {
        const bool tail = !DW && load && (lkt + 1) * 64 > nred;
        if (tail) {
#pragma unroll
            for (int c = 0; c < kCopies; ++c) issue_copy(c, wr, idr, true);
        }
        const bool fast = load && !tail;
        if (DW && load) {
            fetch_next(idw);
#pragma unroll
            for (int c = 0; c < JP; ++c) rid[c] = idr[(c * NW + w) * RPI + ks_l];
        }
        constexpr int kIssue = kUnits - kLast < kUnits / 2 ? kUnits - kLast : kUnits / 2;
        constexpr int kPer = (kCopies + kIssue - 1) / kIssue;       // copies go out in kIssue units
#pragma unroll
        for (int u = 0; u < kAhead; ++u) b[u] = head[u];
#pragma unroll
        for (int u = 0; u < kUnits - kLast; ++u) {
            if (u == 0) read_a(rd, 1);
            read_b(rd, u + kAhead, b[u + kAhead]);
            if (fast) {
#pragma unroll
                for (int c = u * kPer; c < (u + 1) * kPer && c < kCopies; ++c) issue_copy(c, wr, idr, false);
            }
            products(u);
        }
    };
    // the first reads of the stage at rd
    auto read_head = [&](const uint8_t *rd) {
        read_a(rd, 0);
#pragma unroll
        for (int u = 0; u < kAhead; ++u) read_b(rd, u, head[u]);
    };
    // For more than two stages, with the next stage's first reads in the same
    // scope as the copies that they must not wait for.
    auto multiply_head = [&](const uint8_t *__restrict__ rd, uint8_t *__restrict__ wr,
                             const uint8_t *__restrict__ nx, bool load) __attribute__((always_inline)) {
        multiply(rd, wr, sids, sids, load);
        if (load) advance();
        ++done;
        if (issued > done) {
            next_stage();
            read_head(nx);
        }
    };
    Item cur = ld;
    int ckt = 0, cnk = stages_of(cur), cord = 0;
    load_setup();
    if (DW) {
        fetch_ids(ld, 0, sids);
        wait_vmcnt<0>();
        __syncthreads();
    }
    for (int s = 0; s < S - 1 && lit < end; ++s) {
        if (DW) fetch_next(sids + 64);
#pragma unroll
        for (int c = 0; c < kCopies; ++c) issue_copy(c, smem + islot * T::Stage, sids, true);
        advance();
    }
    clear();
    next_stage();
    read_head(smem);
    while (true) {
        const bool load = lit < end;
        const int nslot = slot + 1 == S ? 0 : slot + 1;
        const uint8_t *rd = smem + slot * T::Stage, *nx = smem + nslot * T::Stage;
        uint8_t *wr = smem + islot * T::Stage;
        if constexpr (S > 2) {
            multiply_head(rd, wr, nx, load);
        } else {
            multiply(rd, wr, sids + islot * 64, sids + (islot ^ 1) * 64, load);
            if (load) advance();
            ++done;
            if (issued > done) {
                next_stage();
                read_head(nx);
            }
        }
#pragma unroll
        for (int u = kUnits - kLast; u < kUnits; ++u) products(u);
        slot = nslot;
        if (++ckt == cnk) {
            epilogue(cur, cord);
            cit += step;
            if (cit >= end) break;
            clear();
            cur = item_of(cit);
            ckt = 0;
            cnk = stages_of(cur);
            ++cord;
        }
    }
}

// --------------------------------------------------- few rows: the forward

// The forward product where experts hold a few rows each (decoded tokens):
// the time is that of reading the touched experts' weights once.  A workgroup
// takes 16 weight rows of one plan block; its NW waves split K, load weights
// straight into registers (no LDS ring and no set-up launch to wait for) U
// steps of 64 at a time, and add up in LDS in order.  x rows are loaded in
// the operand's layout too where a row or so is left of an expert; where more
// differ (XL) they are copied to the wave's share of LDS, 8 whole rows of 128
// bytes an instruction: a register load touches 16 rows, 64 bytes of each,
// and costs the L1 twice the accesses (E = 8, K = 4096, N = 2048, 8 rows an
// expert: 28.2 -> 25.7 us).  Plan blocks with more than 16 NQ routes go
// through the weights again for each further 16 NQ.  Measured: one token, 9
// of 257 experts, K = 7168, N = 512: 19 us for 66 MB, 3.5 TB/s with the
// launch; 64 experts of 8 rows, K = 2048, N = 1024: 268 MB at 5.5 TB/s.
template <bool F16, int NQ, int NW, int U, bool XL>
__global__ void __launch_bounds__(64 * NW, 3)
group_stream_kernel(GroupMmArgs g) {
    // a wave's share of LDS: its rows of x (XL), then its sums [NQ][16][17]
    constexpr int kSums = (NQ * 16 * 17 * 4 + 15) / 16 * 16, kRows = XL ? U * NQ * 2048 : 0;
    constexpr int kWave = kRows > kSums ? kRows : kSums;
    __shared__ __attribute__((aligned(16))) uint8_t smem[NW * kWave];
    const int tid = threadIdx.x, l = tid & 63, w = uni(tid >> 6), i16 = l & 15, grp = l >> 4;
    uint8_t *const lds = smem + w * kWave;
    // the lane's rows of x: row 16 n + i16, or in copies of 8 rows x 128 bytes
    // row 8 n + l / 8
    constexpr int NR = XL ? 2 * NQ : NQ;
    auto row_of = [&](int n) { return XL ? 8 * n + (l >> 3) : 16 * n + i16; };
    // the plan's length and the block's routes are read together (the block
    // lies within sorted_cap), its expert once the block is known to exist
    const int b = blockIdx.y, bm = g.block_m;
    int P = *g.ntp, ids[NR];
#pragma unroll
    for (int n = 0; n < NR; ++n) ids[n] = g.sorted[b * bm + min(row_of(n), bm - 1)];
    P = P < g.sorted_cap ? P : (int)g.sorted_cap;
    if ((b + 1) * bm > P) return;
    const int e = uni(g.eids[b]);
    if (e < 0 || e >= g.E) return;
    const int c0 = blockIdx.x * 16;
    const int c = c0 + i16 < g.N ? c0 + i16 : g.N - 1;
    const uint16_t *ap = g.w + ((int64_t)e * g.N + c) * g.K;
    const int nk = (g.K + 63) / 64;
    const int x_off = i16 * 128 + ((grp ^ (i16 & 7)) << 4);
    const u32x4 zero = {0u, 0u, 0u, 0u};

    for (int row0 = b * bm; row0 < (b + 1) * bm; row0 += 16 * NQ) {
        if (row0 > b * bm) {
#pragma unroll
            for (int n = 0; n < NR; ++n) ids[n] = g.sorted[row0 + min(row_of(n), bm - 1)];
        }
        const int r0 = uni(ids[0]);                     // (lane 0: the first row)
        if (r0 < 0 || r0 >= g.R) break;                 // sentinels end the segment
        const uint16_t *bp[NR];
#pragma unroll
        for (int n = 0; n < NR; ++n) {
            int r = ids[n];
            if (r < 0 || r >= g.R) r = r0;              // results of these rows are not stored
            bp[n] = g.x + (int64_t)(g.per_route ? r : g.token_of(r)) * g.ld_x;
        }
        v4f acc[NQ];
#pragma unroll
        for (int n = 0; n < NQ; ++n) acc[n] = v4f{0.f, 0.f, 0.f, 0.f};
        for (int k0 = w; k0 < nk; k0 += NW * U) {
            u32x4 a[U][2], x[U][NQ][2];
            bool ok[U][2];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int ks = (k0 + u * NW) * 64;
                if (ks >= g.K) break;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    // past the end of K: zeros on both sides
                    const int k = ks + 32 * h + 8 * grp;
                    ok[u][h] = k < g.K;
                    a[u][h] = *(const u32x4 *)(ap + (ok[u][h] ? k : 0));
                    if (!XL) {
#pragma unroll
                        for (int n = 0; n < NQ; ++n) x[u][n][h] = *(const u32x4 *)(bp[n] + (ok[u][h] ? k : 0));
                    }
                }
                if (XL) {
                    const int k = ks + 8 * ((l & 7) ^ (l >> 3));       // chunk c of row r lies at c ^ (r & 7)
#pragma unroll
                    for (int n = 0; n < NR; ++n)
                        lds_dma16(k < g.K ? (const void *)(bp[n] + k) : (const void *)kZeros,
                                  lds + (u * NR + n) * 1024);
                }
            }
            __builtin_amdgcn_sched_barrier(0);          // every load above is issued first
            if (XL) {
                asm volatile("s_waitcnt vmcnt(0)" ::: "memory");       // the wave's own copies
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    if ((k0 + u * NW) * 64 >= g.K) break;
#pragma unroll
                    for (int n = 0; n < NQ; ++n) {
                        x[u][n][0] = lds_read16(lds + (u * NQ + n) * 2048 + x_off);
                        x[u][n][1] = lds_read16(lds + (u * NQ + n) * 2048 + (x_off ^ 64));
                    }
                }
                // read before the next steps' copies write there
                asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if ((k0 + u * NW) * 64 >= g.K) break;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const u32x4 av = ok[u][h] ? a[u][h] : zero;
#pragma unroll
                    for (int n = 0; n < NQ; ++n)
                        acc[n] = mfma32<F16>(av, XL || ok[u][h] ? x[u][n][h] : zero, acc[n]);
                }
            }
        }
#pragma unroll
        for (int n = 0; n < NQ; ++n)
#pragma unroll
            for (int v = 0; v < 4; ++v)
                reinterpret_cast<float *>(lds)[(n * 16 + i16) * 17 + 4 * grp + v] = acc[n][v];
        __syncthreads();
        for (int i = tid; i < 16 * NQ * 8; i += 64 * NW) {
            const int cc = (i & 7) * 2, q = i >> 3;
            if (q >= bm || c0 + cc >= g.N) continue;
            const int r = g.sorted[row0 + q];
            if (r < 0 || r >= g.R) continue;
            float z0 = 0.f, z1 = 0.f;
            for (int k = 0; k < NW; ++k) {
                const float *d = reinterpret_cast<const float *>(smem + k * kWave) + q * 17 + cc;
                z0 += d[0];
                z1 += d[1];
            }
            *reinterpret_cast<uint32_t *>((uint16_t *)g.out + (int64_t)r * g.ld_out + c0 + cc) =
                to16x2<F16>(z0, z1);
        }
        __syncthreads();
    }
}

// ------------------------------------------------------------ joining sums

// dx[t] = the sum of the token's routes' FP32 rows, in route order.  A
// workgroup takes 256 / lanes tokens and lanes x 8 columns of them.
template <bool F16>
__global__ void __launch_bounds__(256)
group_sum_kernel(GroupMmArgs g, int lanes, int64_t blocks) {
    const int per = (g.K / 8 + lanes - 1) / lanes, row = threadIdx.x / lanes, col = threadIdx.x % lanes;
    for (int64_t b = blockIdx.x; b < blocks; b += gridDim.x) {
        const int64_t t = b / per * (256 / lanes) + row;
        const int c = ((int)(b % per) * lanes + col) * 8;
        if (t >= g.M || c >= g.K) continue;
        v4f x = {0.f, 0.f, 0.f, 0.f}, y = x;
        for (int j = 0; j < g.top_k; ++j) {
            const int64_t r = t * g.top_k + j;
            if (g.rpos[r] < 0) continue;
            x += *reinterpret_cast<const v4f *>(g.part + r * g.K + c);
            y += *reinterpret_cast<const v4f *>(g.part + r * g.K + c + 4);
        }
        u32x4 o;
        o.x = to16x2<F16>(x[0], x[1]);
        o.y = to16x2<F16>(x[2], x[3]);
        o.z = to16x2<F16>(y[0], y[1]);
        o.w = to16x2<F16>(y[2], y[3]);
        *reinterpret_cast<u32x4 *>((uint16_t *)g.out + t * g.ld_out + c) = o;
    }
}

// dw of the experts whose rows were cut = the sum of their parts' FP32 tiles,
// in order.
template <bool F16>
__global__ void __launch_bounds__(256)
group_join_kernel(GroupMmArgs g) {
    const int64_t n = (int64_t)g.N * g.K, per = (n / 4 + 255) / 256;
    const int64_t items = g.meta[1] * per;
    for (int64_t b = blockIdx.x; b < items; b += gridDim.x) {
        const int4 t = g.joins[b / per];
        const int64_t i = ((b % per) * 256 + threadIdx.x) * 4;
        if (i >= n) continue;
        v4f s = {0.f, 0.f, 0.f, 0.f};
        for (int k = 0; k < t.z; ++k) s += *reinterpret_cast<const v4f *>(g.part + (t.y + k) * n + i);
        if (g.out_f32) {
            v4f *d = reinterpret_cast<v4f *>((float *)g.out + t.x * n + i);
            *d = g.accumulate ? *d + s : s;
        } else {
            uint2 *d = reinterpret_cast<uint2 *>((uint16_t *)g.out + t.x * n + i);
            if (g.accumulate) {
                const uint2 o = *d;
                s[0] += from16<F16>(o.x);
                s[1] += from16<F16>(o.x >> 16);
                s[2] += from16<F16>(o.y);
                s[3] += from16<F16>(o.y >> 16);
            }
            *d = uint2{to16x2<F16>(s[0], s[1]), to16x2<F16>(s[2], s[3])};
        }
    }
}

// ----------------------------------------------------------------- launch

// Most parts that dw cuts the experts' rows into: their list stays in LDS.
constexpr int kMaxParts = 1984;
static_assert(Tile<true, kGmmDw, 256, 256, 4, 2, 2>::Smem + kMaxParts * 16 <= 160 * 1024, "list of parts");

template <bool F16, int OP, int TP, int TQ, int WP, int WQ, int S>
hipError_t launch_tile(const GroupMmArgs &g, int64_t max_items, hipStream_t st) {
    using T = Tile<F16, OP, TP, TQ, WP, WQ, S>;
    static std::atomic<uint64_t> done{0};
    auto fn = group_tile_kernel<F16, OP, TP, TQ, WP, WQ, S>;
    const size_t smem = T::Smem + (OP == kGmmDw ? (size_t)g.max_tiles * 16 : 0);
    hipError_t e = raise_lds_limit(done, (const void *)fn, (int)(T::Smem + (OP == kGmmDw ? kMaxParts * 16 : 0)));
    if (e != hipSuccess) return e;
    const int64_t per_cu = (160 * 1024) / (int64_t)smem;
    int64_t grid = (int64_t)device_cu_count() * (per_cu < 2 ? 1 : 2);
    if (grid > max_items) grid = max_items;
    grid = (grid + 7) / 8 * 8;
    fn<<<(unsigned)grid, 64 * WP * WQ, smem, st>>>(g);
    return hipGetLastError();
}

template <bool F16, int OP>
hipError_t launch_rows(const GroupMmArgs &g, hipStream_t st) {
    const int np = OP == kGmmFwd ? g.N : g.K;
    const int64_t items = (int64_t)g.max_tiles * ((np + 255) / 256);
    switch (g.tile_rows) {
        case 256: return launch_tile<F16, OP, 256, 256, 4, 2, 2>(g, items, st);
        case 128: return launch_tile<F16, OP, 256, 128, 4, 2, 3>(g, items, st);
        case 64: return launch_tile<F16, OP, 256, 64, 4, 2, 3>(g, items, st);
        default: return launch_tile<F16, OP, 256, 32, 8, 1, 4>(g, items, st);
    }
}

template <bool F16>
hipError_t launch_sum(const GroupMmArgs &g, hipStream_t st) {
    int lanes = 256;                                   // threads of a token: K / 8, up to a power of two
    while (lanes > 1 && lanes / 2 >= g.K / 8) lanes /= 2;
    const int64_t tokens = 256 / lanes;
    const int64_t blocks = (g.M + tokens - 1) / tokens * ((g.K / 8 + lanes - 1) / lanes);
    group_sum_kernel<F16><<<(unsigned)std::min(blocks, (int64_t)1 << 23), 256, 0, st>>>(g, lanes, blocks);
    return hipGetLastError();
}

template <bool F16>
hipError_t launch(const GroupMmArgs &g, hipStream_t st) {
    if (g.stream) {
        const dim3 grid((g.N + 15) / 16, (unsigned)(g.sorted_cap / g.block_m));
        if (g.stream == 2) group_stream_kernel<F16, 2, 4, 2, true><<<grid, 256, 0, st>>>(g);
        else if (g.R > 4 * g.E) group_stream_kernel<F16, 1, 4, 4, true><<<grid, 256, 0, st>>>(g);
        else group_stream_kernel<F16, 1, 4, 4, false><<<grid, 256, 0, st>>>(g);
        return hipGetLastError();
    }
    const bool summed = g.op == kGmmDx && !g.per_route;
    const int64_t fill = summed ? (g.R + 8 * kPrepThreads - 1) / (8 * kPrepThreads) : 0;
    group_prep_kernel<<<(unsigned)(1 + (fill < 255 ? fill : 255)), kPrepThreads, 0, st>>>(g, g.tile_rows);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    if (g.op == kGmmDw) {
        const int64_t t = g.dw_tile;
        const int64_t items = (int64_t)g.max_tiles * ((g.N + t - 1) / t) * ((g.K + t - 1) / t);
        e = t == 256 ? launch_tile<F16, kGmmDw, 256, 256, 4, 2, 2>(g, items, st)
                     : launch_tile<F16, kGmmDw, 128, 128, 2, 2, 2>(g, items, st);
        if (e != hipSuccess || g.max_slots == 0) return e;
        const int64_t n = (int64_t)g.max_slots * (((int64_t)g.N * g.K / 4 + 255) / 256);
        group_join_kernel<F16><<<(unsigned)std::min(n, (int64_t)2048), 256, 0, st>>>(g);
        return hipGetLastError();
    }
    e = g.op == kGmmFwd ? launch_rows<F16, kGmmFwd>(g, st) : launch_rows<F16, kGmmDx>(g, st);
    if (e != hipSuccess || !summed) return e;
    return launch_sum<F16>(g, st);
}

}  // namespace

hipError_t launch_group_mm(const GroupMmArgs &g, hipStream_t st) {
    return g.f16 ? launch<true>(g, st) : launch<false>(g, st);
}

hipError_t launch_group_no_routes(GroupMmArgs g, hipStream_t st) {
    g.top_k = 0;                                       // sums of nothing
    return launch_sum<false>(g, st);
}

size_t group_mm_workspace(GroupMmArgs &g, void *ws) {
    // r / top_k for 0 <= r < 2^31 by one high product: with s the least
    // number with 2^s >= top_k and m = floor(2^(31 + s) / top_k) + 1 (below
    // 2^32), m top_k exceeds 2^(31 + s) by at most top_k <= 2^s, so
    // floor(r m / 2^(31 + s)) is the quotient.
    int s = 0;
    while (((int64_t)1 << s) < g.top_k) ++s;
    g.div_m = (uint32_t)((((uint64_t)1 << (31 + s)) / (uint64_t)g.top_k) + 1);
    g.div_s = s;

    const int64_t rpe = g.R / g.E;
    const double R = (double)g.R, E = (double)g.E;
    const double hit = E * -std::expm1(R * std::log1p(-1.0 / E));    // experts with a route
    const double rows = R / hit;
    const double wbytes = hit * g.N * g.K * 2;

    // Forward, dx: the tile by estimated time (us), with routes spread evenly
    // over the experts (rows of one: about normal, variance `rows`).  Per step
    // of 64 of the contraction, measured with every CU busy, 256 columns x
    // 256 / 128 / 64 / 32 rows take 2.1 / 0.95 / 0.65 / 0.55 (128 columns x 64
    // rows 0.72: no gain from narrower tiles); a tile's fill and store about
    // 4.  Each row tile reads its expert's weights, at most 5.5 TB/s of them.
    // Measured at E = 288, K = 4096, N = 2048 with 14, 28, 56, 113, 227 rows
    // an expert: 256 rows 1271, 1267, 1214, 1273, 1545; 128: 938, 938, 878,
    // 1057, 1686; 64: 864, 875, 958, 1313, 2024; 32: 850, 913, 1196, 1692, 3015.
    const int np = g.op == kGmmFwd ? g.N : g.K, nred = g.op == kGmmFwd ? g.K : g.N;
    const int steps = (nred + 63) / 64;
    struct Form {
        int rows;
        double step;
    };
    static const Form forms[4] = {{256, 2.1}, {128, 0.95}, {64, 0.65}, {32, 0.55}};
    auto parts = [&](int size) {                          // of at most `size` rows, of an expert
        double per = 0;
        if (rows > 32.0 * size) per = rows / size + 0.5;
        else
            for (int i = 0; i * size < rows + 5 * std::sqrt(rows) + 1; ++i)
                per += 0.5 * std::erfc((i * size + 0.5 - rows) / std::sqrt(2 * rows));
        return std::max(per, 1.0);
    };
    double t_tile = 1e300;
    g.tile_rows = 32;
    for (const Form &f : forms) {
        const double per = parts(f.rows);
        const double rounds = hit * per * ((np + 255) / 256) / 256;
        const double busy = (rounds < 4 ? std::ceil(rounds) : rounds + 0.5) * (steps * f.step + 4);
        const double mem = per * wbytes / 5.5e6;
        const double t = std::max(busy, mem) + 0.1 * std::min(busy, mem);
        if (t < t_tile) {
            t_tile = t;
            g.tile_rows = f.rows;
        }
    }
    // The few-rows kernel, whose workgroups go through 16 columns' weights
    // once for every 16 or 32 rows of a plan block: about 0.07 or 0.1 us per
    // 64 of K on each CU, or the weights' way from HBM.  The tile kernels need
    // a set-up launch before, some 3 us.  Measured (us, 16 rows / 32 rows /
    // tile): E = 8, K = 4096, N = 2048, block_m 64 with 8, 16, 32, 75 rows an
    // expert 26, 40, 62, 109 / 27, 28, 45, 72 / 45, 45, 46, 54; E = 8, K =
    // 256, N = 512 with 2, 16, 75 rows 3.4, 4.6, 7.6 / 3.7, 3.8, 5.5 / 10, 10,
    // 10.5; E = 32, K = 2048, N = 1024 with 2, 16, 62 rows 28, 41, 89 / 28,
    // 29, 59 / 27, 27, 33.
    double t_few = 0;
    g.stream = 0;
    if (g.op == kGmmFwd && g.sorted_cap / g.block_m <= 65535)
        for (int nq = 1; nq <= 2; ++nq) {
            const double wgs = hit * parts(std::min(g.block_m, 16 * nq)) * ((g.N + 15) / 16);
            const double t = 2.5 + std::max(std::max(wgs / 256, 1.0) * steps * (0.04 + 0.03 * nq), wbytes / 5.5e6);
            if (t < t_tile + 3 && (g.stream == 0 || t < t_few)) {
                g.stream = nq;
                t_few = t;
            }
        }
    if (g.stream) return 0;
    g.max_slots = 0;
    g.dw_tile = 256;
    if (g.op == kGmmDw) {
        // The tile and the splits by estimated time (us): 256-squared tiles
        // take about 2.3 for each 64 rows, one to a CU; 128-squared ones 1.3,
        // or 1.5 with two on a CU; a tile's fill and store 4; the join 4 and
        // the way of the parts out and in.  Measured (us, 128-squared without
        // splits beyond 256 items / so chosen): E = 4, K = 712, N = 1288 with
        // 2048, 8192 rows an expert 59, 187 / 50, 106; E = 1, K = 4096, N =
        // 2048 with 16384 rows 389 / 289; E = 3, K = 1000, N = 2048 with 5461
        // rows 136 / 103.
        double best = 1e300;
        int nsplit = 1;
        for (int t = 128; t <= 256; t += 128) {
            const int64_t tiles = (int64_t)g.E * ((g.N + t - 1) / t) * ((g.K + t - 1) / t);
            for (int sp = 1; sp == 1 || (sp <= 64 && sp <= rpe / 128 && tiles * sp <= 512); ++sp) {
                const int64_t items = tiles * sp, fit = t == 128 && items > 256 ? 512 : 256;
                const double step = t == 256 ? 2.3 : fit == 512 ? 1.5 : 1.3;
                const int64_t stages = (rpe + 64 * sp - 1) / (64 * sp);
                const double cost = (double)((items + fit - 1) / fit) * ((double)stages * step + 4) +
                                    (sp > 1 ? 4 + sp * ((double)g.E * g.N * g.K * 8 / 5e6) : 0);
                if (cost < best) {
                    best = cost;
                    g.dw_tile = t;
                    nsplit = sp;
                }
            }
        }
        // Rows of an expert are cut into parts of tile_rows.  Also where an
        // even spread needs no cut: an expert with more than twice the average
        // would take its time alone (190 experts of K = 152, N = 240 with 230
        // rows on average, one of them with a fifth of all: 141 us uncut, 37
        // cut).  The join's launch costs 4 us and a cut expert's parts FP32
        // slots (an expert with several parts has fewer than 2 rows /
        // tile_rows of them): not for few rows, and not for more than 256 MB.
        // (Room for the spread of a random routing, so that it gives no
        // further part.)
        const int64_t most = rpe + (int64_t)(3 * std::sqrt((double)rpe)) + 1;
        const int64_t even = (most + 64 * nsplit - 1) / (64 * nsplit) * 64;
        int64_t cut = nsplit > 1 ? even : 2 * even;
        if (nsplit == 1 && (g.R < 4096 || g.R * 2 / cut * g.N * g.K > (int64_t)1 << 26)) cut = g.R;
        if (g.R / cut + g.E > kMaxParts) cut = g.R;
        if (cut > g.R) cut = g.R;
        g.tile_rows = (int)cut;
        if (cut < g.R) g.max_slots = (int)(2 * g.R / cut);
    }
    g.max_tiles = (int)(g.R / g.tile_rows + (g.E < g.R || g.op == kGmmDw ? g.E : g.R));
    uint8_t *base = (uint8_t *)ws;
    size_t off = 0;
    auto take = [&](size_t n) {
        uint8_t *p = base + off;
        off += (n + 255) & ~size_t(255);
        return p;
    };
    g.meta = (int32_t *)take(8);
    g.tiles = (int4 *)take((size_t)g.max_tiles * 16);
    if (g.op == kGmmDx && !g.per_route) {
        g.rpos = (int32_t *)take((size_t)g.R * 4);
        g.part = (float *)take((size_t)g.R * g.K * 4);
    }
    if (g.max_slots > 0) {
        g.joins = (int4 *)take((size_t)g.max_slots * 16);
        g.part = (float *)take((size_t)g.max_slots * g.N * g.K * 4);
    }
    return off;
}

}  // namespace moe
