// km_xent_fused.cuh -- gradients of the cross entropy for rows of up to 128 values, P never leaving
// the SM.
//
// For short rows the exponentials, not the products, are the larger part of the gradient, and
// writing P and reading it twice costs more than either. Here a block keeps 128 rows of one side
// (points for dX, table rows for dC) and walks over tiles of 128 rows of the other:
//     S = A B^T (tcgen05, TMEM)  ->  P = w (2^(S s + off) - [label])  ->  TMEM, 16 bits
//     O += P B (tcgen05, P as the row operand from TMEM)
// so each tile of B is loaded once and used by both products: as it lies for the first (K-major), and
// read across (MN-major) for the second. Each gradient computes its own exponentials.
//
// A tile of 128 x 128 at d = 128 takes 16 MMAs of 64 cycles and as many cycles of exponentials (16384 at 16 a
// cycle). Measured at 32768 x 8192: 2200 cycles a tile. The MMAs of a tile come in two runs, O and S, and
// the second waits for the first to complete (about 340 cycles beyond its last MMA); without that wait
// the time was the same within 2%, so what bounds it is the time until the issuing warp sees each barrier
// beside the eight warps of exponentials. What each step gave (dX / dC of that case, us): one group
// of warps in step 189 / 172; two groups with a buffer of S and P each 165 / 157; three buffers, one
// thread issuing, and the loop over 32 columns rolled (the longer body displaced the issuer's
// instructions) 146 / 149; draining O, and the look for infinite rows of the table, 146 / 155.
//
// A block's share is an equal run of the tiles of all row tiles, so that every SM works to the end; a row
// tile that is shared by several blocks is summed from their partials, in block order.
//
// Roles (10 warps): 0 requests, 1 issues the MMAs, 2-9 take the exponentials: two groups of four warps,
// even and odd tiles, so that one group's loads and stores lie under the other's exponentials; a thread
// takes a row of 128. TMEM: three buffers of S, in which P replaces what has been read, and one of O. The
// MMAs of O of tile i, once complete, are followed by those of S of tile i + 3 in the same buffer. Waits
// are bounded as everywhere in the library.
#pragma once

#include "km_xent.cuh"

namespace km {
namespace xe {

constexpr int FR = 128;                  // rows of a tile, either side
constexpr int F_EPI0 = 2, F_GROUP = 4, F_EPI_WARPS = 2 * F_GROUP;
constexpr int F_THREADS = 32 * (F_EPI0 + F_EPI_WARPS);

// What the points bring to P, in tiles of 128: off = log2 |w| - lse log2 e (-inf without a label), w
// (scaled), the label (-1 for none).
struct __align__(16) PointTile {
    float off[FR], w[FR];
    int label[FR];
};

// The same of one point where it is a row of P (dX): relative to its own weight, so that what a row of dX
// holds does not depend on the other points' weights; `factor`, |w| / s, is put back in the result. off = log2 s -
// lse log2 e, w = s with the weight's sign.
struct __align__(16) PointRow {
    float off, w, factor;
    int label;
};

template <int DN, bool COL> struct FShape {
    static constexpr int kChunks = DN / 64;
    static constexpr uint32_t kTile = FR * DN * 2;
    static constexpr uint32_t kParam = COL ? 2048 : 0;         // a PointTile, up to whole swizzle atoms
    static constexpr int kABufs = DN == 64 ? 2 : 1;
    // tiles i .. i + 3 are in use at once, the rest is on its way
    static constexpr int kStages = DN == 64 ? 8 : COL ? 5 : 6;
    static constexpr uint32_t kStage = kTile + kParam;
    static constexpr uint32_t kBarOff = kABufs * kTile + kStages * kStage;
    static constexpr int kBars = 2 * kStages + 13;
    static constexpr uint32_t kTotal = kBarOff + kBars * 8 + 16 + 1024;
};
template <typename T> __device__ __forceinline__ float unpack_lo(uint32_t v) {
    const uint16_t h = static_cast<uint16_t>(v);
    return Cvt<T>::to_f(*reinterpret_cast<const T *>(&h));
}
template <typename T> __device__ __forceinline__ float unpack_hi(uint32_t v) { return unpack_lo<T>(v >> 16); }

// A product's additions into TMEM truncate, about 1e-7 of the sum each where all terms have one sign
// (measured: 28000 of them 2.5e-3), so that a long sum would drift further than its result's own rounding.
// After 1024 of them O is drained and the pieces are added in fp32, through the block's partials: 1e-4 at
// most, less than half of fp16's half step. (32768 x 8192 at d = 128: no slower; 131072 x 8192: dX 502 to
// 508 us, dC 548 to 572.)
constexpr int kMaxChain = 1024;
template <bool LO> constexpr int fused_run() { return kMaxChain / (LO ? 2 * (FR / 16) : FR / 16); }    // tiles

constexpr int F_SBUFS = 3;
constexpr uint32_t F_OCOL = F_SBUFS * FR;          // TMEM: S and P, then O

struct FParams {
    int M, cols, d;           // rows of A, rows of B, values of a row
    int mt, ct;               // tiles of A and of B, a batch
    int tiles;                // mt * ct * batches, shared out over the blocks
    float scale;              // |scale|
    uint32_t idesc_s, idesc_o;
    const PointTile *points;  // [batches][tiles of points] (dC)
    const PointRow *rows;     // [batches][tiles of points][128] (dX)
    const unsigned int *wmax;
    float pscale;
    int withhold;             // test only: the first block never asks for its first tile
    float *parts;             // [blocks][2][128][DN]: a block's first and last row tile, where shared
    void *out;
    int vec;
};

// A block's tiles begin here.
__host__ __device__ inline int fused_begin(int tiles, int blocks, int block) {
    const int q = tiles / blocks, r = tiles % blocks;
    return q * block + (block < r ? block : r);
}

// The parameters of every point, filled up to whole tiles with points that have none.
__global__ void __launch_bounds__(256)
    point_param_kernel(const float *__restrict__ w, const float *__restrict__ lse, const int32_t *__restrict__ ids,
                       int64_t B, int N, int64_t tiles, int K, const unsigned int *__restrict__ wmax, float pscale,
                       PointTile *__restrict__ out, PointRow *__restrict__ rows) {
    const float fac = p_factor(wmax, pscale, false);
    for (int64_t i = blockIdx.x * 256ll + threadIdx.x; i < B * tiles * FR; i += gridDim.x * 256ll) {
        const int64_t t = i / FR, b = t / tiles;
        const int k = static_cast<int>(i % FR);
        const int64_t n = (t - b * tiles) * FR + k;
        float off = -INFINITY, v = 0.f;
        int label = -1;
        PointRow row = {-INFINITY, 0.f, 0.f, -1};
        if (n < N) {
            const int id = ids[b * N + n];
            if (id >= 0 && id < K) {
                const float wn = w[b * N + n], l = lse[b * N + n] * kLog2e;
                v = wn * fac;
                off = __log2f(fabsf(v)) - l;
                label = id;
                row.label = id;
                if (wn != 0.f) {
                    row.off = __log2f(pscale) - l;
                    row.w = wn < 0.f ? -pscale : pscale;
                    row.factor = fabsf(wn) / pscale;
                }
            }
        }
        out[t].off[k] = off;
        out[t].w[k] = v;
        out[t].label[k] = label;
        rows[i] = row;
    }
}

// D[tmem] (+)= A B^T with descriptors whose upper words are the same; the row operand from shared memory
// or from TMEM.
template <bool ACC> __device__ __forceinline__ void f_mma_ss(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t hi, uint32_t idesc) {
    asm volatile("{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\t"
                 "mov.b64 da, {%1, %3};\n\tmov.b64 db, {%2, %3};\n\t"
                 "setp.ne.b32 p, %5, 0;\n\t"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %4, p;\n\t}" ::"r"(d),
                 "r"(a_lo), "r"(b_lo), "r"(hi), "r"(idesc), "n"(ACC ? 1 : 0)
                 : "memory");
}
__device__ __forceinline__ void f_mma_ts(uint32_t d, uint32_t a, uint32_t b_lo, uint32_t hi, uint32_t idesc, uint32_t acc) {
    asm volatile("{\n\t.reg .pred p;\n\t.reg .b64 db;\n\t"
                 "mov.b64 db, {%2, %3};\n\t"
                 "setp.ne.b32 p, %5, 0;\n\t"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %4, p;\n\t}" ::"r"(d),
                 "r"(a), "r"(b_lo), "r"(hi), "r"(idesc), "r"(acc)
                 : "memory");
}

// Entry k of a row of P is its label's: w (2^(S s + off) / |w| - 1), rounded once.
template <typename T>
__device__ __forceinline__ void label_entry(const uint32_t (&v)[32], uint32_t (&o)[16], int k, float s2, float off, float w) {
    asm volatile("");                        // (a branch, not 48 selections for every chunk)
    float z = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) z = i == k ? __uint_as_float(v[i]) : z;
    float e = ex2f(fmaf(z, s2, off)) - fabsf(w);
    e = w < 0.f ? -e : e;
    const uint32_t e16 = pack2<T>(e, e), sel = k & 1 ? 0x7610 : 0x3254;
#pragma unroll
    for (int i = 0; i < 16; ++i)
        o[i] = __byte_perm(o[i], e16, i == k >> 1 ? sel : 0x3210);
}

// The entries of P of 32 points (two to a word), those of points without a label zeroed; lane k looks at the
// label of point k.
__device__ __forceinline__ void drop_unlabelled(uint32_t (&o)[16], uint32_t label_addr) {
    int l;
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(l) : "r"(label_addr));
    const uint32_t none = __ballot_sync(0xffffffffu, l < 0);
#pragma unroll
    for (int k = 0; k < 16; ++k)
        o[k] &= ((none >> (2 * k)) & 1 ? 0u : 0xffffu) | ((none >> (2 * k + 1)) & 1 ? 0u : 0xffff0000u);
}

// COL: the points are the columns of P (dC), else the rows (dX). LO: P in two 16-bit parts, the second
// what the first's rounding left: with few table rows (128 at most) an entry is a large share of its
// row's sum, and its rounding, which a sum over many entries averages away, would be as large as the result's own.
// In TMEM the parts of 32 columns lie side by side where their S was.
template <typename T, int DN, bool COL, bool LO>
__global__ void __launch_bounds__(F_THREADS, 1)
    fused_grad_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB, const FParams p) {
    using Sh = FShape<DN, COL>;
    constexpr int S = Sh::kStages, RUN = fused_run<LO>();
    extern __shared__ uint8_t smem_raw[];
    __shared__ int abort_flag;
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t sbase = (raw + 1023u) & ~1023u;
    uint8_t *sgen = smem_raw + (sbase - raw);
    const uint32_t bar0 = sbase + Sh::kBarOff;
    auto B_FULL = [&](int s) { return bar0 + 8u * s; };
    auto B_EMPTY = [&](int s) { return bar0 + 8u * (S + s); };
    auto S_FULL = [&](int i) { return bar0 + 8u * (2 * S + i); };
    auto P_FULL = [&](int i) { return bar0 + 8u * (2 * S + 3 + i); };
    auto A_FULL = [&](int i) { return bar0 + 8u * (2 * S + 6 + i); };
    auto A_EMPTY = [&](int i) { return bar0 + 8u * (2 * S + 8 + i); };
    const uint32_t O_FULL = bar0 + 8u * (2 * S + 10), O_EMPTY = bar0 + 8u * (2 * S + 11);
    const uint32_t DRAIN = bar0 + 8u * (2 * S + 12);
    const uint32_t slot_addr = bar0 + 8u * Sh::kBars;
    const uint32_t asm_ = sbase, ring = sbase + Sh::kABufs * Sh::kTile;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    volatile int *abortp = &abort_flag;
    if (threadIdx.x == 0) {
        abort_flag = 0;
        for (int s = 0; s < S; ++s) {
            mbar_init(B_FULL(s), 1);
            mbar_init(B_EMPTY(s), 1);
        }
        for (int i = 0; i < F_SBUFS; ++i) {
            mbar_init(S_FULL(i), 1);
            mbar_init(P_FULL(i), F_GROUP);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(A_FULL(i), 1);
            mbar_init(A_EMPTY(i), 1);
        }
        mbar_init(O_FULL, 1);
        mbar_init(O_EMPTY, F_EPI_WARPS);
        mbar_init(DRAIN, 1);
        fence_mbar_init();
        tma_prefetch_desc(&tmA);
        tma_prefetch_desc(&tmB);
    }
    if (warp == 1) {
        tmem_alloc(slot_addr, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(sgen + (slot_addr - sbase));
    const int t0 = fused_begin(p.tiles, gridDim.x, blockIdx.x), t1 = fused_begin(p.tiles, gridDim.x, blockIdx.x + 1);

    if (warp == 0) {
        // ------------------------------------------------------------ requests
        const uint64_t pol = l2_policy_evict_last();
        int slot = 0, uses = 0, seg = 0;
        uint32_t ph = 1;
        bool ok = true;
        for (int t = t0; t < t1 && ok; ++seg) {
            const int r = t / p.ct, b = r / p.mt, m = r - b * p.mt;
            int j = t - r * p.ct;
            const int je = min(p.ct, j + (t1 - t)), ab = seg % Sh::kABufs;
            t += je - j;
            if (!mbar_wait_warp(A_EMPTY(ab), ((seg / Sh::kABufs) & 1) ^ 1u, abortp)) break;
            if (lane == 0) {
                mbar_arrive_expect_tx(A_FULL(ab), Sh::kTile);
#pragma unroll
                for (int c = 0; c < Sh::kChunks; ++c)
                    tma_load_3d(asm_ + ab * Sh::kTile + c * FR * 128, &tmA, A_FULL(ab), c * 64, m * FR, b, pol);
            }
            __syncwarp();
            for (; j < je; ++j) {
                if (!mbar_wait_warp(B_EMPTY(slot), ph, abortp)) { ok = false; break; }
                if (lane == 0 && !(p.withhold && uses == 0 && blockIdx.x == 0)) {
                    const uint32_t dst = ring + slot * Sh::kStage;
                    mbar_arrive_expect_tx(B_FULL(slot), Sh::kTile + (COL ? static_cast<uint32_t>(sizeof(PointTile)) : 0u));
#pragma unroll
                    for (int c = 0; c < Sh::kChunks; ++c)
                        tma_load_3d(dst + c * FR * 128, &tmB, B_FULL(slot), c * 64, j * FR, b, pol);
                    if (COL)
                        asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                                         dst + Sh::kTile),
                                     "l"(p.points + static_cast<int64_t>(b) * p.ct + j),
                                     "r"(static_cast<uint32_t>(sizeof(PointTile))), "r"(B_FULL(slot))
                                     : "memory");
                }
                __syncwarp();
                ++uses;
                if (++slot == S) { slot = 0; ph ^= 1u; }
            }
        }
        // the copies asked for land before shared memory goes away
        for (int s = max(0, seg - Sh::kABufs); s < seg; ++s)
            mbar_wait_warp(A_FULL(s % Sh::kABufs), (s / Sh::kABufs) & 1, nullptr);
        for (int s = max(0, uses - S); s < uses; ++s) mbar_wait_warp(B_FULL(s % S), (s / S) & 1, nullptr);
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMAs
        if (elect_one()) {
            constexpr uint32_t kDescHi = 1024u >> 4 | 1u << 14 | 2u << 29;   // 8-row groups 1 KB apart, version 1, 128-byte swizzle
            const int n = t1 - t0;
            int js = t0 % p.ct, jo = js;          // column tiles of the next S and of the next O
            int slot_s = 0, slot_o = 0, seg_s = 0, run_o = 0, in_run = 0;
            int bs = 0, bo = 0;                                     // their buffers
            uint32_t ph_s = 0, ph_o = 0, pho = 0;
            for (int i = -F_SBUFS; i < n; ++i) {
                if (i >= 0) {
                    // O of tile i
                    const bool first = in_run == 0, last = jo + 1 == p.ct || i + 1 == n || in_run + 1 == RUN;
                    if (!mbar_wait(P_FULL(bo), pho, abortp) || (first && !mbar_wait(O_EMPTY, (run_o & 1) ^ 1u, abortp))) break;
                    tc_fence_after();
                    // MN-major: 64-value blocks 16 KB apart (leading offset), 8-row groups 1 KB apart
                    const uint32_t bd = ((FR * 128) >> 4) << 16 | (ring + slot_o * Sh::kStage) >> 4, po = tmem + bo * FR;
                    f_mma_ts(tmem + F_OCOL, po, bd, kDescHi, p.idesc_o, first ? 0u : 1u);
#pragma unroll
                    for (int kk = 1; kk < FR / 16; ++kk)
                        f_mma_ts(tmem + F_OCOL, po + (kk >> 1) * 32 + (kk & 1) * 8, bd + kk * (2048 >> 4), kDescHi, p.idesc_o, 1u);
                    if (LO) {
#pragma unroll
                        for (int kk = 0; kk < FR / 16; ++kk)
                            f_mma_ts(tmem + F_OCOL, po + 16 + (kk >> 1) * 32 + (kk & 1) * 8, bd + kk * (2048 >> 4), kDescHi, p.idesc_o, 1u);
                    }
                    // (the group has read the tile's parameters before it gave P)
                    tc_commit(B_EMPTY(slot_o));
                    ++in_run;
                    if (last) {
                        tc_commit(O_FULL);
                        ++run_o;
                        in_run = 0;
                    }
                    if (++jo == p.ct) jo = 0;
                    if (++bo == F_SBUFS) { bo = 0; pho ^= 1u; }
                    if (i + F_SBUFS < n && !mbar_wait(B_EMPTY(slot_o), ph_o, abortp)) break;
                    if (++slot_o == S) { slot_o = 0; ph_o ^= 1u; }
                }
                if (i + F_SBUFS < n) {
                    // S of tile i + 3
                    const int ab = seg_s % Sh::kABufs;
                    const bool first = i + F_SBUFS == 0 || js == 0, last = js + 1 == p.ct || i + F_SBUFS + 1 == n;
                    if ((first && !mbar_wait(A_FULL(ab), (seg_s / Sh::kABufs) & 1, abortp)) || !mbar_wait(B_FULL(slot_s), ph_s, abortp)) break;
                    tc_fence_after();
                    const uint32_t al = 1u << 16 | (asm_ + ab * Sh::kTile) >> 4, bl = 1u << 16 | (ring + slot_s * Sh::kStage) >> 4;
                    f_mma_ss<false>(tmem + bs * FR, al, bl, kDescHi, p.idesc_s);
#pragma unroll
                    for (int kk = 1; kk < DN / 16; ++kk) {
                        const uint32_t o = ((kk >> 2) * (FR * 128) + (kk & 3) * 32) >> 4;
                        f_mma_ss<true>(tmem + bs * FR, al + o, bl + o, kDescHi, p.idesc_s);
                    }
                    tc_commit(S_FULL(bs));
                    if (last) {
                        tc_commit(A_EMPTY(ab));
                        ++seg_s;
                    }
                    if (++js == p.ct) js = 0;
                    if (++slot_s == S) { slot_s = 0; ph_s ^= 1u; }
                    if (++bs == F_SBUFS) bs = 0;
                }
            }
            // every MMA issued above completes before TMEM is released
            tc_commit(DRAIN);
            mbar_wait(DRAIN, 0, nullptr);
        }
        __syncwarp();
    } else {
        // ------------------------------------------------------------ exponentials, results
        const int q = warp & 3, grp = (warp - F_EPI0) / F_GROUP, row = q * 32 + lane;
        const uint32_t tl = tmem + (static_cast<uint32_t>(q * 32) << 16);
        const float s2 = p.scale * kLog2e;
        const uint64_t s22 = pair_f32(s2, s2);
        float inv = COL ? p_factor(p.wmax, p.pscale, true) : 0.f;
        int slot = 0, run = 0;
        uint32_t ph = 0, sph = 0, odd = 0;          // phases; parity of the tile
        int buf = 0;
        bool ok = true;
        for (int t = t0; t < t1 && ok; ++run) {
            const int r = t / p.ct, b = r / p.mt, m = r - b * p.mt;
            int j = t - r * p.ct;
            // the block's tiles of this row tile are [j0, j1), this run's [j, je)
            const int j0 = max(0, t0 - r * p.ct), j1 = min(p.ct, j + (t1 - t)), je = min(j1, j + RUN);
            const bool whole = j1 - j0 == p.ct, head = r * p.ct <= t0, begun = j > j0, more = je < j1;
            t += je - j;
            const int grow = m * FR + row;
            float off = 0.f, w = 0.f;
            int label = -1;
            if (!COL) {
                const PointRow pt = p.rows[static_cast<int64_t>(r) * FR + row];
                off = pt.off;
                w = pt.w;
                label = pt.label;
                inv = pt.factor;
            }
            const uint32_t sgn = w < 0.f ? 0x80008000u : 0u;
            const uint64_t off2 = pair_f32(off, off);
            for (; j < je; ++j, odd ^= 1u) {
                const uint32_t pp = ring + slot * Sh::kStage + Sh::kTile;
                const uint32_t b_full = B_FULL(slot), b_ph = ph;
                if (++slot == S) { slot = 0; ph ^= 1u; }
                const int sb = buf;
                const uint32_t s_ph = sph;
                if (++buf == F_SBUFS) { buf = 0; sph ^= 1u; }
                if (odd != static_cast<uint32_t>(grp)) continue;
                // (the MMAs have waited for the parameters' copy already; the wait here makes it visible)
                if (!mbar_wait_warp(S_FULL(sb), s_ph, abortp) || (COL && !mbar_wait_warp(b_full, b_ph, abortp))) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                // 32 columns at a time; rolled, since a longer body displaces the MMA warp's instructions
                const uint32_t ts = tl + sb * FR;
#pragma unroll 1
                for (int c = 0; c < 4; ++c) {
                    uint32_t v[32], o[16];
                    tmem_ld_32x32b_x32(ts + c * 32, v);
                    tmem_wait_ld(v);
                    const int col0 = j * FR + c * 32;           // B's row of the first column
                    // Points without a label are rows of zeros, which an infinite value of the table (a row masked
                    // so) turns into NaN. Such a table row has no finite S at all, so one column shows it. (The check: dC of 32768 x
                    // 8192 at d = 128 152.5 to 155.3 us.)
                    const bool fix = COL && __any_sync(0xffffffffu, !(fabsf(__uint_as_float(v[0])) < INFINITY));
                    if constexpr (LO) {
                        uint32_t rest[16];
#pragma unroll
                        for (int k = 0; k < 32; k += 2) {
                            float e[2];
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                float off_k = off, w_k = w;
                                bool mine = col0 + k + h == label;
                                if (COL) {
                                    const uint32_t at = pp + (c * 32 + k + h) * 4;
                                    int l;
                                    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(off_k) : "r"(at));
                                    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(w_k) : "r"(at + FR * 4));
                                    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(l) : "r"(at + FR * 8));
                                    mine = l == grow;
                                }
                                e[h] = ex2f(fmaf(__uint_as_float(v[k + h]), s2, off_k));
                                if (mine) e[h] -= fabsf(w_k);
                                if (w_k < 0.f) e[h] = -e[h];
                                if (!COL && col0 + k + h >= p.cols) e[h] = 0.f;
                            }
                            const uint32_t hi = pack2<T>(e[0], e[1]);
                            o[k >> 1] = hi;
                            rest[k >> 1] = pack2<T>(e[0] - unpack_lo<T>(hi), e[1] - unpack_hi<T>(hi));
                        }
                        if (COL && fix) drop_unlabelled(rest, pp + FR * 8 + (c * 32 + lane) * 4);
                        __syncwarp();
                        tmem_st_x16(ts + c * 32 + 16, rest);
                    } else if constexpr (!COL) {
#pragma unroll
                        for (int k = 0; k < 16; ++k) {
                            float x, y;
                            unpair_f32(fma2(pair_f32(__uint_as_float(v[2 * k]), __uint_as_float(v[2 * k + 1])), s22, off2), x, y);
                            o[k] = pack2<T>(ex2f(x), ex2f(y)) ^ sgn;
                        }
                        if (col0 + 32 > p.cols) {
                            // no rows of B: their zeros would meet 2^off, which may be infinite
                            asm volatile("");
#pragma unroll
                            for (int k = 0; k < 16; ++k) {
                                if (col0 + 2 * k >= p.cols) o[k] = 0;
                                else if (col0 + 2 * k + 1 >= p.cols) o[k] &= 0xffff;
                            }
                        }
                        if (label >= col0 && label < col0 + 32) label_entry<T>(v, o, label - col0, s2, off, w);
                    } else {
                        const uint32_t pc = pp + c * 128;
#pragma unroll
                        for (int k = 0; k < 16; k += 2) {
                            float f[4], x, y;
                            asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                                         : "=f"(f[0]), "=f"(f[1]), "=f"(f[2]), "=f"(f[3])
                                         : "r"(pc + k * 8));
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                const int at = 2 * (k + h);
                                unpair_f32(fma2(pair_f32(__uint_as_float(v[at]), __uint_as_float(v[at + 1])), s22,
                                                pair_f32(f[2 * h], f[2 * h + 1])),
                                           x, y);
                                o[k + h] = pack2<T>(ex2f(x), ex2f(y));
                            }
                        }
                        // lane k looks at point k of the 32: a negative weight, a label among the warp's rows?
                        float wk;
                        int lk;
                        asm volatile("ld.shared.f32 %0, [%1];" : "=f"(wk) : "r"(pc + FR * 4 + lane * 4));
                        asm volatile("ld.shared.b32 %0, [%1];" : "=r"(lk) : "r"(pc + FR * 8 + lane * 4));
                        const uint32_t neg = __ballot_sync(0xffffffffu, wk < 0.f);
                        if (neg) {
#pragma unroll
                            for (int k = 0; k < 16; ++k) o[k] ^= ((neg >> (2 * k)) & 1u) << 15 | ((neg >> (2 * k + 1)) & 1u) << 31;
                        }
                        const int from = grow - lane;
                        const uint32_t here = __ballot_sync(0xffffffffu, lk >= from && lk < from + 32);
                        if (here) {
                            uint32_t mine = 0;              // the points whose label is this thread's row
                            for (uint32_t h = here; h; h &= h - 1) {
                                const int k = __ffs(h) - 1;
                                if (__shfl_sync(0xffffffffu, lk, k) == grow) mine |= 1u << k;
                            }
                            while (__any_sync(0xffffffffu, mine != 0)) {
                                if (mine) {
                                    const uint32_t k = __ffs(mine) - 1;
                                    mine &= mine - 1;
                                    float off_k, w_k;
                                    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(off_k) : "r"(pc + k * 4));
                                    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(w_k) : "r"(pc + FR * 4 + k * 4));
                                    label_entry<T>(v, o, k, s2, off_k, w_k);
                                }
                                __syncwarp();
                            }
                        }
                    }
                    if (COL && fix) drop_unlabelled(o, pp + FR * 8 + (c * 32 + lane) * 4);
                    __syncwarp();       // lanes part at a label; the store wants the whole warp
                    tmem_st_x16(ts + c * 32, o);
                }
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(P_FULL(sb));
            }
            if (!ok || !mbar_wait_warp(O_FULL, run & 1, abortp)) break;
            tc_fence_after();
            const bool rin = grow < p.M;
            uint32_t v[DN / 64][32];
#pragma unroll
            for (int c = 0; c < DN / 64; ++c) tmem_ld_32x32b_x32(tl + F_OCOL + grp * (DN / 2) + c * 32, v[c]);
#pragma unroll
            for (int c = 0; c < DN / 64; ++c) tmem_wait_ld(v[c]);
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(O_EMPTY);
#pragma unroll
            for (int c = 0; c < DN / 64; ++c) {
                const int col = grp * (DN / 2) + c * 32;
                // the block's place for its first row tile, or for the one it is at (a thread's own part:
                // nobody else reads it before the kernel's end)
                float4 *part = reinterpret_cast<float4 *>(
                    p.parts + ((static_cast<int64_t>(blockIdx.x) * 2 + (head ? 0 : 1)) * FR + row) * DN + col);
                if (begun) {
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const float4 a = part[k];
                        v[c][k * 4] = __float_as_uint(__uint_as_float(v[c][k * 4]) + a.x);
                        v[c][k * 4 + 1] = __float_as_uint(__uint_as_float(v[c][k * 4 + 1]) + a.y);
                        v[c][k * 4 + 2] = __float_as_uint(__uint_as_float(v[c][k * 4 + 2]) + a.z);
                        v[c][k * 4 + 3] = __float_as_uint(__uint_as_float(v[c][k * 4 + 3]) + a.w);
                    }
                }
                if (more || !whole) {
                    // (rows and values beyond the result too: nothing reads them)
                    uint4 *dst = reinterpret_cast<uint4 *>(part);
#pragma unroll
                    for (int k = 0; k < 8; ++k) dst[k] = make_uint4(v[c][k * 4], v[c][k * 4 + 1], v[c][k * 4 + 2], v[c][k * 4 + 3]);
                    continue;
                }
                if (!rin || col >= p.d) continue;
                T *dst = static_cast<T *>(p.out) + (static_cast<int64_t>(b) * p.M + grow) * p.d + col;
                float f[32];
#pragma unroll
                for (int k = 0; k < 32; ++k) f[k] = !COL && label < 0 ? 0.f : __uint_as_float(v[c][k]) * inv;
                if (p.vec && col + 32 <= p.d) {
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        reinterpret_cast<uint4 *>(dst)[k] =
                            make_uint4(pack2<T>(f[k * 8], f[k * 8 + 1]), pack2<T>(f[k * 8 + 2], f[k * 8 + 3]),
                                       pack2<T>(f[k * 8 + 4], f[k * 8 + 5]), pack2<T>(f[k * 8 + 6], f[k * 8 + 7]));
                } else {
#pragma unroll
                    for (int k = 0; k < 32; ++k)
                        if (col + k < p.d) dst[k] = Cvt<T>::from_f(f[k]);
                }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem, 512);
}

// The block whose share holds a tile.
__host__ __device__ inline int fused_owner(int tiles, int blocks, int tile) {
    const int q = tiles / blocks, r = tiles % blocks;
    return tile < r * (q + 1) ? tile / (q + 1) : r + (tile - r * (q + 1)) / q;
}

// The row tiles that blocks share: their partials in block order. PARTS == 1: few partials to a row tile;
// each product block c > 0 stands for the row tile in which it begins, and the first that begins inside it
// (not at its start) answers. PARTS > 1: few row tiles, with up to all blocks' partials each, which PARTS
// threads take in runs. rows: the factors of dX's rows, null for dC.
template <typename T, int DN, int PARTS>
__global__ void __launch_bounds__(DN)
    fused_join_kernel(const float *__restrict__ parts, int tiles, int blocks, int M, int d, int mt, int ct,
                      const PointRow *__restrict__ rows, const unsigned int *__restrict__ wmax, float pscale,
                      T *__restrict__ out) {
    constexpr int ROWS = 4 / PARTS;      // rows of a row tile that a block takes
    __shared__ float4 sums[PARTS][DN / 4];
    const int unit = blockIdx.x / (FR / ROWS), part = PARTS == 1 ? 0 : threadIdx.x / (DN / 4);
    const int row = blockIdx.x % (FR / ROWS) * ROWS + (PARTS == 1 ? threadIdx.x / (DN / 4) : 0);
    const int col = threadIdx.x % (DN / 4) * 4;
    int r = unit;
    if (PARTS == 1) {
        const int at = fused_begin(tiles, blocks, 1 + unit), before = fused_begin(tiles, blocks, unit);
        r = at / ct;
        if (at == r * ct || (before > r * ct && unit > 0)) return;
    }
    const int b = r / mt, grow = (r - b * mt) * FR + row;
    const int c0 = fused_owner(tiles, blocks, r * ct), n = fused_owner(tiles, blocks, (r + 1) * ct - 1) - c0 + 1;
    if (n == 1 || (PARTS == 1 ? grow : grow - row % ROWS) >= M) return;
    const int which = fused_begin(tiles, blocks, c0) == r * ct ? 0 : 1;
    auto load = [&](int k) {
        return *reinterpret_cast<const float4 *>(parts + ((static_cast<int64_t>(c0 + k) * 2 + (k ? 0 : which)) * FR + row) * DN + col);
    };
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    auto add = [&](const float4 &x) {
        s.x += x.x;
        s.y += x.y;
        s.z += x.z;
        s.w += x.w;
    };
    const int k1 = n * (part + 1) / PARTS;
    for (int k = n * part / PARTS; k < k1; k += 8) {
        float4 x[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = k + i < k1 ? load(k + i) : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int i = 0; i < 8; ++i) add(x[i]);
    }
    if (PARTS > 1) {
        sums[part][col / 4] = s;
        __syncthreads();
        if (part) return;
#pragma unroll
        for (int i = 1; i < PARTS; ++i) add(sums[i][col / 4]);
    }
    const float inv = rows ? rows[static_cast<int64_t>(r) * FR + row].factor : p_factor(wmax, pscale, true);
    // (a row without a label is zero, whatever its zeros met in the table)
    if (rows && rows[static_cast<int64_t>(r) * FR + row].label < 0) s = make_float4(0.f, 0.f, 0.f, 0.f);
    const float f[4] = {s.x * inv, s.y * inv, s.z * inv, s.w * inv};
#pragma unroll
    for (int k = 0; k < 4; ++k)
        if (col + k < d) out[(static_cast<int64_t>(b) * M + grow) * d + col + k] = Cvt<T>::from_f(f[k]);
}

}  // namespace xe
}  // namespace km
