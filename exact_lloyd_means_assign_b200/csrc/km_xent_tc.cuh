// km_xent_tc.cuh -- the products of the cross entropy and its gradients on the 5th-generation
// tensor cores (tcgen05, TMEM, TMA), one SM pair per 256 x 256 tile (cta_group::2).
//
// One kernel forms D[m,n] = sum_k A(m,k) B(n,k) for the three products and differs in how the
// operands lie in memory and in what becomes of a tile:
//   kLse   A = X, B = C, reduction over d: the tile's logits become one (maximum, sum of
//          exponentials) pair per row and 128 columns
//   kProb  the same logits become P, in the points' type
//   kOut   dX = P C (reduction over the table piece) and dC = P^T X (reduction over the points)
// An operand whose reduction index is the contiguous one is staged K-major, the others MN-major,
// so P, X and C are read as they lie and nothing is transposed in memory.
//
// Bound by the tensor pipe: 8192 points x 32768 rows at d = 1024, bf16: the logits 339 us (1.62
// PFLOP/s, the pipe 94 % busy); with the gradients 1524 us: P at 81 % of the pipe, the products with it at
// 77 and 73, their 128 and 256 tiles leaving part of the last wave of 74 pairs empty. At d = 128
// the epilogue bounds the logits: 32768 x 8192 116 us, the special-function pipe some 60 % busy (moving a
// quarter of the exponentials to the FMA pipe did not help).
//
// Shared memory per CTA and stage of 64 reduction steps: 128 rows of A (16 KB) and of B;
// each CTA of a pair stages half of B, which the pair's MMAs share. The 512 TMEM columns hold two
// accumulators, so a tile's epilogue runs while the next tile is computed.
//
// Roles per CTA (12 warps): warp 0 requests the tiles; warp 1 of the leader issues the MMAs;
// warps 4-11 are the epilogue (TMEM lane quarter = warp % 4, column half = (warp - 4) / 4, one row
// per thread; sixteen warps with half the columns each were no faster). Waits are bounded like
// everywhere in the library: a role that gives up sets the CTA's abort flag, the producer waits for the
// copies it asked for, the issuer for its MMAs, the pair synchronises and frees TMEM. No TMA load uses
// multicast.
#pragma once

#include "km_assign_tc.cuh"
#include "km_xent.cuh"

namespace km {
namespace xe {

constexpr int TBM = 128;                 // rows per CTA, 256 per pair
constexpr int TBN = 256;                 // columns of a tile
constexpr int TKC = 64;                  // reduction steps per stage (128 bytes of 16-bit values)
constexpr int T_EPI0 = 4, T_EPI_WARPS = 8;
constexpr int T_THREADS = 32 * (T_EPI0 + T_EPI_WARPS);
constexpr uint32_t kOutBuf = 32 * 128;    // bytes of a P store
constexpr int T_GROUP = 8;               // row tiles that share their column tiles in L2

template <int MODE> struct TcShape {
    static constexpr uint32_t kA = TBM * 128u, kB = (TBN / 2) * 128u;
    static constexpr uint32_t kStage = kA + kB;
    // kProb: two 32-row x 64-column buffers per epilogue warp, from which P is stored by TMA
    static constexpr uint32_t kOutBytes = MODE == kProb ? T_EPI_WARPS * 2 * kOutBuf : 0;
    static constexpr int kStages = MODE == kProb ? 5 : 6;
    static constexpr uint32_t kOutOff = kStages * kStage;
    static constexpr uint32_t kBarOff = kOutOff + kOutBytes;
    static constexpr int kBars = 2 * kStages + 5;
    static constexpr uint32_t kTotal = kBarOff + kBars * 8 + 16 + 1024;
};

struct TcParams {
    int M, N;             // rows and columns of D
    int mt, nt;           // pair tiles
    int nb;               // batches
    int kchunks, kper;    // 64-wide chunks of the reduction, and per split
    int Kk;
    uint32_t idesc;
    int vec;              // rows of the output start on 16-byte boundaries
    int withhold;         // test only: the first pair never asks for its first stage
    FastDiv div_batch, div_split, div_group, div_last;   // items per batch, per split, per group of
                                                         // row tiles; row tiles of the last group
};

struct TcItem {
    int m, n, split, b;
};
// Work item t: batches, splits, groups of T_GROUP row tiles, columns, row tiles (fastest).
__device__ __forceinline__ TcItem tc_item(const TcParams &p, int t) {
    TcItem it;
    it.b = fd_div(p.div_batch, t);
    int r = t - it.b * static_cast<int>(p.div_batch.d);
    it.split = fd_div(p.div_split, r);
    r -= it.split * static_cast<int>(p.div_split.d);
    const int g = fd_div(p.div_group, r);
    r -= g * static_cast<int>(p.div_group.d);
    const int left = p.mt - g * T_GROUP;
    it.n = left >= T_GROUP ? r / T_GROUP : static_cast<int>(fd_div(p.div_last, r));
    it.m = g * T_GROUP + (r - it.n * min(T_GROUP, left));
    return it;
}

__device__ __forceinline__ float max3f(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
__device__ __forceinline__ float ex2f(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Descriptor words of an operand. K-major: 128-byte rows, the 8-row groups 1024 bytes apart, 16
// reduction steps = 32 bytes further. MN-major: blocks of 64 rows (128 bytes) x 64 reduction steps,
// the blocks 8192 bytes apart (leading offset), groups of 8 steps 1024 bytes apart, 16 reduction
// steps = 2048 bytes further.
template <bool MN> __device__ __forceinline__ uint32_t op_desc_lo(uint32_t saddr) {
    return ((MN ? 8192u >> 4 : 1u) << 16) | (saddr >> 4);
}
template <bool MN> __device__ __forceinline__ constexpr uint32_t op_step() { return MN ? 2048u >> 4 : 2u; }

template <typename T> __device__ __forceinline__ uint32_t pack2(float lo, float hi);
template <> __device__ __forceinline__ uint32_t pack2<__half>(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}
template <> __device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float lo, float hi) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}

__device__ __forceinline__ void ld_cols(uint32_t a, uint32_t (&v)[32]) { tmem_ld_32x32b_x32(a, v); }
__device__ __forceinline__ void ld_cols(uint32_t a, uint32_t (&v)[64]) { tmem_ld_32x32b_x64(a, v); }

template <typename T, int MODE, bool AMN, bool BMN>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(T_THREADS, 1)
    tc_product_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                      const __grid_constant__ CUtensorMap tmP, const TcParams p, const Epi ep) {
    using Sh = TcShape<MODE>;
    using namespace km::tc;
    constexpr int S = Sh::kStages;
    constexpr int HALF = TBN / 2;             // columns per epilogue warp
    extern __shared__ uint8_t smem_raw[];
    __shared__ int abort_flag;
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t sbase = (raw + 1023u) & ~1023u;
    uint8_t *sgen = smem_raw + (sbase - raw);
    const uint32_t bar0 = sbase + Sh::kBarOff;
    auto FULL = [&](int s) { return bar0 + 8u * s; };
    auto EMPTY = [&](int s) { return bar0 + 8u * (S + s); };
    auto ACC_FULL = [&](int i) { return bar0 + 8u * (2 * S + i); };
    auto ACC_EMPTY = [&](int i) { return bar0 + 8u * (2 * S + 2 + i); };
    const uint32_t DRAIN = bar0 + 8u * (2 * S + 4);
    const uint32_t slot = bar0 + 8u * Sh::kBars;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    const bool leader = rank == 0;
    volatile int *abortp = &abort_flag;
    if (threadIdx.x == 0) {
        abort_flag = 0;
        for (int s = 0; s < S; ++s) {
            mbar_init(FULL(s), 1);
            mbar_init(EMPTY(s), 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(ACC_FULL(i), 1);
            mbar_init(ACC_EMPTY(i), 2 * T_EPI_WARPS);   // (leader) the epilogue warps of both CTAs
        }
        mbar_init(DRAIN, 1);
        fence_mbar_init();
        tma_prefetch_desc(&tmA);
        tma_prefetch_desc(&tmB);
    }
    if (warp == 1) {
        tmem_alloc_pair(slot, TMEM_COLS);
        tmem_relinquish_pair();
    }
    tc_fence_before();
    cluster_sync_all();
    tc_fence_after();
    const uint32_t tmem_base = *reinterpret_cast<volatile uint32_t *>(sgen + (slot - sbase));
    const int total = p.mt * p.nt * ep.splits * p.nb;
    const int t0 = blockIdx.x >> 1, tstep = gridDim.x >> 1;

    if (warp == 0) {
        // ------------------------------------------------------------ producer
        const uint64_t pol = l2_policy_evict_last();
        int stage = 0;
        uint32_t ph = 0;
        long long uses = 0;
        bool ok = true;
        for (int t = t0; t < total && ok; t += tstep) {
            const TcItem it = tc_item(p, t);
            const int mrow = it.m * (2 * TBM) + static_cast<int>(rank) * TBM;
            const int nrow = it.n * TBN + static_cast<int>(rank) * (TBN / 2);
            const int kc1 = min(p.kchunks, (it.split + 1) * p.kper);
            for (int kc = it.split * p.kper; kc < kc1; ++kc) {
                if (!mbar_wait_warp(EMPTY(stage), ph ^ 1u, abortp)) { ok = false; break; }
                if (lane == 0 && !(p.withhold && uses == 0 && blockIdx.x < 2)) {
                    if (leader) mbar_arrive_expect_tx(FULL(stage), 2 * Sh::kStage);
                    const uint32_t a = sbase + stage * Sh::kStage, bsm = a + Sh::kA;
                    const uint32_t bar = map_to_rank(FULL(stage), 0);
                    if (AMN) {
#pragma unroll
                        for (int i = 0; i < TBM / 64; ++i)
                            tma_load_3d_pair(a + i * 8192, &tmA, bar, mrow + i * 64, kc * TKC, it.b, pol);
                    } else {
                        tma_load_3d_pair(a, &tmA, bar, kc * TKC, mrow, it.b, pol);
                    }
                    if (BMN) {
#pragma unroll
                        for (int i = 0; i < TBN / 128; ++i)
                            tma_load_3d_pair(bsm + i * 8192, &tmB, bar, nrow + i * 64, kc * TKC, it.b, pol);
                    } else {
                        tma_load_3d_pair(bsm, &tmB, bar, kc * TKC, nrow, it.b, pol);
                    }
                }
                __syncwarp();
                ++uses;
                if (++stage == S) { stage = 0; ph ^= 1u; }
            }
        }
        if (!ok && leader && lane == 0) {
            // the copies asked for land before shared memory goes away
            for (int s = 0; s < S; ++s) {
                const long long n = uses > s ? (uses - 1 - s) / S + 1 : 0;
                if (n) mbar_wait(FULL(s), static_cast<uint32_t>((n - 1) & 1), nullptr);
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMA issuer
        if (leader) {
            const bool issuer = elect_one();
            int stage = 0, buf = 0;
            uint32_t ph = 0, aph = 0;
            bool ok = true;
            for (int t = t0; t < total && ok; t += tstep) {
                const TcItem it = tc_item(p, t);
                const int kc0 = it.split * p.kper, kc1 = min(p.kchunks, kc0 + p.kper);
                if (!mbar_wait_warp(ACC_EMPTY(buf), aph ^ 1u, abortp)) break;
                tc_fence_after();
                const uint32_t dcol = tmem_base + buf * ACC_STRIDE;
                for (int kc = kc0; kc < kc1; ++kc) {
                    if (!mbar_wait_warp(FULL(stage), ph, abortp)) { ok = false; break; }
                    tc_fence_after();
                    if (issuer) {
                        const uint32_t a_lo = op_desc_lo<AMN>(sbase + stage * Sh::kStage);
                        const uint32_t b_lo = op_desc_lo<BMN>(sbase + stage * Sh::kStage + Sh::kA);
                        const int nk = min(4, (p.Kk - kc * TKC + 15) / 16);
                        for (int kk = 0; kk < nk; ++kk)
                            tc_mma_pair(dcol, a_lo + kk * op_step<AMN>(), DESC_HI_SW128, b_lo + kk * op_step<BMN>(),
                                        DESC_HI_SW128, p.idesc, (kc > kc0 || kk) ? 1u : 0u);
                        tc_commit_pair_both(EMPTY(stage));
                        if (kc + 1 == kc1) tc_commit_pair_both(ACC_FULL(buf));
                    }
                    __syncwarp();
                    if (++stage == S) { stage = 0; ph ^= 1u; }
                }
                buf ^= 1;
                if (buf == 0) aph ^= 1u;
            }
            // every MMA issued above completes before TMEM is released
            if (issuer) tc_commit_pair_self(DRAIN);
            __syncwarp();
            mbar_wait_warp(DRAIN, 0, nullptr);
        }
        __syncwarp();
    } else if (warp >= T_EPI0) {
        // ------------------------------------------------------------ epilogue
        const int q = warp & 3, half = (warp - T_EPI0) >> 2;
        const uint32_t empty0 = map_to_rank(ACC_EMPTY(0), 0), empty1 = map_to_rank(ACC_EMPTY(1), 0);
        const uint32_t tl = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + half * HALF;
        // The products are formed with |scale| (a negative scale negates the points in the MMA).
        const float sc = fabsf(ep.scale), s2 = sc * kLog2e;
        const uint64_t s22 = pair_f32(s2, s2);
        // kLse: a maximum below this (every logit so far masked by an infinity or by the type's lowest value) would
        // overflow as the sums' base; their terms are 0 then.
        const float floor_ = -3e38f / fmaxf(s2, 1.f);
        const float fac = MODE == kProb ? p_factor(ep.wmax, ep.pscale, false) : 1.f;
        const int max_exp = kShifts<T> && MODE != kLse ? exponent_of(ep.wmax[kMaxW]) : 0;
        // (of dC too: its points' common shift)
        const float inv = MODE == kOut && ep.splits == 1
            ? p_factor(ep.wmax, ep.pscale, true) * (kShifts<T> && !ep.rows ? pow2f(-point_shift(ep.wmax)) : 1.f) : 1.f;
        const uint32_t obuf = sbase + Sh::kOutOff + (warp - T_EPI0) * 2 * kOutBuf;
        int buf = 0, ob = 0;
        uint32_t aph = 0;
        // The row's label, weight and lse, read one tile ahead: their latency would otherwise stand
        // before every tile's first exponential.
        int id_n = -1;
        float w_n = 0.f, lse_n = 0.f;
        TcItem next = {};
        auto read_row = [&](int t) {
            if (t >= total) return;
            next = tc_item(p, t);
            if (MODE == kOut && !(kShifts<T> && ep.rows)) return;
            const int row = next.m * (2 * TBM) + static_cast<int>(rank) * TBM + q * 32 + lane;
            id_n = -1;
            if (row < p.M) {
                const int64_t br = static_cast<int64_t>(next.b) * p.M + row;
                if (MODE != kOut) id_n = __ldg(ep.ids + br);
                if (MODE != kLse) w_n = __ldg(ep.w + br);
                if (MODE == kProb) lse_n = __ldg(ep.lse + br);
            }
        };
        read_row(t0);
        for (int t = t0; t < total; t += tstep) {
            const TcItem it = next;
            const int row0 = it.m * (2 * TBM) + static_cast<int>(rank) * TBM + q * 32, row = row0 + lane;
            const int c0 = it.n * TBN + half * HALF;
            const bool rin = row < p.M;
            const int64_t br = static_cast<int64_t>(it.b) * p.M + row;
            const float back = kShifts<T> && MODE == kOut && ep.rows ? inv * pow2f(-row_shift(max_exp, w_n)) : inv;
            int label = -1;
            // kProb: P = sign (2^(z log2e + off) - |w| [label]) with off = log2 |w| - lse log2e
            float aw = 0.f, off = 0.f;
            uint32_t sign = 0, keep = 0;
            if (MODE != kOut) {
                const bool has = id_n >= 0 && id_n < ep.K;
                label = has ? id_n - ep.k0 : -1;
                if (MODE == kProb) {
                    const float w = has ? w_n * fac * (kShifts<T> ? pow2f(row_shift(max_exp, w_n)) : 1.f) : 0.f;
                    aw = fabsf(w);
                    off = __log2f(aw) - lse_n * kLog2e;
                    sign = w < 0.f ? 0x80008000u : 0u;
                    keep = has ? ~0u : 0u;
                }
            }
            read_row(t + tstep);
            if (!mbar_wait_warp(ACC_FULL(buf), aph, abortp)) break;
            tc_fence_after();
            float m = 0.f;
            uint64_t s4[4] = {0, 0, 0, 0};
            // columns in chunks of 32, 64 for the loss (fewer corrections of the sums by a new maximum: 32768 x
            // 8192 at d = 128 122 to 116 us), the next chunk's load in flight while one is worked on
            constexpr int CH = MODE == kLse ? 64 : 32;
            uint32_t v2[2][CH];
            ld_cols(tl + buf * ACC_STRIDE, v2[0]);
#pragma unroll
            for (int ch = 0; ch < HALF / CH; ++ch) {
                uint32_t(&v)[CH] = v2[ch & 1];
                __syncwarp();        // lanes part in a chunk's work; these instructions want the whole warp
                tmem_wait_ld(v);
                if (ch + 1 < HALF / CH) {
                    ld_cols(tl + buf * ACC_STRIDE + (ch + 1) * CH, v2[(ch + 1) & 1]);
                } else {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive_cluster_relaxed(buf ? empty1 : empty0);
                }
                const int col = c0 + ch * CH;
                if (MODE == kLse) {
                    if (col < p.N) {
                        if (col + CH > p.N) {
                            asm volatile("");      // a branch: this is the table's last tile only
#pragma unroll
                            for (int i = 0; i < CH; ++i)
                                if (col + i >= p.N) v[i] = 0xff800000u;      // -inf
                        }
                        float cm = __uint_as_float(v[0]), cm2 = __uint_as_float(v[1]);
#pragma unroll
                        for (int i = 2; i < CH - 2; i += 4) {
                            cm = max3f(cm, __uint_as_float(v[i]), __uint_as_float(v[i + 1]));
                            cm2 = max3f(cm2, __uint_as_float(v[i + 2]), __uint_as_float(v[i + 3]));
                        }
                        cm = max3f(max3f(cm, __uint_as_float(v[CH - 2]), __uint_as_float(v[CH - 1])), cm2, cm);
                        const float nm = ch ? fmaxf(m, cm) : cm;
                        if (label >= col && label < col + CH) {
                            asm volatile("");
                            float zt = 0.f;
#pragma unroll
                            for (int i = 0; i < CH; ++i)
                                if (col + i == label) zt = __uint_as_float(v[i]) * sc;
                            ep.zt[br] = zt;
                        }
                        if (ch) {
                            const float corr = ex2f((fmaxf(m, floor_) - fmaxf(nm, floor_)) * s2);
                            const uint64_t c2 = pair_f32(corr, corr);
#pragma unroll
                            for (int i = 0; i < 4; ++i) s4[i] = fma2(s4[i], c2, 0ull);
                        }
                        m = nm;
                        // the product rounded down where its rounding could pass for a large exponent
                        const float top = fmaxf(nm, floor_), d = fabsf(top) * s2 > 0x1p20f ? __fmul_rd(-top, s2) : -top * s2;
                        const uint64_t d2 = pair_f32(d, d);
#pragma unroll
                        for (int i = 0; i < CH; i += 2) {
                            float a, b;
                            unpair_f32(fma2(pair_f32(__uint_as_float(v[i]), __uint_as_float(v[i + 1])), s22, d2), a, b);
                            s4[(i >> 1) & 3] = add2(s4[(i >> 1) & 3], pair_f32(ex2f(a), ex2f(b)));
                        }
                    }
                } else if (MODE == kProb) {
                    const uint64_t o2 = pair_f32(off, off);
                    uint32_t o[16];
#pragma unroll
                    for (int i = 0; i < 32; i += 2) {
                        float a, b;
                        unpair_f32(fma2(pair_f32(__uint_as_float(v[i]), __uint_as_float(v[i + 1])), s22, o2), a, b);
                        o[i >> 1] = (pack2<T>(ex2f(a), ex2f(b)) ^ sign) & keep;
                    }
                    if (label >= col && label < col + 32) {
                        asm volatile("");
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            if (col + i == label) {
                                const float e = ex2f(fmaf(__uint_as_float(v[i]), s2, off)) - aw;
                                const uint32_t e16 = (pack2<T>(e, e) ^ sign) & keep;
                                o[i >> 1] = i & 1 ? __byte_perm(o[i >> 1], e16, 0x7610) : __byte_perm(o[i >> 1], e16, 0x3254);
                            }
                    }
                    // 64 columns (two chunks) per buffer, in the 128-byte swizzle of the store's map
                    const uint32_t dst = obuf + ob * kOutBuf + lane * 128;
                    if ((ch & 1) == 0) {
                        // the buffer's store before last has been read out
                        if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
                        __syncwarp();
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(
                                         dst + ((((ch & 1) * 4 + i) ^ (lane & 7)) * 16)),
                                     "r"(o[i * 4]), "r"(o[i * 4 + 1]), "r"(o[i * 4 + 2]), "r"(o[i * 4 + 3])
                                     : "memory");
                    if (ch & 1) {
                        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                        __syncwarp();
                        // columns behind the piece's last are inside the row's padding or cut off
                        if (lane == 0) {
                            if (row0 < p.M && col - 32 < p.N)
                                asm volatile(
                                    "cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
                                        &tmP),
                                    "r"(obuf + ob * kOutBuf), "r"(col - 32), "r"(row0), "r"(it.b)
                                    : "memory");
                            asm volatile("cp.async.bulk.commit_group;" ::: "memory");
                        }
                        ob ^= 1;
                    }
                } else {
                    if (!rin || col >= p.N) continue;
                    const int64_t at = br * p.N + col;
                    if (ep.splits > 1) {
                        float *dst = ep.out32 + static_cast<int64_t>(it.split) * p.nb * p.M * p.N + at;
                        if (p.vec && col + 32 <= p.N) {
#pragma unroll
                            for (int i = 0; i < 8; ++i)
                                reinterpret_cast<uint4 *>(dst)[i] = make_uint4(v[i * 4], v[i * 4 + 1], v[i * 4 + 2], v[i * 4 + 3]);
                        } else {
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                if (col + i < p.N) dst[i] = __uint_as_float(v[i]);
                        }
                    } else {
                        float f[32];
                        const bool whole = p.vec && col + 32 <= p.N;
#pragma unroll
                        for (int i = 0; i < 32; ++i) f[i] = __uint_as_float(v[i]) * back;
                        if (ep.acc) {
                            if (whole) {
#pragma unroll
                                for (int i = 0; i < 8; ++i) {
                                    const float4 a = reinterpret_cast<const float4 *>(ep.acc + at)[i];
                                    f[i * 4] += a.x;
                                    f[i * 4 + 1] += a.y;
                                    f[i * 4 + 2] += a.z;
                                    f[i * 4 + 3] += a.w;
                                }
                            } else {
#pragma unroll
                                for (int i = 0; i < 32; ++i)
                                    if (col + i < p.N) f[i] += ep.acc[at + i];
                            }
                        }
                        if (ep.out32) {
                            if (whole) {
#pragma unroll
                                for (int i = 0; i < 8; ++i)
                                    reinterpret_cast<float4 *>(ep.out32 + at)[i] =
                                        make_float4(f[i * 4], f[i * 4 + 1], f[i * 4 + 2], f[i * 4 + 3]);
                            } else {
#pragma unroll
                                for (int i = 0; i < 32; ++i)
                                    if (col + i < p.N) ep.out32[at + i] = f[i];
                            }
                        } else {
                            T *dst = static_cast<T *>(ep.outT) + at;
                            if (whole) {
#pragma unroll
                                for (int i = 0; i < 4; ++i)
                                    reinterpret_cast<uint4 *>(dst)[i] =
                                        make_uint4(pack2<T>(f[i * 8], f[i * 8 + 1]), pack2<T>(f[i * 8 + 2], f[i * 8 + 3]),
                                                   pack2<T>(f[i * 8 + 4], f[i * 8 + 5]), pack2<T>(f[i * 8 + 6], f[i * 8 + 7]));
                            } else {
#pragma unroll
                                for (int i = 0; i < 32; ++i)
                                    if (col + i < p.N) dst[i] = Cvt<T>::from_f(f[i]);
                            }
                        }
                    }
                }
            }
            if (MODE == kLse && rin && c0 < p.N) {
                float a, b;
                unpair_f32(add2(add2(s4[0], s4[1]), add2(s4[2], s4[3])), a, b);
                const int64_t tiles = (p.N + ST - 1) / ST;
                ep.pairs[(static_cast<int64_t>(it.b) * tiles + it.n * 2 + half) * p.M + row] = make_float2(m * sc, a + b);
            }
            buf ^= 1;
            if (buf == 0) aph ^= 1u;
        }
        if (MODE == kProb) {      // every store has been read out of shared memory and written
            if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
            __syncwarp();
        }
    }
    // both CTAs are done with each other's barriers and the leader's MMAs have drained
    tc_fence_before();
    __syncthreads();
    cluster_sync_all();
    tc_fence_after();
    if (warp == 1) tmem_dealloc_pair(tmem_base, TMEM_COLS);
}

}  // namespace xe
}  // namespace km
