// km_matvec4_tc.cuh -- products with 4-bit codebook weights on tcgen05 (the weights decoded into
// tensor memory).
//
// A tile is 128 rows of weights, one per TMEM lane, and a step 256 (or 128) codes of each. A thread
// decodes a part of its own row: a byte of codes indexes a table of 256 value pairs kept for every
// row in shared memory, so the 32 lanes of a warp always read 32 different banks, and the pairs go
// straight to the row's TMEM lane (column c of a step holds codes 2c and 2c + 1), which is the
// layout of a tensor-core row operand. Nothing is decoded twice whatever the number of tokens (up
// to 32 per pass), and the only shared-memory traffic is the codes, one word per pair and the table
// itself. (The mma.sync form looks a pair up for every eight tokens.)
//
// Two half-tables of 64 rows x 256 entries (64 KB each) start on multiples of 64 KB of the shared
// window, so that one byte permutation of (codes, row) is the address of a pair. The ring of
// steps takes what is left on either side: codes by TMA, swizzled so that the rows a warp reads at
// once lie in different banks, and the tokens' values. Steps are long because every hand-over
// between the roles costs hundreds of cycles whatever it hands over.
//
// What it measured (16 tokens x 8192 x 8192 bf16, a scale per 64 weights, GPU time): 21.6 us, where the
// mma.sync form took 32; a step of 256 codes takes about 1040 cycles, of which the lookups are 640 and
// the codes' bytes at full memory rate 700; some 6 us of the launch pass before the first step (codebooks read,
// tables built) and after the last (the cluster's barriers). A single token is served by the mma.sync
// form: as fast on large weights (48 us here, 47 there for 32768 x 8192) and quicker to start on small
// ones (11 us here, 5.7 there for 4096 x 4096).
//
// Roles (22 warps): 0-15 decode (lane quarter = warp % 4, quarter of the step's codes = warp / 4);
// 16-19 read the accumulators, multiply by the group scales and keep the sums in fp32 registers;
// 20 requests; 21 issues the MMAs. Blocks are persistent over tiles; where tiles are few, a cluster
// shares one, each block a part of the reduction, and the first block adds the parts in order.
#pragma once

#include "km_common.cuh"

namespace km {
namespace mv4 {

constexpr int kTcDecode = 16;
constexpr int kTcEpi = 16, kTcProd = 20, kTcMma = 21;
constexpr int kTcThreads = 32 * 22;
constexpr int kTcRows = 128;
constexpr uint32_t kHalfTab = 65536;
constexpr uint32_t kValuePitch = 48;               // bytes of a row's 16 codebook values, padded
constexpr uint32_t kValueBytes = kTcRows * kValuePitch;
constexpr uint32_t kTcEnd = 4 * kHalfTab - 29696;  // end of the used window: 64 KB, tables, 35 KB

// NTOK tokens per pass; SC: 0 no scales, 1, 2, 3 scale groups of multiples of 128, 64, 32 codes.
template <int NTOK, int SC> struct TcMv {
    static constexpr int kStep = NTOK == 32 ? 128 : 256;           // codes of a row per step
    static constexpr uint32_t kCodeBytes = kTcRows * kStep / 2;
    static constexpr uint32_t kXChunk = NTOK * 128;                // 64 positions of every token
    static constexpr uint32_t kXBytes = kStep / 64 * kXChunk;
    static constexpr uint32_t kStage = kCodeBytes + kXBytes;
    static constexpr int kSub = SC ? kStep / (256 >> SC) : 1;      // accumulators per step
    // Without scales a sum ends after kMaxChain products all the same: their additions truncate.
    static constexpr int kRun = SC ? 1 : kMaxChain / (kStep / 16);  // steps to a set of accumulators
    static constexpr uint32_t kAcc = kSub * NTOK;                 // their TMEM columns
    static constexpr int kDBufs = 2 * kAcc + kStep > 512 ? 1 : 2;  // sets of accumulators
    static constexpr uint32_t kACol = kDBufs * kAcc;               // decoded steps behind them
    static constexpr int kABufs = (512 - kACol) / (kStep / 2) < 4 ? (512 - kACol) / (kStep / 2) : 4;
    // the window below the tables (1 KB reserved by the system, up to 1 KB of barriers) and above
    static constexpr int kBelow = (kHalfTab - 2048) / kStage;
    static constexpr int kAbove = (kTcEnd - 3 * kHalfTab - kValueBytes) / kStage;
    static constexpr int kStages = kBelow + kAbove;
    static_assert(kABufs >= 2 && kStages >= 3, "buffers");
};

struct TcMvParams {
    const float *C, *scales;
    int64_t R, M;
    int N, K, ngroups;
    int rtiles, mtiles, steps;     // tiles of 128 rows, of NTOK tokens; steps of a row
    int split, sper;               // blocks that share a tile, steps of each
    int x3d, svec;                 // tokens by one copy per step; rows of scales on 16-byte boundaries
    FastDiv cpg;                   // 32-code chunks per scale group
    uint32_t idesc;
    int withhold;                  // test only: the first block never asks for its first step
};

__device__ __forceinline__ uint4 lds128(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ void sts32(uint32_t a, uint32_t v) {
    asm volatile("st.shared.b32 [%0], %1;" ::"r"(a), "r"(v) : "memory");
}
__device__ __forceinline__ void cluster_barrier() {
    __syncwarp();          // .aligned: the whole warp at once
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

template <typename T, int NTOK, int SC>
__global__ void __launch_bounds__(kTcThreads, 1)
    matvec4_tc_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX,
                      const TcMvParams p, T *__restrict__ y) {
    using L = TcMv<NTOK, SC>;
    constexpr int S = L::kStages, NA = L::kABufs, ND = L::kDBufs, STEP = L::kStep;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ __align__(8) uint64_t bars[2 * S + 2 * NA + 5];
    __shared__ uint32_t tmem_slot;
    __shared__ int abort_flag;
    const uint32_t base = smem_u32(smem);
    // (in a cluster every block's shared memory has a window of its own, 16 MB from the next)
    const uint32_t window = base & ~(4 * kHalfTab - 1);
    const uint32_t low = (base + 1023) & ~1023u, tab = window + kHalfTab, above = window + 3 * kHalfTab;
    // (uniform; never: the dynamic window starts within the first 2 KB and reaches kTcEnd)
    uint32_t dynamic;
    asm("mov.u32 %0, %%dynamic_smem_size;" : "=r"(dynamic));
    if (low + L::kBelow * L::kStage > tab || base + dynamic < window + kTcEnd) {
        if (threadIdx.x == 0) record_dev_error(kDevErrTimeout);
        return;
    }
    const uint32_t values = above + L::kAbove * L::kStage;
    auto stage_addr = [&](int s) {
        return s < L::kBelow ? low + s * L::kStage : above + (s - L::kBelow) * L::kStage;
    };
    const uint32_t bar0 = smem_u32(bars);
    auto FULL = [&](int s) { return bar0 + 8u * s; };
    auto EMPTY = [&](int s) { return bar0 + 8u * (S + s); };
    auto A_FULL = [&](int i) { return bar0 + 8u * (2 * S + i); };
    auto A_EMPTY = [&](int i) { return bar0 + 8u * (2 * S + NA + i); };
    auto D_FULL = [&](int i) { return bar0 + 8u * (2 * S + 2 * NA + i); };
    auto D_EMPTY = [&](int i) { return bar0 + 8u * (2 * S + 2 * NA + 2 + i); };
    const uint32_t DRAIN = bar0 + 8u * (2 * S + 2 * NA + 4);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    volatile int *abortp = &abort_flag;
    if (threadIdx.x == 0) {
        abort_flag = 0;
        for (int s = 0; s < S; ++s) {
            mbar_init(FULL(s), 1);
            mbar_init(EMPTY(s), kTcDecode + 1);      // the decoding warps and the MMAs that read the tokens
        }
        for (int i = 0; i < NA; ++i) {
            mbar_init(A_FULL(i), kTcDecode);
            mbar_init(A_EMPTY(i), 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(D_FULL(i), 1);
            mbar_init(D_EMPTY(i), 4);
        }
        mbar_init(DRAIN, 1);
        fence_mbar_init();
    }
    if (warp == kTcMma) {
        tmem_alloc(smem_u32(&tmem_slot), 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(&tmem_slot);
    const int rank = static_cast<int>(blockIdx.x) % p.split, first = static_cast<int>(blockIdx.x) / p.split;
    const int stride = static_cast<int>(gridDim.x) / p.split, items = p.rtiles * p.mtiles;
    const int st0 = rank * p.sper, st1 = min(p.steps, st0 + p.sper);     // this block's steps of every item
    const int nst = max(0, st1 - st0);

    if (warp < kTcDecode) {
        // ------------------------------------------------------------ decode
        constexpr int CODES = STEP / 4, COLS = CODES / 2;    // of a row, per warp and step
        const int q = warp & 3, part = warp >> 2, row = q * 32 + lane;
        const int dt = threadIdx.x;                       // 0 .. 511
        // codebook values dt, dt + 512, ... of an item's 128 x 16 (0 beyond the codebook or the rows)
        float cv[4];
        auto read_values = [&](int item) {
            const int64_t r0 = static_cast<int64_t>(item % p.rtiles) * kTcRows;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int e = i * 512 + dt;
                const int64_t r = r0 + (e >> 4);
                cv[i] = item < items && r < p.R && (e & 15) < p.K ? __ldg(p.C + r * p.K + (e & 15)) : 0.f;
            }
        };
        read_values(first);
        const uint32_t rowbits = tab + (row >> 6) * kHalfTab + (row & 63) * 4;   // byte 0 the row, 2-3 the table
        // 16-byte unit u of row r lies at u ^ (r % 8) (rows of 128 bytes) or u ^ (r / 2 % 4) (64 bytes)
        const uint32_t code_row = row * (STEP / 2), swz = (STEP == 256 ? row & 7 : (row >> 1) & 3) * 16;
        const uint32_t at = tmem + (static_cast<uint32_t>(q * 32) << 16) + L::kACol + part * COLS;
        int slot = 0, ab = 0;
        uint32_t ph = 0, aph = 1;
        bool ok = true;
        for (int item = first; item < items; item += stride) {
            // everybody is done with the previous table; a warp that gave up takes all with it
            __syncwarp();
            if (named_barrier_or(1, 32 * kTcDecode, !ok)) break;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int e = i * 512 + dt;
                asm volatile("st.shared.b16 [%0], %1;" ::"r"(values + (e >> 4) * kValuePitch + (e & 15) * 2),
                             "h"(static_cast<uint16_t>(bits16(Cvt<T>::from_f(cv[i]))))
                             : "memory");
            }
            named_barrier_sync(1, 32 * kTcDecode);
            read_values(item + stride);
            {
                // this thread: row dt % 128, high codes 4 (dt / 128) .. + 3
                const int tr = dt & 127;
                const uint32_t va = values + tr * kValuePitch;
                const uint4 c0 = lds128(va), c1 = lds128(va + 16);
                const uint32_t c[8] = {c0.x, c0.y, c0.z, c0.w, c1.x, c1.y, c1.z, c1.w};
                const uint32_t dst = tab + (tr >> 6) * kHalfTab + (tr & 63) * 4;
#pragma unroll 1      // (unrolled, the code alone takes longer to fetch than to run)
                for (int hh = 0; hh < 4; ++hh) {
                    const int hi = (dt >> 7) * 4 + hh;
                    uint32_t w;
                    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(w) : "r"(va + (hi & ~1) * 2) : "memory");
                    const uint32_t vh = hi & 1 ? w & 0xffff0000u : w << 16;
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        sts32(dst + (hi * 16 + 2 * k) * 256, __byte_perm(c[k], vh, 0x7610));
                        sts32(dst + (hi * 16 + 2 * k + 1) * 256, __byte_perm(c[k], vh, 0x7632));
                    }
                }
            }
            named_barrier_sync(1, 32 * kTcDecode);
#pragma unroll 1
            for (int s = 0; s < nst; ++s) {
                if (!mbar_ready(FULL(slot), ph, abortp)) { ok = false; break; }
                uint32_t cw[CODES / 8];
                const uint32_t src = stage_addr(slot) + code_row;
#pragma unroll
                for (int i = 0; i < CODES / 32; ++i) {
                    const uint4 w = lds128(src + (((part * (CODES / 32) + i) * 16) ^ swz));
                    cw[i * 4] = w.x, cw[i * 4 + 1] = w.y, cw[i * 4 + 2] = w.z, cw[i * 4 + 3] = w.w;
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(EMPTY(slot));
                uint32_t v[COLS];
#pragma unroll
                for (int i = 0; i < CODES / 8; ++i)
#pragma unroll
                    for (int b = 0; b < 4; ++b) v[i * 4 + b] = lds_tab<0>(__byte_perm(cw[i], rowbits, 0x7604 | b << 4));
                const int k0 = (st0 + s) * STEP + part * CODES;
                if (k0 + CODES > p.N) {
                    // codes behind the row's end are no weights (a codebook value may be infinite)
#pragma unroll
                    for (int i = 0; i < COLS; ++i) {
                        if (k0 + 2 * i >= p.N) v[i] = 0;
                        else if (k0 + 2 * i + 1 >= p.N) v[i] &= 0xffff;
                    }
                }
                if (!mbar_ready(A_EMPTY(ab), aph, abortp)) { ok = false; break; }
                tc_fence_after();
                if constexpr (COLS == 32) tmem_st_x32(at + ab * (STEP / 2), v);
                else tmem_st_x16(at + ab * (STEP / 2), v);
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(A_FULL(ab));
                if (++slot == S) { slot = 0; ph ^= 1u; }
                if (++ab == NA) { ab = 0; aph ^= 1u; }
            }
        }
    } else if (warp < kTcEpi + 4) {
        // ------------------------------------------------------------ accumulators, scales, sums
        const int q = warp & 3, row = q * 32 + lane;
        const uint32_t tl = tmem + (static_cast<uint32_t>(q * 32) << 16);
        int db = 0;
        uint32_t dph = 0;
        bool ok = true;
        const int chunks = (p.N + 31) / 32;
        for (int item = first; item < items && ok; item += stride) {
            const int64_t r0 = static_cast<int64_t>(item % p.rtiles) * kTcRows;
            const int64_t m0 = static_cast<int64_t>(item / p.rtiles) * NTOK;
            float tot[NTOK];
#pragma unroll
            for (int i = 0; i < NTOK; ++i) tot[i] = 0.f;
            // The row's scales, four groups at a time and four ahead: a lane's row is its own line,
            // so the load pipe is busy 32 cycles per load however little it brings.
            const float *srow = SC ? p.scales + min(r0 + row, p.R - 1) * p.ngroups : nullptr;
            float4 cur = {}, nxt = {};
            int unit = 0;
            auto load4 = [&](int u) {
                float4 f = {};
                const int g = u * 4;
                if (p.svec) {
                    if (g < p.ngroups) f = __ldg(reinterpret_cast<const float4 *>(srow + g));
                } else {
                    if (g < p.ngroups) f.x = __ldg(srow + g);
                    if (g + 1 < p.ngroups) f.y = __ldg(srow + g + 1);
                    if (g + 2 < p.ngroups) f.z = __ldg(srow + g + 2);
                    if (g + 3 < p.ngroups) f.w = __ldg(srow + g + 3);
                }
                return f;
            };
            if (SC && nst) {
                unit = static_cast<int>(fd_div(p.cpg, st0 * (STEP / 32))) >> 2;
                cur = load4(unit);
                nxt = load4(unit + 1);
                // and the next tile's into L2
                const int64_t r1 = static_cast<int64_t>((item + stride) % p.rtiles) * kTcRows + row;
                if (item + stride < items && r1 < p.R)
                    for (int o = 0; o < p.ngroups; o += 32) prefetch_l2(p.scales + r1 * p.ngroups + o);
            }
            const int reads = (nst + L::kRun - 1) / L::kRun;
#pragma unroll 1
            for (int s = 0; s < reads; ++s) {
                float sc[L::kSub];
                if (SC) {
#pragma unroll
                    for (int u = 0; u < L::kSub; ++u) {
                        // (behind the row's end lie sums of zeros: no group, since the last may be infinite)
                        const int chunk = (st0 + s) * (STEP / 32) + u * (STEP / 32 / L::kSub);
                        const int g = chunk < chunks ? static_cast<int>(fd_div(p.cpg, chunk)) : p.ngroups;
                        if ((g >> 2) != unit) {      // groups come in order, one unit after the other
                            unit = g >> 2;
                            cur = nxt;
                            nxt = load4(unit + 1);
                        }
                        sc[u] = g & 2 ? (g & 1 ? cur.w : cur.z) : (g & 1 ? cur.y : cur.x);
                    }
                }
                if (!mbar_ready(D_FULL(db), dph, abortp)) { ok = false; break; }
                tc_fence_after();
                // 32 columns of accumulators per wait
                constexpr int UB = NTOK == 16 && L::kSub > 1 ? 2 : 1;
#pragma unroll
                for (int u = 0; u < L::kSub; u += UB) {
                    uint32_t v[32];
                    const uint32_t src = tl + db * L::kAcc + u * NTOK;
                    if constexpr (UB * NTOK == 32) {
                        tmem_ld_32x32b_x32(src, v);
                        tmem_wait_ld(v);
                    } else {
                        uint32_t(&lo)[16] = *reinterpret_cast<uint32_t(*)[16]>(&v[0]);
                        tmem_ld_32x32b_x16(src, lo);
                        tmem_wait_ld(lo);
                    }
#pragma unroll
                    for (int k = 0; k < UB; ++k)
#pragma unroll
                        for (int i = 0; i < NTOK; ++i)
                            tot[i] = SC ? fmaf(sc[u + k], __uint_as_float(v[k * NTOK + i]), tot[i])
                                        : tot[i] + __uint_as_float(v[i]);
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(D_EMPTY(db));
                if (++db == ND) { db = 0; dph ^= 1u; }
            }
            if (!ok) break;
            if (p.split > 1) {
                // The parts of the cluster's blocks, in the first one's table space and, with 32 tokens and eight
                // blocks, the first 4 KB of the ring above it (one item per cluster then; behind the barrier nobody
                // needs a table any more, and every block's copies have landed and been used).
                static_assert(kHalfTab + 8 * kTcRows * (NTOK + 1) * 4 <= kTcEnd, "parts of eight blocks");
                const uint32_t mine = tab + (rank * kTcRows + row) * (NTOK + 1) * 4;
                cluster_barrier();
                uint32_t dst;
                asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(dst) : "r"(mine), "r"(0u));
#pragma unroll
                for (int i = 0; i < NTOK; ++i)
                    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(dst + i * 4), "f"(tot[i]) : "memory");
                cluster_barrier();
                if (rank == 0) {
#pragma unroll
                    for (int i = 0; i < NTOK; ++i) tot[i] = 0.f;
                    for (int k = 0; k < p.split; ++k)
#pragma unroll
                        for (int i = 0; i < NTOK; ++i) {
                            float a;
                            asm volatile("ld.shared.f32 %0, [%1];" : "=f"(a) : "r"(tab + ((k * kTcRows + row) * (NTOK + 1) + i) * 4) : "memory");
                            tot[i] += a;
                        }
                }
            }
            if (rank == 0 && r0 + row < p.R) {
#pragma unroll
                for (int i = 0; i < NTOK; ++i)
                    if (m0 + i < p.M) y[(m0 + i) * p.R + r0 + row] = Cvt<T>::from_f(tot[i]);
            }
        }
        if (p.split > 1 && !ok) {      // the cluster's other blocks wait for these two
            cluster_barrier();
            cluster_barrier();
        }
    } else if (warp == kTcProd) {
        // ------------------------------------------------------------ requests
        const uint64_t pol = l2_policy_evict_first(), polx = l2_policy_evict_last();
        int g = 0, slot = 0;
        uint32_t ph = 1;
        bool ok = true;
        for (int item = first; item < items && ok; item += stride) {
            const int r0 = (item % p.rtiles) * kTcRows, m0 = (item / p.rtiles) * NTOK;
#pragma unroll 1
            for (int s = st0; s < st1; ++s) {
                if (!mbar_ready(EMPTY(slot), ph, abortp)) { ok = false; break; }
                if (lane == 0 && !(p.withhold && g == 0 && blockIdx.x == 0)) {
                    const uint32_t dst = stage_addr(slot);
                    mbar_arrive_expect_tx(FULL(slot), L::kStage);
                    tma_load_2d(dst, &tmW, FULL(slot), s * (STEP / 2), r0, pol);
                    if (p.x3d) {
                        tma_load_3d(dst + L::kCodeBytes, &tmX, FULL(slot), 0, m0, s * (STEP / 64), polx);
                    } else {
                        for (int c = 0; c < STEP / 64; ++c)
                            tma_load_2d(dst + L::kCodeBytes + c * L::kXChunk, &tmX, FULL(slot), s * STEP + c * 64, m0, polx);
                    }
                }
                __syncwarp();
                ++g;
                if (++slot == S) { slot = 0; ph ^= 1u; }
            }
        }
        // every copy lands before its memory goes away, after a wait that ran out too
        for (int s = max(0, g - S); s < g; ++s) mbar_wait_warp(FULL(s % S), (s / S) & 1, nullptr);
    } else {
        // ------------------------------------------------------------ MMA issuer
        const bool issuer = elect_one();
        int slot = 0, ab = 0, db = 0;
        uint32_t ph = 0, aph = 0, dph = 1;
        bool ok = true;
        for (int item = first; item < items && ok; item += stride) {
#pragma unroll 1
            for (int s = 0; s < nst; ++s) {
                const bool new_acc = s % L::kRun == 0, end_acc = (s + 1) % L::kRun == 0 || s + 1 == nst;
                if (new_acc && !mbar_ready(D_EMPTY(db), dph, abortp)) { ok = false; break; }
                if (!mbar_ready(FULL(slot), ph, abortp) || !mbar_ready(A_FULL(ab), aph, abortp)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                if (issuer) {
                    const uint64_t bd = sw128_kmajor_desc(stage_addr(slot) + L::kCodeBytes);
                    const uint32_t a = tmem + L::kACol + ab * (STEP / 2), d = tmem + db * L::kAcc;
                    constexpr int PER = STEP / 16 / L::kSub;      // MMAs per accumulator
#pragma unroll
                    for (int kk = 0; kk < STEP / 16; ++kk)
                        tc_mma_ts(d + kk / PER * NTOK, a + kk * 8, bd + (kk >> 2) * (L::kXChunk >> 4) + (kk & 3) * 2,
                                  p.idesc, SC ? (kk % PER ? 1u : 0u) : (kk || !new_acc ? 1u : 0u));
                    tc_commit(A_EMPTY(ab));
                    tc_commit(EMPTY(slot));
                    if (end_acc) tc_commit(D_FULL(db));
                }
                __syncwarp();
                if (++slot == S) { slot = 0; ph ^= 1u; }
                if (++ab == NA) { ab = 0; aph ^= 1u; }
                if (end_acc && ++db == ND) { db = 0; dph ^= 1u; }
            }
        }
        // every MMA issued above completes before TMEM is released
        if (issuer) tc_commit(DRAIN);
        __syncwarp();
        mbar_wait_warp(DRAIN, 0, nullptr);
    }
    if (p.split > 1 && (warp < kTcDecode || warp >= kTcEpi + 4)) {
        cluster_barrier();
        cluster_barrier();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kTcMma) tmem_dealloc(tmem, 512);
}

}  // namespace mv4
}  // namespace km
