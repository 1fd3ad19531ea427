// km_matvec4.cu -- products with weights held as 4-bit codes of per-row codebooks.
//
//   y[m,r] = sum_n s[r, n / group] * T(C[r, code[r,n]]) * x[m,n]
//
// T() rounds a codebook value to x's dtype, as the assignment rounds its centroids; the products
// with the group scales and all sums are fp32. Two codes share a byte (even position in the low
// half); rows are padded to 16 bytes so that every row starts on a vector boundary.
#include <type_traits>

#include "km_common.cuh"
#include "km_host.h"

namespace km {
namespace mv4 {

constexpr int kKmax = 16;
// Additions of the tensor cores truncate, up to 1.3e-7 of the sum each where all terms have one sign (measured:
// rows of 2^22 codes, 32768 products to a warp, 3.3e-3 too small). After this many the sum goes on in fp32: 1.3e-4,
// less than half of fp16's half step.
constexpr int kMaxChain = 1024;

// codes [R,N] -> packed [R, pitch]; one thread per 16 bytes (32 codes), padding codes 0. VEC: rows are
// whole 16-byte units (32768 x 8192: 58 us, 6.9 TB/s; byte by byte 246).
template <bool VEC>
__global__ void __launch_bounds__(256)
    pack4_kernel(const uint8_t *__restrict__ codes, int64_t R, int64_t N, int64_t chunks, uint4 *__restrict__ packed) {
    const int64_t u = blockIdx.x * 256ll + threadIdx.x;
    if (u >= R * chunks) return;
    const int64_t r = u / chunks, n0 = (u - r * chunks) * 32;
    const uint8_t *src = codes + r * N + n0;
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (VEC) {
            if (i % 2) continue;
            uint4 v = make_uint4(0u, 0u, 0u, 0u);
            if (n0 + i * 8 < N) v = __ldg(reinterpret_cast<const uint4 *>(src + i * 8));
            // four codes, a byte each, to 16 bits: every odd one beside the one before it
            auto four = [](uint32_t c) { c &= 0x0f0f0f0fu; return c | c >> 4; };
            w[i] = __byte_perm(four(v.x), four(v.y), 0x6420);
            w[i + 1] = __byte_perm(four(v.z), four(v.w), 0x6420);
            continue;
        }
        w[i] = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (n0 + i * 8 + j < N) w[i] |= static_cast<uint32_t>(src[i * 8 + j] & 15) << (4 * j);
    }
    packed[u] = make_uint4(w[0], w[1], w[2], w[3]);
}

// fp32 tokens, on the CUDA cores: a warp per row, eight consecutive codes per lane and step. The
// row's 16 codebook values lie in 16 different banks, so the 32 lanes' lookups never conflict.
// The tokens are staged in shared memory kSimtChunk positions at a time, every group of eight in two
// 16-byte halves 16 * kSimtChunk / 8 bytes apart, which a warp reads without conflicts; the codes of
// the next chunk are read before that. (1003 rows x 1999, three tokens: with the tokens read from
// L2 element by element 17.5 us, staged 9.8.)
constexpr int kSimtWarps = 8;
constexpr int kSimtChunk = 1024;

template <int MT>
__global__ void __launch_bounds__(32 * kSimtWarps)
    matvec4_f32_kernel(const float *__restrict__ x, int64_t M, const uint8_t *__restrict__ packed, int64_t pitch,
                       const float *__restrict__ C, int64_t R, int N, int K, const float *__restrict__ scales,
                       FastDiv cpg, int ngroups, float *__restrict__ y) {
    constexpr int kSteps = kSimtChunk / 256;
    __shared__ float tab[kSimtWarps][kKmax];
    __shared__ float4 xs[MT][2][kSimtChunk / 8];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t r = static_cast<int64_t>(blockIdx.x) * kSimtWarps + warp, rr = min(r, R - 1);
    if (lane < kKmax) tab[warp][lane] = lane < K ? C[rr * K + lane] : 0.f;
    __syncwarp();
    const uint32_t *row = reinterpret_cast<const uint32_t *>(packed + rr * pitch);
    const float *srow = scales ? scales + rr * ngroups : nullptr;
    const int64_t m0 = static_cast<int64_t>(blockIdx.y) * MT;
    uint32_t next[kSteps];
    auto read_codes = [&](int n0) {
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
            const int n = n0 + i * 256 + lane * 8;
            next[i] = n < N ? __ldg(row + (n >> 3)) : 0u;
        }
    };
    read_codes(0);
    float acc[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m) acc[m] = 0.f;
    for (int n0 = 0; n0 < N; n0 += kSimtChunk) {
        uint32_t w[kSteps];
#pragma unroll
        for (int i = 0; i < kSteps; ++i) w[i] = next[i];
        __syncthreads();      // the chunk before is used up
#pragma unroll
        for (int m = 0; m < MT; ++m)
            for (int i = threadIdx.x; i < kSimtChunk; i += 32 * kSimtWarps) {
                const float v = n0 + i < N && m0 + m < M ? __ldg(x + (m0 + m) * N + n0 + i) : 0.f;
                reinterpret_cast<float *>(&xs[m][(i >> 2) & 1][i >> 3])[i & 3] = v;
            }
        if (n0 + kSimtChunk < N) read_codes(n0 + kSimtChunk);
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
            const int n = n0 + i * 256 + lane * 8;
            if (n >= N) break;
            float c[8];
#pragma unroll
            for (int j = 0; j < 8; ++j)
                c[j] = n + j < N ? tab[warp][(w[i] >> (4 * j)) & 15] : 0.f;   // (none behind the row's end)
            const float s = srow ? __ldg(srow + fd_div(cpg, n >> 5)) : 1.f;
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                const float4 a = xs[m][0][i * 32 + lane], b = xs[m][1][i * 32 + lane];
                const float p = fmaf(c[3], a.w, fmaf(c[2], a.z, fmaf(c[1], a.y, c[0] * a.x))) +
                                fmaf(c[7], b.w, fmaf(c[6], b.z, fmaf(c[5], b.y, c[4] * b.x)));
                acc[m] = fmaf(s, p, acc[m]);
            }
        }
    }
#pragma unroll
    for (int m = 0; m < MT; ++m) {
        const float t = warp_sum(acc[m]);
        if (lane == 0 && r < R && m0 + m < M) y[(m0 + m) * R + r] = t;
    }
}

// ------------------------------------------------------------------ 16-bit tokens: mma form
//
// Tiles of 16 rows of weights. The product runs as m16n8k16 matrix instructions with the weights
// as the row operand, so eight tokens cost what one costs. What bounds it: the lookups and the latencies around
// them. At 32768 x 8192, one token, a scale per 128 weights, the profile has shared memory's wavefronts 63 % busy,
// the fullest pipe, the tensor pipe 15 %, and short scoreboard, fixed waits and long scoreboard as the stalls; the
// tables are built anew for every tile. Measured there: 47 us, 3.1 TB/s (the bytes would take 22); 4096 x 4096
// 5.7 us. Turning codes into operands takes one
// shared-memory read per pair of codes: a byte indexes a 256-entry table of value pairs. A table
// row is 256 bytes, one word per lane and row half, so every lane reads its own bank (lane l of a
// fragment serves rows l / 4 and l / 4 + 8, whose tables are repeated for the four lanes of a
// row): 32 pairs per clock and SM whatever the codes are. The table starts on a multiple of 64 KB
// of the shared window, so a single byte permutation of (codes, lane) is the address.
//
// A block is one per SM and persistent; its two halves of eight warps work on tiles of their own
// (one builds its table while the other multiplies) and share nothing. The codes come through a
// ring of TMA copies per half (a stage is four boxes of 16 rows x 128 bytes, requested ahead across
// tiles), which keeps them off the load pipe that the lookups need; with the 128-byte swizzle the
// eight rows a warp reads at once lie in different banks. (Plain bulk copies, one per row, took a
// warp longer to issue than the whole stage takes to multiply.) A pair of
// instructions multiplies 32 consecutive codes, lane t of a row holding codes 8t .. 8t + 7 (the
// order of the reduction index inside an instruction is free), so its tokens are one 64-byte
// piece per row and every scale group of a multiple of 32 codes ends between two pairs: a scale
// multiplies an fp32 sum, never a weight.
constexpr int kMmaWarps = 8;                   // per half: each takes 128 codes of a stage's 1024
constexpr int kHalfThreads = 32 * kMmaWarps;
constexpr int kMmaThreads = 2 * kHalfThreads + 64;   // and a requesting warp per half
constexpr uint32_t kTabBytes = 65536;          // [entry][row half][lane] words
constexpr int kMmaStages = 4;
constexpr int kStageRow = 512;                 // bytes of a row per stage
constexpr uint32_t kBoxBytes = 16 * 128;
constexpr uint32_t kStageBytes = 16 * kStageRow;
constexpr uint32_t kRingBytes = kMmaStages * kStageBytes;
// One ring below the 64 KB boundary that the tables start on, one behind the tables.
constexpr uint32_t kMmaSmem = 3 * kTabBytes + kRingBytes;

struct MmaParams {
    const float *C, *scales;
    int64_t pitch, R, M;
    int N, K, ngroups;
    int rtiles, items;           // tiles of 16 rows, times tiles of 8 NT tokens
    FastDiv cpg;                 // 32-code chunks per scale group
    int withhold;                // test only: the first half block never asks for its first stage
};

__device__ __forceinline__ uint32_t lds32(uint32_t a) {
    uint32_t v;
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
    return v;
}
// A word of the tables, which do not change while a tile's lookups run: no memory clobber, the
// barriers around the tile order the accesses.
template <int OFF> __device__ __forceinline__ uint32_t lds_tab(uint32_t a) {
    uint32_t v;
    asm volatile("ld.shared.b32 %0, [%1+%2];" : "=r"(v) : "r"(a), "n"(OFF));
    return v;
}
__device__ __forceinline__ void prefetch_l2(const void *a) {
    asm volatile("prefetch.global.L2 [%0];" ::"l"(a));
}
__device__ __forceinline__ void sts128(uint32_t a, uint32_t v) {
    asm volatile("st.shared.v4.b32 [%0], {%1,%1,%1,%1};" ::"r"(a), "r"(v) : "memory");
}

template <typename T>
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1);
template <>
__device__ __forceinline__ void mma16816<__half>(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <>
__device__ __forceinline__ void mma16816<__nv_bfloat16>(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <typename T> __device__ __forceinline__ uint32_t bits16(T v) {
    return *reinterpret_cast<const uint16_t *>(&v);
}

// One token's values of eight consecutive positions, zeros past the end of the row.
template <typename T, bool XV>
__device__ __forceinline__ void load_x(const T *xr, int at, int N, uint32_t (&b)[4]) {
    if (XV) {              // rows are whole 16-byte units
        uint4 v = make_uint4(0u, 0u, 0u, 0u);
        if (at < N) v = __ldg(reinterpret_cast<const uint4 *>(xr + at));
        b[0] = v.x, b[1] = v.y, b[2] = v.z, b[3] = v.w;
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            b[i] = 0;
            if (at + 2 * i < N) b[i] = bits16(xr[at + 2 * i]);
            if (at + 2 * i + 1 < N) b[i] |= bits16(xr[at + 2 * i + 1]) << 16;
        }
    }
}

// Warp-wide bounded wait whose waiting part is kept out of the loops it is used in.
__device__ __noinline__ bool mbar_wait_long(uint32_t bar, uint32_t parity, volatile int *abort_flag) {
    return mbar_wait_warp(bar, parity, abort_flag);
}
__device__ __forceinline__ bool mbar_ready(uint32_t bar, uint32_t parity, volatile int *abort_flag) {
    if (__all_sync(0xffffffffu, mbar_test_wait(bar, parity))) return true;
    return mbar_wait_long(bar, parity, abort_flag);
}

}  // namespace mv4
}  // namespace km

#include "km_matvec4_tc.cuh"

namespace km {
namespace mv4 {

// SC: 0 no scales, 1 groups of whole 128-code blocks, 2 any multiple of 32, 3 no scales and rows so long that a
// warp's sum must end after kMaxChain products (a form of its own: the second sum's registers cost 32 tokens
// x 4096 x 4096 13.0 to 14.4 us).
template <typename T, bool XV, int NT, int SC>
__global__ void __launch_bounds__(kMmaThreads, 1)
    matvec4_mma_kernel(const __grid_constant__ CUtensorMap tm, const T *__restrict__ x, const MmaParams p,
                       T *__restrict__ y) {
    constexpr int XD = NT > 2 ? 2 : 4;       // chunks of tokens held ahead
    constexpr bool scaled = SC == 1 || SC == 2;
    constexpr int kRun = kMaxChain / 8;      // (SC 3) stages, of eight products a warp, to a sum
    constexpr int kCodesPerStage = 2 * kStageRow;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ __align__(8) uint64_t bars[2][2 * kMmaStages];
    __shared__ __align__(16) uint16_t values[2][16][24];   // the tile's codebooks (rows 48 bytes apart)
    __shared__ int abort_flags[2];
    const uint32_t base = smem_u32(smem);
    const uint32_t tab0 = (base + 1024 + kRingBytes + kTabBytes - 1) & ~(kTabBytes - 1);
    if (tab0 + 2 * kTabBytes + kRingBytes > base + kMmaSmem) {   // never: the window starts near 0
        if (threadIdx.x == 0) record_dev_error(kDevErrTimeout);
        return;
    }
    const int lane = threadIdx.x & 31;
    const bool producer = threadIdx.x >= 2 * kHalfThreads;
    const int half = producer ? (threadIdx.x - 2 * kHalfThreads) >> 5 : threadIdx.x / kHalfThreads;
    const uint32_t ring = half ? tab0 + 2 * kTabBytes : (base + 1023) & ~1023u;
    const uint32_t full0 = smem_u32(bars[half]), empty0 = full0 + 8 * kMmaStages;
    volatile int *abortp = &abort_flags[half];
    const int nstages = static_cast<int>((p.pitch + kStageRow - 1) / kStageRow);
    if (threadIdx.x < 2) {
        abort_flags[threadIdx.x] = 0;
        const uint32_t b = smem_u32(bars[threadIdx.x]);
        for (int s = 0; s < kMmaStages; ++s) {
            mbar_init(b + 8 * s, 1);
            mbar_init(b + 8 * (kMmaStages + s), kMmaWarps);
        }
        fence_mbar_init();
    }
    __syncthreads();
    const int item0 = half * static_cast<int>(gridDim.x) + static_cast<int>(blockIdx.x), step = 2 * static_cast<int>(gridDim.x);

    if (producer) {
        // Requests the stages of the half's tiles one after the other. Rows and bytes behind the end
        // arrive as zeros.
        const uint64_t pol = l2_policy_evict_first();
        int slot = 0, asked = 0;
        uint32_t ph = 1;
        for (int item = item0; item < p.items; item += step) {
            const int row = (item % p.rtiles) * 16;
            for (int s = 0; s < nstages; ++s) {
                if (!mbar_wait_warp(empty0 + 8 * slot, ph, abortp)) { item = p.items - step; break; }
                if (lane == 0 && !(p.withhold && asked == 0 && blockIdx.x == 0 && half == 0)) {
                    mbar_arrive_expect_tx(full0 + 8 * slot, kStageBytes);
#pragma unroll
                    for (int i = 0; i < kStageRow / 128; ++i)
                        tma_load_2d(ring + slot * kStageBytes + i * kBoxBytes, &tm, full0 + 8 * slot, s * kStageRow + i * 128,
                                    row, pol);
                }
                __syncwarp();
                ++asked;
                if (++slot == kMmaStages) { slot = 0; ph ^= 1u; }
            }
        }
        // every copy lands before its memory goes away, after a wait that ran out too
        for (int s = max(0, asked - kMmaStages); s < asked; ++s)
            mbar_wait_warp(full0 + 8 * (s % kMmaStages), (s / kMmaStages) & 1, nullptr);
        return;
    }

    const int ht = threadIdx.x % kHalfThreads, warp = ht >> 5;
    const int g = lane >> 2, t = lane & 3;
    const uint32_t tab = tab0 + half * kTabBytes;
    // Codebook value ht % 16 of row ht / 16 of an item's tile (0 beyond the codebook or the rows).
    auto codebook_value = [&](int item) {
        const int64_t row = static_cast<int64_t>(item % p.rtiles) * 16 + (ht >> 4);
        return item < p.items && row < p.R && (ht & 15) < p.K ? __ldg(p.C + row * p.K + (ht & 15)) : 0.f;
    };
    float cval = codebook_value(item0);
    const uint32_t lane4 = tab + lane * 4;                    // byte 0 the lane's word, 2-3 the table
    // this lane's word of chunk h: 16-byte unit (warp % 2) * 4 + h of row g (or g + 8) in box warp / 2,
    // swizzled: unit u of row r lies at u ^ (r % 8)
    const uint32_t my_codes = ring + (warp >> 1) * kBoxBytes + g * 128 + t * 4;
    const uint32_t unit0 = (((warp & 1) * 4) ^ g) * 16;       // of chunk h: unit0 ^ 16 h
    int slot = 0;
    uint32_t ph = 0;
    bool ok = true;
    for (int item = item0; item < p.items; item += step) {
        const int64_t r0 = static_cast<int64_t>(item % p.rtiles) * 16;
        const int64_t m0 = static_cast<int64_t>(item / p.rtiles) * (8 * NT);
        // Lanes without a token load nothing and multiply whatever they hold: columns do not mix,
        // and theirs are not written. (A 16-byte load costs the load pipe a cycle per eight lanes
        // even where all lanes name the same address.)
        const T *xr[NT];       // this lane's positions of the warp's block in the current stage
        bool xin[NT];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            xin[n] = m0 + n * 8 + g < p.M;
            xr[n] = x + min(m0 + n * 8 + g, p.M - 1) * p.N + warp * 128 + t * 8;
        }
        const float *sa = nullptr, *sb = nullptr;
        if (scaled) {
            sa = p.scales + min(r0 + g, p.R - 1) * p.ngroups;
            sb = p.scales + min(r0 + g + 8, p.R - 1) * p.ngroups;
        }
        const int nfull = p.N / kCodesPerStage;
        // Tokens and scales are read one stage ahead: chunk h of the next stage replaces chunk h of
        // this one as soon as that is multiplied (after the last stage it is read again).
        uint32_t xb[XD][NT][4];
#pragma unroll
        for (int h = 0; h < XD; ++h)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) xb[h][n][i] = 0;
        auto next_x = [&](int h, int add, int b) {
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                if (!xin[n]) continue;
                if (XV) {
                    const uint4 v = __ldg(reinterpret_cast<const uint4 *>(xr[n] + add + h * 32));
                    xb[b][n][0] = v.x, xb[b][n][1] = v.y, xb[b][n][2] = v.z, xb[b][n][3] = v.w;
                } else {
                    load_x<T, false>(xr[n] + add + h * 32, 0, 8, xb[b][n]);
                }
            }
        };
        // The four lanes of a row hold four of its scales each time: those of the warp's blocks in
        // four consecutive stages (SC 1) or of the four chunks of its block (SC 2).
        float sca = 1.f, scb = 1.f, nxa = 1.f, nxb = 1.f;
        auto read_scales = [&](int s, float &a, float &b) {
            const uint32_t q = SC == 1 ? (min(s + t, nfull - 1) * kMmaWarps + warp) * 4 : (s * kMmaWarps + warp) * 4 + t;
            const uint32_t gi = fd_div(p.cpg, q);
            a = __ldg(sa + gi);
            b = __ldg(sb + gi);
        };
        if (nfull > 0) {
#pragma unroll
            for (int h = 0; h < XD; ++h) next_x(h, 0, h);
            if (scaled) read_scales(0, nxa, nxb);
        }
        {
            // pair tables: this thread's row, the 16 entries with high code `hi`; every thread holds
            // one codebook value of the tile, read while the tile before was multiplied
            values[half][ht >> 4][ht & 15] = bits16(Cvt<T>::from_f(cval));
            named_barrier_sync(1 + half, kHalfThreads);       // and the previous tile's sums are read
            cval = codebook_value(item + step);
            if (scaled) {
                // the next tile's scales into L2
                const int64_t r1 = static_cast<int64_t>((item + step) % p.rtiles) * 16 + (ht >> 4);
                if (item + step < p.items && r1 < p.R)
                    for (int o = (ht & 15) * 32; o < p.ngroups; o += 512) prefetch_l2(p.scales + r1 * p.ngroups + o);
            }
            const int row = ht & 15, hi = ht >> 4;
            const uint4 c0 = *reinterpret_cast<const uint4 *>(&values[half][row][0]);
            const uint4 c1 = *reinterpret_cast<const uint4 *>(&values[half][row][8]);
            const uint32_t c[8] = {c0.x, c0.y, c0.z, c0.w, c1.x, c1.y, c1.z, c1.w};
            const uint32_t vh = static_cast<uint32_t>(values[half][row][hi]) << 16;
            const uint32_t dst = tab + hi * 4096 + (row >> 3) * 128 + (row & 7) * 16;
#pragma unroll
            for (int k = 0; k < 16; k += 2) {
                sts128(dst + k * 256, __byte_perm(c[k / 2], vh, 0x7610));
                sts128(dst + k * 256 + 256, __byte_perm(c[k / 2], vh, 0x7632));
            }
        }
        named_barrier_sync(1 + half, kHalfThreads);
        float tot[NT][4], acc[NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) tot[n][i] = acc[n][i] = 0.f;
        auto add = [&](float a0, float a1) {
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                tot[n][0] = fmaf(a0, acc[n][0], tot[n][0]);
                tot[n][1] = fmaf(a0, acc[n][1], tot[n][1]);
                tot[n][2] = fmaf(a1, acc[n][2], tot[n][2]);
                tot[n][3] = fmaf(a1, acc[n][3], tot[n][3]);
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[n][i] = 0.f;
            }
        };
        // the four operand words of instruction j of a pair
        auto operand = [&](uint32_t wa, uint32_t wb, int j, uint32_t (&f)[4]) {
            const uint32_t k0 = 0x7604 | (2 * j) << 4, k1 = 0x7604 | (2 * j + 1) << 4;
            f[0] = lds_tab<0>(__byte_perm(wa, lane4, k0));
            f[1] = lds_tab<128>(__byte_perm(wb, lane4, k0));
            f[2] = lds_tab<0>(__byte_perm(wa, lane4, k1));
            f[3] = lds_tab<128>(__byte_perm(wb, lane4, k1));
        };
#pragma unroll 1
        for (int s = 0; s < nfull; ++s) {
            if (!mbar_ready(full0 + 8 * slot, ph, abortp)) { ok = false; break; }
            uint32_t wa[4], wb[4];
            {
                const uint32_t src = my_codes + slot * kStageBytes + unit0;
#pragma unroll
                for (int h = 0; h < 4; ++h) {
                    // (unit0 ^ 16 h) == unit0 +- 16 h bit by bit: xor on the address, whose bits 4-6 it is
                    wa[h] = lds32(src ^ (h * 16));
                    wb[h] = lds32((src ^ (h * 16)) + 8 * 128);
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(empty0 + 8 * slot);
            const int ahead = s + 1 < nfull ? kCodesPerStage : 0;
            if (SC == 2 || (SC == 1 && (s & 3) == 0)) {
                sca = nxa, scb = nxb;
                const int ns = s + (SC == 1 ? 4 : 1);
                if (ns < nfull) read_scales(ns, nxa, nxb);
            }
#pragma unroll
            for (int h = 0; h < 4; ++h) {
                __syncwarp();        // lanes without a token read none; the products want the whole warp
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    uint32_t f[4];
                    operand(wa[h], wb[h], j, f);
#pragma unroll
                    for (int n = 0; n < NT; ++n)
                        mma16816<T>(SC ? acc[n] : tot[n], f, xb[h % XD][n][2 * j], xb[h % XD][n][2 * j + 1]);
                }
                if (h + XD < 4) next_x(h + XD, 0, h % XD);
                else next_x(h + XD - 4, ahead, h % XD);
                if (SC == 2) add(__shfl_sync(0xffffffffu, sca, (lane & 28) + h), __shfl_sync(0xffffffffu, scb, (lane & 28) + h));
            }
            if (SC == 3 && s % kRun == kRun - 1) add(1.f, 1.f);
            if (SC == 1) add(__shfl_sync(0xffffffffu, sca, (lane & 28) + (s & 3)), __shfl_sync(0xffffffffu, scb, (lane & 28) + (s & 3)));
#pragma unroll
            for (int n = 0; n < NT; ++n) xr[n] += kCodesPerStage;
            if (++slot == kMmaStages) { slot = 0; ph ^= 1u; }
        }
        if (ok && nfull < nstages) {
            // the last, partly filled stage
            if (!mbar_ready(full0 + 8 * slot, ph, abortp)) ok = false;
            const uint32_t src = my_codes + slot * kStageBytes + unit0;
            const int q0 = (nfull * kMmaWarps + warp) * 4;
            for (int h = 0; ok && h < 4 && (q0 + h) * 32 < p.N; ++h) {
                const int at = (q0 + h) * 32 + 8 * t;        // this lane's first code
                uint32_t xt[NT][4];
#pragma unroll
                for (int n = 0; n < NT; ++n) load_x<T, XV>(xr[n] + h * 32, 0, xin[n] ? p.N - at : 0, xt[n]);
                const uint32_t wa = lds32(src ^ (h * 16)), wb = lds32((src ^ (h * 16)) + 8 * 128);
                __syncwarp();
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    uint32_t f[4];
                    operand(wa, wb, j, f);
                    // codes behind the row's end are no weights (a codebook value may be infinite)
                    const int c = at + 4 * j;
                    if (c >= p.N) f[0] = f[1] = 0;
                    else if (c + 1 >= p.N) f[0] &= 0xffff, f[1] &= 0xffff;
                    if (c + 2 >= p.N) f[2] = f[3] = 0;
                    else if (c + 3 >= p.N) f[2] &= 0xffff, f[3] &= 0xffff;
#pragma unroll
                    for (int n = 0; n < NT; ++n) mma16816<T>(SC ? acc[n] : tot[n], f, xt[n][2 * j], xt[n][2 * j + 1]);
                }
                if (scaled) {
                    const uint32_t gi = fd_div(p.cpg, q0 + h);
                    add(sa[gi], sb[gi]);
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(empty0 + 8 * slot);
            if (++slot == kMmaStages) { slot = 0; ph ^= 1u; }
        }
        if (SC == 3) add(1.f, 1.f);
        // the warps' sums, joined in warp order, through the table's place: [warp][token][17]
        __syncwarp();
        if (named_barrier_or(1 + half, kHalfThreads, !ok)) break;
        float *red = reinterpret_cast<float *>(smem + (tab - base));
        float *w = red + warp * (8 * NT * 17);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            w[(n * 8 + 2 * t) * 17 + g] = tot[n][0];
            w[(n * 8 + 2 * t + 1) * 17 + g] = tot[n][1];
            w[(n * 8 + 2 * t) * 17 + g + 8] = tot[n][2];
            w[(n * 8 + 2 * t + 1) * 17 + g + 8] = tot[n][3];
        }
        named_barrier_sync(1 + half, kHalfThreads);
        for (int i = ht; i < 16 * 8 * NT; i += kHalfThreads) {
            const int r = i & 15, mm = i >> 4;
            float v = 0.f;
#pragma unroll
            for (int k = 0; k < kMmaWarps; ++k) v += red[k * (8 * NT * 17) + mm * 17 + r];
            if (r0 + r < p.R && m0 + mm < p.M) y[(m0 + mm) * p.R + r0 + r] = Cvt<T>::from_f(v);
        }
    }
}

}  // namespace mv4
}  // namespace km

namespace {

using namespace km::mv4;

// The tcgen05 form decodes once for all tokens, where the mma.sync form pays for every eight, but it
// takes some 8 us to start and end. GPU times, tcgen05 / mma.sync: 16 tokens x 8192 x 8192 21 / 32 us,
// x 4096 x 4096 13.5 / 8.8; 32 tokens x 8192 x 8192 26 / 46, x 4096 x 4096 23 / 19.
constexpr int64_t kTcMinTokens = 8, kTcMinWeights = int64_t{1} << 25;

inline int64_t pitch_of(int64_t N) { return ceil_div(N, 32) * 16; }

template <int MT>
km_status f32_launch(const float *x, int64_t M, const uint8_t *packed, const float *C, int64_t R, int64_t N, int64_t K,
                     const float *scales, int64_t group, float *y, cudaStream_t st) {
    const int64_t blocks = ceil_div(R, kSimtWarps), per = static_cast<int64_t>(kMaxGridY) * MT;
    for (int64_t m0 = 0; m0 < M; m0 += per) {
        const int64_t mn = std::min(per, M - m0);
        const dim3 grid(static_cast<unsigned>(blocks), static_cast<unsigned>(ceil_div(mn, MT)));
        matvec4_f32_kernel<MT><<<grid, 32 * kSimtWarps, 0, st>>>(
            x + m0 * N, mn, packed, pitch_of(N), C, R, static_cast<int>(N), static_cast<int>(K), scales,
            km::make_fastdiv(static_cast<uint32_t>(scales ? group / 32 : 1)),
            scales ? static_cast<int>(ceil_div(N, group)) : 0, y + m0 * R);
        if (launch_status() != KM_OK) return KM_ERR_CUDA;
    }
    return KM_OK;
}
km_status matvec4_f32(const void *xv, int64_t M, const uint8_t *packed, const float *C, int64_t R, int64_t N, int64_t K,
                      const float *scales, int64_t group, void *yv, cudaStream_t st) {
    const float *x = static_cast<const float *>(xv);
    float *y = static_cast<float *>(yv);
    if (M == 1) return f32_launch<1>(x, M, packed, C, R, N, K, scales, group, y, st);
    return f32_launch<4>(x, M, packed, C, R, N, K, scales, group, y, st);
}

template <typename T, bool XV, int NT, int SC>
km_status mma_launch(const CUtensorMap &tm, const T *x, MmaParams p, T *y, cudaStream_t st) {
    auto kernel = matvec4_mma_kernel<T, XV, NT, SC>;
    static std::atomic<uint64_t> ready{0};
    if (!allow_smem(kernel, kMmaSmem, ready)) return KM_ERR_CUDA;
    const int64_t rtiles = ceil_div(p.R, 16);
    if (rtiles > kMaxIndex / 4) return KM_ERR_UNSUPPORTED;
    // as many token tiles per launch as keep the item number below 2^30
    const int64_t per = std::max<int64_t>(1, (int64_t{1} << 30) / rtiles) * 8 * NT, M = p.M;
    for (int64_t m0 = 0; m0 < M; m0 += per) {
        p.M = std::min(per, M - m0);
        p.rtiles = static_cast<int>(rtiles);
        p.items = static_cast<int>(rtiles * ceil_div(p.M, 8 * NT));
        kernel<<<static_cast<unsigned>(std::min(p.items, num_sms())), kMmaThreads, kMmaSmem, st>>>(
            tm, x + m0 * p.N, p, y + m0 * p.R);
        if (launch_status() != KM_OK) return KM_ERR_CUDA;
    }
    return KM_OK;
}
template <typename T, bool XV, int SC>
km_status mma_tokens(const CUtensorMap &tm, const T *x, const MmaParams &p, T *y, cudaStream_t st) {
    if (p.M <= 8) return mma_launch<T, XV, 1, SC>(tm, x, p, y, st);
    if (p.M <= 16) return mma_launch<T, XV, 2, SC>(tm, x, p, y, st);
    return mma_launch<T, XV, 4, SC>(tm, x, p, y, st);
}
template <typename T, bool XV>
km_status mma_scales(const CUtensorMap &tm, const T *x, const MmaParams &p, T *y, cudaStream_t st) {
    // a warp takes an eighth of the row, 16 codes to a product
    if (!p.scales) return p.N <= 8 * 16 * kMaxChain ? mma_tokens<T, XV, 0>(tm, x, p, y, st) : mma_tokens<T, XV, 3>(tm, x, p, y, st);
    return p.cpg.d % 4 == 0 ? mma_tokens<T, XV, 1>(tm, x, p, y, st) : mma_tokens<T, XV, 2>(tm, x, p, y, st);
}
// tcgen05 form: rows of x in whole 16-byte units.
template <typename T, int NTOK, int SC>
km_status tc_launch(const uint8_t *packed, const T *x, TcMvParams p, T *y, cudaStream_t st) {
    using L = TcMv<NTOK, SC>;
    const EncodeTiledFn enc = encode_fn();
    if (!enc) return KM_ERR_CUDA;
    CUtensorMap tmW, tmX;
    const cuuint32_t estr[3] = {1, 1, 1};
    {
        const int64_t pitch = pitch_of(p.N);
        const cuuint64_t dims[2] = {static_cast<cuuint64_t>(pitch), static_cast<cuuint64_t>(p.R)};
        const cuuint64_t strides[1] = {static_cast<cuuint64_t>(pitch)};
        const cuuint32_t box[2] = {L::kStep / 2, kTcRows};
        if (enc(&tmW, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t *>(packed), dims, strides, box, estr,
                CU_TENSOR_MAP_INTERLEAVE_NONE, L::kStep == 256 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
            return KM_ERR_CUDA;
    }
    const bool bf16 = std::is_same<T, __nv_bfloat16>::value;
    {
        // Rows of whole 64-position chunks: one copy brings a step's chunks of all tokens (chunks as a
        // third index); else a copy per chunk, whose positions behind the row's end arrive as zeros.
        p.x3d = p.N % 64 == 0 ? 1 : 0;
        const cuuint64_t dims3[3] = {64, static_cast<cuuint64_t>(p.M), static_cast<cuuint64_t>(p.N / 64)};
        const cuuint64_t strides3[2] = {static_cast<cuuint64_t>(p.N) * 2, 128};
        const cuuint32_t box3[3] = {64, NTOK, L::kStep / 64};
        const cuuint64_t dims2[2] = {static_cast<cuuint64_t>(p.N), static_cast<cuuint64_t>(p.M)};
        if (enc(&tmX, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, p.x3d ? 3 : 2,
                const_cast<T *>(x), p.x3d ? dims3 : dims2, strides3, box3, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
            return KM_ERR_CUDA;
    }
    p.svec = p.scales && p.ngroups % 4 == 0 && aligned(p.scales, 16) ? 1 : 0;
    constexpr size_t smem = kTcEnd - 1024;      // the window's first 1024 bytes are the system's
    auto kernel = matvec4_tc_kernel<T, NTOK, SC>;
    static std::atomic<uint64_t> ready{0};
    if (!allow_smem(kernel, smem, ready)) return KM_ERR_CUDA;
    p.idesc = km::mma_idesc_f16(bf16 ? 1u : 0u, kTcRows, NTOK);
    p.withhold = km::g_withhold;
    p.rtiles = static_cast<int>(ceil_div(p.R, kTcRows));
    p.mtiles = static_cast<int>(ceil_div(p.M, NTOK));
    p.steps = static_cast<int>(ceil_div(p.N, L::kStep));
    const int64_t items = static_cast<int64_t>(p.rtiles) * p.mtiles;
    if (items > kMaxIndex / 16) return KM_ERR_UNSUPPORTED;
    // Few tiles: a cluster of 2, 4 or 8 blocks shares each, as long as all have an SM and two steps.
    const int sms = num_sms();
    p.split = 1;
    while (p.split < 8 && items * p.split * 2 <= sms && p.steps >= p.split * 2 * 2) p.split *= 2;
    p.sper = static_cast<int>(ceil_div(p.steps, p.split));
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(p.split > 1 ? items * p.split : std::min<int64_t>(items, sms)));
    cfg.blockDim = dim3(kTcThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = static_cast<unsigned>(p.split);
    attr.val.clusterDim.y = 1;
    attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, kernel, tmW, tmX, static_cast<const TcMvParams &>(p), y) != cudaSuccess) {
        cudaGetLastError();
        return KM_ERR_CUDA;
    }
    return KM_OK;
}
template <typename T, int NTOK>
km_status tc_scales(const uint8_t *packed, const T *x, const TcMvParams &p, T *y, cudaStream_t st) {
    if (!p.scales) return tc_launch<T, NTOK, 0>(packed, x, p, y, st);
    if (p.cpg.d % 4 == 0) return tc_launch<T, NTOK, 1>(packed, x, p, y, st);
    return p.cpg.d % 2 == 0 ? tc_launch<T, NTOK, 2>(packed, x, p, y, st) : tc_launch<T, NTOK, 3>(packed, x, p, y, st);
}
template <typename T>
km_status matvec4_tc(const T *x, int64_t M, const uint8_t *packed, const float *C, int64_t R, int64_t N, int64_t K,
                     const float *scales, int64_t group, T *y, cudaStream_t st) {
    TcMvParams p = {};
    p.C = C;
    p.scales = scales;
    p.R = R;
    p.N = static_cast<int>(N);
    p.K = static_cast<int>(K);
    p.ngroups = scales ? static_cast<int>(ceil_div(N, group)) : 0;
    p.cpg = km::make_fastdiv(static_cast<uint32_t>(scales ? group / 32 : 4));
    // as many tokens per launch as keep the item number small
    const int64_t per = std::max<int64_t>(1, (int64_t{1} << 24) / ceil_div(R, kTcRows)) * 32;
    for (int64_t m0 = 0; m0 < M; m0 += per) {
        p.M = std::min(per, M - m0);
        const km_status s = p.M <= 16 ? tc_scales<T, 16>(packed, x + m0 * N, p, y + m0 * R, st)
                                      : tc_scales<T, 32>(packed, x + m0 * N, p, y + m0 * R, st);
        if (s != KM_OK) return s;
    }
    return KM_OK;
}

template <typename T>
km_status matvec4_mma(const void *xv, int64_t M, const uint8_t *packed, const float *C, int64_t R, int64_t N,
                      int64_t K, const float *scales, int64_t group, void *yv, cudaStream_t st) {
    const T *x = static_cast<const T *>(xv);
    T *y = static_cast<T *>(yv);
    const bool xvec = N % 8 == 0 && aligned(x, 16);
    if (xvec && M > kTcMinTokens && R * N >= kTcMinWeights) return matvec4_tc<T>(x, M, packed, C, R, N, K, scales, group, y, st);
    const EncodeTiledFn enc = encode_fn();
    if (!enc) return KM_ERR_CUDA;
    CUtensorMap tm;
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(pitch_of(N)), static_cast<cuuint64_t>(R)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(pitch_of(N))};
    const cuuint32_t box[2] = {128, 16}, estr[2] = {1, 1};
    if (enc(&tm, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t *>(packed), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
        return KM_ERR_CUDA;
    MmaParams p = {};
    p.withhold = km::g_withhold;
    p.C = C;
    p.scales = scales;
    p.pitch = pitch_of(N);
    p.R = R;
    p.M = M;
    p.N = static_cast<int>(N);
    p.K = static_cast<int>(K);
    p.ngroups = scales ? static_cast<int>(ceil_div(N, group)) : 0;
    p.cpg = km::make_fastdiv(static_cast<uint32_t>(scales ? group / 32 : 4));
    return xvec ? mma_scales<T, true>(tm, x, p, y, st) : mma_scales<T, false>(tm, x, p, y, st);
}

}  // namespace

namespace km {
namespace mv4 {

cudaError_t take_device_error(unsigned int *bits) {
    const unsigned int zero = 0;
    const cudaError_t e = cudaMemcpyFromSymbol(bits, g_km_dev_error, sizeof(*bits));
    return e != cudaSuccess ? e : cudaMemcpyToSymbol(g_km_dev_error, &zero, sizeof(zero));
}
cudaError_t set_wait_limit(unsigned long long limit_ns) {
    return cudaMemcpyToSymbol(g_km_wait_limit_ns, &limit_ns, sizeof(limit_ns));
}

}  // namespace mv4
}  // namespace km

extern "C" {

km_status km_pack4(const uint8_t *codes, int64_t R, int64_t N, uint8_t *packed, void *stream) {
    if (!codes || !packed || !sizes_ok(R, N, 1, 1) || N > kMaxIndex - 256 || !aligned(packed, 16)) return KM_ERR_INVALID_ARG;
    const int64_t chunks = ceil_div(N, 32), blocks = ceil_div(R * chunks, 256);
    if (blocks > kMaxIndex) return KM_ERR_UNSUPPORTED;
    auto kernel = N % 16 == 0 && aligned(codes, 16) ? pack4_kernel<true> : pack4_kernel<false>;
    kernel<<<static_cast<unsigned>(blocks), 256, 0, S(stream)>>>(codes, R, N, chunks, reinterpret_cast<uint4 *>(packed));
    return launch_status();
}

km_status km_matvec4(const void *x, km_dtype dtype, int64_t M, const uint8_t *packed, const float *C, int64_t R,
                     int64_t N, int64_t K, const float *scales, int64_t group, void *y, void *stream) {
    if (!x || !packed || !C || !y || !valid_dtype(dtype) || !sizes_ok(R, N, K, 1) || M < 1 || M > kMaxIndex ||
        N > kMaxIndex - 1024 || !aligned(x, dtype_size(dtype)) || !aligned(y, dtype_size(dtype)) ||
        !aligned(packed, 16) || !aligned(C, 4) || (scales && !aligned(scales, 4)) ||
        (scales ? (group < 1 || group > kMaxIndex) : group != 0))
        return KM_ERR_INVALID_ARG;
    if (K > kKmax || (scales && group % 32 != 0)) return KM_ERR_UNSUPPORTED;
    switch (dtype) {
        case KM_F32: return matvec4_f32(x, M, packed, C, R, N, K, scales, group, y, S(stream));
        case KM_F16: return matvec4_mma<__half>(x, M, packed, C, R, N, K, scales, group, y, S(stream));
        default: return matvec4_mma<__nv_bfloat16>(x, M, packed, C, R, N, K, scales, group, y, S(stream));
    }
}

}  // extern "C"
