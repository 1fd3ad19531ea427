// km_xent.cuh -- kernels of the softmax cross entropy of points against all K table rows.
//
//   z[n,k]  = scale * <x_n, c_k>            lse[n] = log sum_k exp(z[n,k])
//   loss[n] = lse[n] - z[n, id_n]
//   P[n,k]  = w_n (exp(z[n,k] - lse[n]) - [k == id_n])     w_n = g_n * scale, 0 without a label
//   dX = P C          dC = P^T X
//
// The N x K logits are never stored. The loss reduces every tile of logits to one (maximum, sum of
// exponentials) pair per row where the tile was computed, the same idea as the assignment's
// running argmin, and joins the pairs of a row afterwards in tile order. The gradients recompute
// the logits one piece of the table at a time into P (in the points' type) and multiply that; 16-bit rows
// of up to 128 values keep P on the chip instead (km_xent_fused.cuh).
#pragma once

#include <type_traits>

#include "km_common.cuh"

namespace km {
namespace xe {

constexpr float kLog2e = 1.4426950408889634f;

enum Mode { kLse = 0, kProb = 1, kOut = 2 };

// What a product's tile does with its accumulators.
struct Epi {
    float scale;
    // kLse: pairs[(b * tiles + tile) * M + row], zt[b * M + row] where the label's column falls
    // in the tile
    float2 *pairs;
    float *zt;
    const int32_t *ids;    // labels (kLse, kProb); the table piece starts at row k0 of K
    int k0, K;
    // kProb
    const float *lse, *w;  // [B, M]
    void *P;               // [B, M, ldp]
    int64_t ldp;
    // kOut: out = acc (fp32) + value / f, or the fp32 partial of one split of the reduction
    const unsigned int *wmax;   // bits of max |w| (16-bit points), and see Stat; or null
    float pscale;          // s of p_factor
    bool rows;             // kOut, fp16: the result's rows are P's, whose shifts are undone (by the weights in w),
                           // else the points' common one is
    const float *acc;      // added, or null
    float *out32;          // fp32 result or partials [split][B][M][N], or null
    void *outT;            // result in the points' type, or null
    int splits;
};

// With 16-bit points P is held relative to the largest weight: P = (w_n / max |w|) s (p - [label]).
// The label's entry is the largest of its row, about -w_n, and in a mean of losses all w_n are
// equal: rounded as they are, every token's largest term would be off by the same fraction of
// itself (half a step of the type), which no sum over tokens averages away; relative to the maximum it
// is near -1, which has none of that. s is 1, and 2^14 for fp16, whose normal range ends at 2^-14:
// probabilities down to 2^-28 keep their bits. The products are multiplied by max |w| / s in fp32.
// (The rows of P of dX alone, in km_xent_fused.cuh, are each relative to their own weight.)
__device__ __forceinline__ float p_factor(const unsigned int *wmax, float s, bool inverse) {
    if (!wmax) return 1.f;
    const float m = fminf(fmaxf(__uint_as_float(*wmax), 0x1p-100f), 0x1p100f);
    return inverse ? m / s : s / m;
}

// What a sum of exponentials is taken against, given the maximum of its logits: the maximum, or 0 where that
// is infinite (every logit masked: the sum is then 0 instead of NaN).
__device__ __forceinline__ float sum_base(float m) { return isinf(m) ? 0.f : m; }

// fp16's range is too narrow for rows of P whose weights differ by many orders: beside a weight of 2^13, a row that
// weighs 2^-13 would keep its label's entry alone. Every row of P is therefore multiplied by 2^h, which brings its
// weight to the largest one's power of two; dX's rows are divided by it, and for dC, which sums over the points, the
// points are: X 2^(q - h), with q bringing the largest of them to the top of fp16's range, so that those
// divided by much keep their bits. All powers of two; with weights within a factor of two nothing changes.
// (bf16 has fp32's range and needs none of it.)
template <typename T> constexpr bool kShifts = std::is_same<T, __half>::value;
enum Stat { kMaxW = 0, kMinW = 1, kMaxX = 2, kStats = 3 };      // bits of max |w|, ~bits of min |w| > 0, bits of max |x|
__device__ __forceinline__ float pow2f(int e) { return __uint_as_float(static_cast<uint32_t>(127 + e) << 23); }
__device__ __forceinline__ int exponent_of(uint32_t bits) { return static_cast<int>(bits >> 23 & 255); }
// max_exp: exponent_of the largest weight
__device__ __forceinline__ int row_shift(int max_exp, float w) {
    return w == 0.f ? 0 : min(24, max(0, max_exp - exponent_of(__float_as_uint(w))));
}
__device__ __forceinline__ bool any_shift(const unsigned int *stat) {
    return stat[kMinW] != 0 && exponent_of(~stat[kMinW]) < exponent_of(stat[kMaxW]);
}
__device__ __forceinline__ int point_shift(const unsigned int *stat) {
    return any_shift(stat) && stat[kMaxX] ? min(24, max(0, 14 + 127 - exponent_of(stat[kMaxX]))) : 0;
}

// Two fp32 values in one register pair, for the packed fp32 arithmetic of sm_100.
__device__ __forceinline__ uint64_t pair_f32(float lo, float hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void unpair_f32(uint64_t v, float &lo, float &hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// What undoes the shifts in row br of a result.
__device__ __forceinline__ float out_shift(const Epi &p, int64_t br) {
    return pow2f(p.rows ? -row_shift(exponent_of(p.wmax[kMaxW]), p.w[br]) : -point_shift(p.wmax));
}

// ------------------------------------------------------------------ CUDA-core products

// One operand of a product: element (row, k) of batch b at base + b * batch + row * row_s + k * k_s,
// one of the two strides being 1.
struct Operand {
    const void *base;
    int64_t batch, row_s, k_s;
};

constexpr int ST = 128;        // tile rows and columns
constexpr int SK = 8;          // reduction step
constexpr int kSimtThreads = 256;

constexpr int kSimtLoads = ST * SK / kSimtThreads;

// A thread's part of the steps of one operand: value i is (row, step) = (u / SK, u % SK) of
// u = i * kSimtThreads + thread where the steps are contiguous, else (u % ST, u / ST).
template <typename T> struct SimtSrc {
    const T *p;                 // value 0 of the next step
    int64_t apart, advance;     // from value to value, from step to step
    uint32_t rows;              // bit i: value i's row exists
    int k, dk;                  // step index of value 0, from value to value
    bool km;
    __device__ __forceinline__ SimtSrc(const Operand &o, int64_t b, int row0, int nrows, int64_t k0) {
        const int t = threadIdx.x;
        km = o.k_s == 1;
        const int r = km ? t / SK : t % ST, dr = km ? kSimtThreads / SK : 0;
        k = km ? t % SK : t / ST;
        dk = km ? 0 : kSimtThreads / ST;
        p = static_cast<const T *>(o.base) + b * o.batch + (row0 + r) * o.row_s + (k0 + k) * o.k_s;
        apart = km ? dr * o.row_s : dk * o.k_s;
        advance = SK * o.k_s;
        rows = 0;
#pragma unroll
        for (int i = 0; i < kSimtLoads; ++i) rows |= static_cast<uint32_t>(row0 + r + i * dr < nrows) << i;
    }
    // `left` steps of the reduction remain
    __device__ __forceinline__ void load(int64_t left, float (&v)[kSimtLoads]) {
        const int lim = left < SK ? static_cast<int>(left) : SK;
#pragma unroll
        for (int i = 0; i < kSimtLoads; ++i) {
            v[i] = 0.f;
            if (((rows >> i) & 1) && k + i * dk < lim) v[i] = Cvt<T>::to_f(p[i * apart]);
        }
        p += advance;
    }
    __device__ __forceinline__ void store(const float (&v)[kSimtLoads], float (&dst)[SK][ST + 4]) const {
        float *d = &dst[0][0] + (km ? k * (ST + 4) + threadIdx.x / SK : k * (ST + 4) + threadIdx.x % ST);
        const int step = km ? kSimtThreads / SK : kSimtThreads / ST * (ST + 4);
#pragma unroll
        for (int i = 0; i < kSimtLoads; ++i) d[i * step] = v[i];
    }
};

// D[b, m, n] = sum_k A[b, m, k] B[b, n, k]; 128 x 128 tiles, 8 x 8 accumulators per thread (four
// 4 x 4 blocks 64 apart), operands staged as fp32 in two buffers, the next step's values on their way
// while one is multiplied, two products to an instruction. grid.x = tiles * splits * batches.
// Bound by the FMA pipe (62 % busy). fp32, 8192 x 8192 at d = 256: the loss 797 us, 43 TFLOP/s, both
// gradients 2950; with one buffer and an address computed for every value 1144 and 3930.
template <typename T, int MODE>
__global__ void __launch_bounds__(kSimtThreads, 2)
    simt_product_kernel(Operand A, Operand Bo, int M, int N, int64_t Kk, int mt, int nt, int64_t kper, Epi p) {
    __shared__ __align__(16) float sa[2][SK][ST + 4], sb[2][SK][ST + 4];
    int64_t id = blockIdx.x;
    const int n0 = static_cast<int>(id % nt) * ST;
    const int tile = static_cast<int>(id % nt);
    id /= nt;
    const int m0 = static_cast<int>(id % mt) * ST;
    id /= mt;
    const int split = static_cast<int>(id % p.splits);
    const int64_t b = id / p.splits, nb = gridDim.x / (static_cast<int64_t>(nt) * mt * p.splits);
    const int64_t kb = split * kper, ke = min(Kk, kb + kper);
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    uint64_t sum[8][4];
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) sum[i][j] = pair_f32(0.f, 0.f);
    float va[kSimtLoads], vb[kSimtLoads];
    SimtSrc<T> srca(A, b, m0, M, kb), srcb(Bo, b, n0, N, kb);
    srca.load(ke - kb, va);
    srcb.load(ke - kb, vb);
    int cur = 0;
    for (int64_t k = kb; k < ke; k += SK, cur ^= 1) {
        srca.store(va, sa[cur]);
        srcb.store(vb, sb[cur]);
        __syncthreads();         // (the other buffer was read before it)
        if (k + SK < ke) {
            srca.load(ke - k - SK, va);
            srcb.load(ke - k - SK, vb);
        }
#pragma unroll
        for (int q = 0; q < SK; ++q) {
            float av[8];
            uint64_t bv[4];
            *reinterpret_cast<float4 *>(av) = *reinterpret_cast<const float4 *>(&sa[cur][q][ty * 4]);
            *reinterpret_cast<float4 *>(av + 4) = *reinterpret_cast<const float4 *>(&sa[cur][q][64 + ty * 4]);
            *reinterpret_cast<ulonglong2 *>(bv) = *reinterpret_cast<const ulonglong2 *>(&sb[cur][q][tx * 4]);
            *reinterpret_cast<ulonglong2 *>(bv + 2) = *reinterpret_cast<const ulonglong2 *>(&sb[cur][q][64 + tx * 4]);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint64_t a2 = pair_f32(av[i], av[i]);
#pragma unroll
                for (int j = 0; j < 4; ++j) sum[i][j] = fma2(a2, bv[j], sum[i][j]);
            }
        }
    }
    float acc[8][8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) unpair_f32(sum[i][j], acc[i][2 * j], acc[i][2 * j + 1]);
    const float inv = MODE == kOut && p.splits == 1 ? p_factor(p.wmax, p.pscale, true) : 1.f;
    const float fac = MODE == kProb ? p_factor(p.wmax, p.pscale, false) : 1.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int row = m0 + (i & 3) + ty * 4 + (i >> 2) * 64;
        const bool rin = row < M;
        const int64_t br = b * M + row;
        if (MODE == kLse) {
            float m = -INFINITY;
            const int label = rin ? p.ids[br] : -1;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int col = n0 + (j & 3) + tx * 4 + (j >> 2) * 64;
                acc[i][j] *= p.scale;
                if (col < N) {
                    m = fmaxf(m, acc[i][j]);
                    if (col == label) p.zt[br] = acc[i][j];
                }
            }
#pragma unroll
            for (int o = 8; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
            float s = 0.f;
            const float base = sum_base(m);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int col = n0 + (j & 3) + tx * 4 + (j >> 2) * 64;
                if (col < N) s += expf(acc[i][j] - base);
            }
#pragma unroll
            for (int o = 8; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
            if (tx == 0 && rin) p.pairs[(b * nt + tile) * M + row] = make_float2(m, s);
        } else if (MODE == kProb) {
            if (!rin) continue;
            const int label = p.ids[br];
            const bool has = label >= 0 && label < p.K;
            const float w = p.w[br] * fac * (kShifts<T> ? pow2f(row_shift(exponent_of(p.wmax[kMaxW]), p.w[br])) : 1.f), lse = p.lse[br];
            T *Pr = static_cast<T *>(p.P) + br * p.ldp;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int col = n0 + (j & 3) + tx * 4 + (j >> 2) * 64;
                if (col < N) {
                    const float q = expf(fmaf(p.scale, acc[i][j], -lse)) - (p.k0 + col == label ? 1.f : 0.f);
                    Pr[col] = Cvt<T>::from_f(has ? w * q : 0.f);
                }
            }
        } else {
            if (!rin) continue;
            const float back = kShifts<T> && p.splits == 1 ? out_shift(p, br) : 1.f;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int col = n0 + (j & 3) + tx * 4 + (j >> 2) * 64;
                if (col >= N) continue;
                const int64_t at = br * N + col;
                if (p.splits > 1) {
                    p.out32[(split * nb * M) * N + at] = acc[i][j];
                } else {
                    const float v = acc[i][j] * (inv * back) + (p.acc ? p.acc[at] : 0.f);
                    if (p.out32) p.out32[at] = v;
                    else static_cast<T *>(p.outT)[at] = Cvt<T>::from_f(v);
                }
            }
        }
    }
}

// ------------------------------------------------------------------ small kernels around them

// loss and lse from the per-tile pairs: 32 rows x 8 slices of the tiles per block. The row's maximum
// first, then the sums against it; slices and tiles are joined in a fixed order.
__global__ void __launch_bounds__(256)
    lse_join_kernel(const float2 *__restrict__ pairs, const float *__restrict__ zt, const int32_t *__restrict__ ids,
                    int64_t B, int N, int K, int tiles, float *__restrict__ loss, float *__restrict__ lse) {
    __shared__ float part[8][32];
    const int x = threadIdx.x & 31, q = threadIdx.x >> 5;
    const int64_t per = (N + 31) / 32;
    const int64_t b = blockIdx.x / per;
    const int row = static_cast<int>(blockIdx.x % per) * 32 + x;
    const bool in = row < N;
    const float2 *pr = pairs + b * tiles * N + row;
    float m = -INFINITY;
    if (in)
#pragma unroll 8
        for (int t = q; t < tiles; t += 8) m = fmaxf(m, pr[static_cast<int64_t>(t) * N].x);
    part[q][x] = m;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 8; ++i) m = fmaxf(m, part[i][x]);
    __syncthreads();
    // Each addition's rounding is carried to the next: over many tiles of alike sums it has one direction (2^24 table
    // rows: lse off by 1.2e-4).
    float s = 0.f, lost = 0.f;
    if (in)
#pragma unroll 8
        for (int t = q; t < tiles; t += 8) {
            const float2 v = pr[static_cast<int64_t>(t) * N];
            const float term = v.y * (v.x == m ? 1.f : expf(v.x - m)) - lost;      // (equal infinities)
            const float sum = s + term;
            lost = (sum - s) - term;
            s = sum;
        }
    part[q][x] = s;
    __syncthreads();
    if (q == 0 && in) {
#pragma unroll
        for (int i = 1; i < 8; ++i) s += part[i][x];
        const float l = s == 0.f ? m : m + logf(s);     // (0: all logits at the ends of fp32, or masked)
        const int64_t at = b * N + row;
        const int id = ids[at];
        if (lse) lse[at] = l;
        if (loss) loss[at] = id >= 0 && id < K ? l - zt[at] : 0.f;
    }
}

// w[b,n] = g[b,n] * scale, 0 without a label; with wmax the bits of max |w| and, wanted, of min |w| > 0 (order of the
// atomics does not matter to a maximum).
__global__ void __launch_bounds__(256)
    weight_kernel(const float *__restrict__ g, const int32_t *__restrict__ ids, int64_t rows, int K, float scale,
                  float *__restrict__ w, unsigned int *__restrict__ wmax, bool want_min) {
    const int64_t i = blockIdx.x * 256ll + threadIdx.x;
    float v = 0.f;
    if (i < rows) {
        const int id = ids[i];
        if (id >= 0 && id < K) v = (g ? g[i] : 1.f) * scale;
        w[i] = v;
    }
    if (wmax) {
        // (a weight that is not finite spoils its own terms only)
        const unsigned int m = __reduce_max_sync(0xffffffffu, isfinite(v) ? __float_as_uint(fabsf(v)) : 0u);
        if ((threadIdx.x & 31) == 0 && m) atomicMax(wmax + kMaxW, m);
        if (want_min) {
            const unsigned int least = __reduce_max_sync(0xffffffffu, isfinite(v) && v != 0.f ? ~__float_as_uint(fabsf(v)) : 0u);
            if ((threadIdx.x & 31) == 0 && least) atomicMax(wmax + kMinW, least);
        }
    }
}

// The largest |x| of the points with a label, infinities left out; only where weights differ at all.
__global__ void __launch_bounds__(256)
    max_point_kernel(const __half *__restrict__ X, const int32_t *__restrict__ ids, int64_t rows, int d, int K,
                     unsigned int *__restrict__ stat) {
    if (!any_shift(stat)) return;
    uint32_t m = 0;
    for (int64_t r = blockIdx.x; r < rows; r += gridDim.x) {
        const int id = ids[r];
        if (id < 0 || id >= K) continue;
        for (int c = threadIdx.x; c < d; c += 256) {
            const float v = fabsf(__half2float(X[r * d + c]));
            if (v < INFINITY) m = max(m, __float_as_uint(v));
        }
    }
    m = __reduce_max_sync(0xffffffffu, m);
    if ((threadIdx.x & 31) == 0 && m) atomicMax(stat + kMaxX, m);
}

// The points as dC sums them: X 2^(q - h), rows without a label zeros; [rows, d] to rows of `per`
// units of V values: eight, or one where rows are no whole 16-byte units.
template <int V>
__global__ void __launch_bounds__(256)
    shift_points_kernel(const __half *__restrict__ X, const int32_t *__restrict__ ids, const float *__restrict__ w,
                        int64_t rows, int d, FastDiv per, int K, const unsigned int *__restrict__ stat,
                        __half *__restrict__ dst) {
    struct alignas(2 * V) Unit {
        __half v[V];
    };
    const int q = point_shift(stat), max_exp = exponent_of(stat[kMaxW]);
    for (int64_t i = blockIdx.x * 256ll + threadIdx.x; i < rows * per.d; i += gridDim.x * 256ll) {
        const int64_t r = fd_div64(per, i);
        const int c = static_cast<int>(i - r * per.d) * V, id = ids[r];
        Unit u = {};
        if (id >= 0 && id < K && c < d) {
            u = *reinterpret_cast<const Unit *>(X + r * d + c);
            const int e = q - row_shift(max_exp, w[r]);
            if (e) {
                const float f = pow2f(e);
#pragma unroll
                for (int k = 0; k < V; ++k) u.v[k] = __float2half_rn(__half2float(u.v[k]) * f);
            }
        }
        reinterpret_cast<Unit *>(dst)[i] = u;
    }
}

// Rows of src [rows, d] to dst [rows, dp] (dp >= d, the rest zeros); with ids, rows without a
// label become zeros, so that whatever they hold cannot reach a sum over rows.
// U is the unit of copying: T, or uint4 where rows are whole 16-byte units and dp == d (both counted
// in units).
template <typename U>
__global__ void __launch_bounds__(256)
    copy_rows_kernel(const U *__restrict__ src, const int32_t *__restrict__ ids, int64_t rows, int d, FastDiv dp, int K,
                     U *__restrict__ dst) {
    // rows in slices whose units number less than 2^31
    const int64_t slice = ((int64_t{1} << 31) - 1) / dp.d;
    for (int64_t r0 = 0; r0 < rows; r0 += slice) {
        const uint32_t total = static_cast<uint32_t>(min(slice, rows - r0)) * dp.d;
        for (uint64_t i = blockIdx.x * 256ull + threadIdx.x; i < total; i += gridDim.x * 256ull) {
            const uint32_t r = fd_div(dp, static_cast<uint32_t>(i)), c = static_cast<uint32_t>(i) - r * dp.d;
            bool keep = c < static_cast<uint32_t>(d);
            if (ids && keep) {
                const int id = ids[r0 + r];
                keep = id >= 0 && id < K;
            }
            U v = {};
            if (keep) v = src[(r0 + r) * d + c];
            dst[r0 * dp.d + i] = v;
        }
    }
}

// Joins the splits of a product in split order; adds acc, scales back, writes fp32 or T: V values at a time, of one
// row (8192 x 256 in two splits, under the profiler: 12 us value by value, with a row's factor 15, four at a time 8).
template <typename T, int V>
__global__ void __launch_bounds__(256)
    split_join_kernel(const float *__restrict__ parts, int splits, int64_t units, FastDiv units_per_row, Epi p) {
    struct alignas(4 * V) F {
        float v[V];
    };
    struct alignas(sizeof(T) * V) O {
        T v[V];
    };
    const float inv = p_factor(p.wmax, p.pscale, true);
    for (int64_t i = blockIdx.x * 256ll + threadIdx.x; i < units; i += gridDim.x * 256ll) {
        F s = {};
        for (int k = 0; k < splits; ++k) {
            const F x = reinterpret_cast<const F *>(parts)[k * units + i];
#pragma unroll
            for (int j = 0; j < V; ++j) s.v[j] += x.v[j];
        }
        const float f = inv * (kShifts<T> ? out_shift(p, p.rows ? fd_div64(units_per_row, i) : 0) : 1.f);
        F a = {};
        if (p.acc) a = reinterpret_cast<const F *>(p.acc)[i];
        O o;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            s.v[j] = s.v[j] * f + a.v[j];
            o.v[j] = Cvt<T>::from_f(s.v[j]);
        }
        if (p.out32) reinterpret_cast<F *>(p.out32)[i] = s;
        else static_cast<O *>(p.outT)[i] = o;
    }
}

}  // namespace xe
}  // namespace km
