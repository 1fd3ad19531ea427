// km_matvec4.cu -- products with weights held as 4-bit codes of per-row codebooks.
//
//   y[m,r] = sum_n s[r, n / group] * T(C[r, code[r,n]]) * x[m,n]
//
// T() rounds a codebook value to x's dtype, as the assignment rounds its centroids; the products
// with the group scales and all sums are fp32. Two codes share a byte (even position in the low
// half); rows are padded to 16 bytes so that every row starts on a vector boundary.
#include "km_common.cuh"
#include "km_host.h"

namespace km {
namespace mv4 {

constexpr int kKmax = 16;

// codes [R,N] -> packed [R, pitch]; one thread per 16 bytes (32 codes), padding codes 0.
__global__ void __launch_bounds__(256)
    pack4_kernel(const uint8_t *__restrict__ codes, int64_t R, int64_t N, int64_t chunks, uint4 *__restrict__ packed) {
    const int64_t u = blockIdx.x * 256ll + threadIdx.x;
    if (u >= R * chunks) return;
    const int64_t r = u / chunks, n0 = (u - r * chunks) * 32;
    const uint8_t *src = codes + r * N + n0;
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        w[i] = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (n0 + i * 8 + j < N) w[i] |= static_cast<uint32_t>(src[i * 8 + j] & 15) << (4 * j);
    }
    packed[u] = make_uint4(w[0], w[1], w[2], w[3]);
}

// CUDA-core form: one warp per row, eight consecutive codes per lane and step. The row's 16
// codebook values lie in 16 different banks, so the 32 lanes' lookups never conflict.
constexpr int kSimtWarps = 4;

template <typename T, int MT>
__global__ void __launch_bounds__(32 * kSimtWarps)
    matvec4_simt_kernel(const T *__restrict__ x, int64_t M, const uint8_t *__restrict__ packed, int64_t pitch,
                        const float *__restrict__ C, int64_t R, int N, int K, const float *__restrict__ scales,
                        int group, int ngroups, bool xvec, T *__restrict__ y) {
    __shared__ float tab[kSimtWarps][kKmax];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t r = static_cast<int64_t>(blockIdx.x) * kSimtWarps + warp;
    if (r >= R) return;
    if (lane < kKmax) tab[warp][lane] = lane < K ? round_through<T>(C[r * K + lane]) : 0.f;
    __syncwarp();
    const uint32_t *row = reinterpret_cast<const uint32_t *>(packed + r * pitch);
    const float *srow = scales ? scales + r * ngroups : nullptr;
    for (int64_t m0 = 0; m0 < M; m0 += MT) {
        float acc[MT];
#pragma unroll
        for (int m = 0; m < MT; ++m) acc[m] = 0.f;
#pragma unroll 2
        for (int n = lane * 8; n < N; n += 256) {
            const uint32_t w = row[n >> 3];
            float part[MT];
#pragma unroll
            for (int m = 0; m < MT; ++m) part[m] = 0.f;
            const bool whole = xvec && n + 8 <= N;
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                if (m0 + m >= M) continue;
                const T *xr = x + (m0 + m) * N + n;
                if (whole) {
                    struct alignas(sizeof(T) * 4) V4 { T v[4]; };
                    const V4 a = *reinterpret_cast<const V4 *>(xr), b = *reinterpret_cast<const V4 *>(xr + 4);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        part[m] = fmaf(tab[warp][(w >> (4 * j)) & 15], Cvt<T>::to_f(a.v[j]), part[m]);
                        part[m] = fmaf(tab[warp][(w >> (4 * j + 16)) & 15], Cvt<T>::to_f(b.v[j]), part[m]);
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        if (n + j < N) part[m] = fmaf(tab[warp][(w >> (4 * j)) & 15], Cvt<T>::to_f(xr[j]), part[m]);
                }
            }
            const float s = srow ? srow[n / group] : 1.f;
#pragma unroll
            for (int m = 0; m < MT; ++m) acc[m] = fmaf(s, part[m], acc[m]);
        }
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            const float t = warp_sum(acc[m]);
            if (lane == 0 && m0 + m < M) y[(m0 + m) * R + r] = Cvt<T>::from_f(t);
        }
    }
}

// ------------------------------------------------------------------ 16-bit tokens: mma form
//
// One block per 16 rows of weights. The product runs as m16n8k16 matrix instructions with the weights
// as the row operand: their rate is far above what the codes' bytes need, so eight tokens cost
// what one costs, and what bounds the kernel is turning codes into operands. That takes one
// shared-memory read per pair of codes: a byte indexes a 256-entry table of value pairs. A table
// row is 128 bytes, one word per lane, so every lane reads its own bank (lane l of a fragment
// serves rows l / 4 and l / 4 + 8, whose tables are repeated for the four lanes of a row): 32
// pairs per clock and SM whatever the codes are.
//
// Within a block of 4 * CH consecutive codes, lane t of a row holds the CH codes from t * CH on (one
// vector load), and instruction j multiplies its codes 4j .. 4j + 3 with the same positions of
// x: the order of the reduction index inside an instruction is free. CH is the largest of 32, 16
// and 8 for which a block lies in one scale group, so a scale multiplies an fp32 sum, never a
// weight.
constexpr int kMmaWarps = 8;
constexpr int kMmaThreads = 32 * kMmaWarps;
constexpr uint32_t kTabBytes = 256 * 256;      // [entry][row half][lane] words

struct MmaParams {
    const uint8_t *packed;
    const float *C, *scales;
    int64_t pitch, R, M;
    int N, K, ngroups, blocks;   // blocks of 4 * CH codes per row
    FastDiv bpg;                 // blocks per scale group
    int xvec;                    // rows of x start on 16-byte boundaries
};

template <typename T>
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1);
template <>
__device__ __forceinline__ void mma16816<__half>(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <>
__device__ __forceinline__ void mma16816<__nv_bfloat16>(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <typename T> __device__ __forceinline__ uint32_t bits16(T v) {
    return *reinterpret_cast<const uint16_t *>(&v);
}

// CH codes (CH / 8 words) at p.
template <int CH> struct Codes {
    uint32_t w[CH / 8];
};
template <int CH> __device__ __forceinline__ Codes<CH> load_codes(const uint8_t *p) {
    Codes<CH> c;
    if constexpr (CH == 32) {
        const uint4 v = __ldcs(reinterpret_cast<const uint4 *>(p));
        c.w[0] = v.x, c.w[1] = v.y, c.w[2] = v.z, c.w[3] = v.w;
    } else if constexpr (CH == 16) {
        const uint2 v = __ldcs(reinterpret_cast<const uint2 *>(p));
        c.w[0] = v.x, c.w[1] = v.y;
    } else {
        c.w[0] = __ldg(reinterpret_cast<const uint32_t *>(p));
    }
    return c;
}

template <typename T, int CH, int NT>
__global__ void __launch_bounds__(kMmaThreads, NT == 1 ? 3 : 2)
    matvec4_mma_kernel(const T *__restrict__ x, const MmaParams p, T *__restrict__ y) {
    extern __shared__ __align__(16) uint8_t tab[];
    __shared__ float red[kMmaWarps][16][8 * NT + 1];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = lane >> 2, t = lane & 3;
    const int64_t r0 = static_cast<int64_t>(blockIdx.x) * 16;
    const int64_t m0 = static_cast<int64_t>(blockIdx.y) * (8 * NT);
    // rows behind the last one repeat it; their sums are not written
    const int64_t ra = min(r0 + g, p.R - 1), rb = min(r0 + g + 8, p.R - 1);
    const uint8_t *pa = p.packed + ra * p.pitch, *pb = p.packed + rb * p.pitch;
    const int chunk0 = t * CH;
    auto in_row = [&](int blk) { return blk < p.blocks && blk * (4 * CH) + chunk0 < p.N; };
    Codes<CH> ca = {}, cb = {};
    if (in_row(warp)) {
        ca = load_codes<CH>(pa + (static_cast<int64_t>(warp) * (4 * CH) + chunk0) / 2);
        cb = load_codes<CH>(pb + (static_cast<int64_t>(warp) * (4 * CH) + chunk0) / 2);
    }
    {
        // pair tables: this thread's row, the 16 entries with high code `hi`
        const int row = threadIdx.x & 15, hi = threadIdx.x >> 4;
        const float *Cr = p.C + min(r0 + row, p.R - 1) * p.K;
        uint32_t v[16];
#pragma unroll
        for (int k = 0; k < 16; ++k) v[k] = k < p.K ? bits16(Cvt<T>::from_f(Cr[k])) : 0u;
        uint32_t vh = 0;
#pragma unroll
        for (int k = 0; k < 16; ++k)
            if (k == hi) vh = v[k] << 16;
#pragma unroll
        for (int k = 0; k < 16; ++k) {
            const uint32_t e = v[k] | vh;
            *reinterpret_cast<uint4 *>(tab + (hi * 16 + k) * 256 + (row >> 3) * 128 + (row & 7) * 16) = make_uint4(e, e, e, e);
        }
    }
    __syncthreads();
    float tot[NT][4];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) tot[n][i] = 0.f;
    const T *xr[NT];
    bool xin[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        xin[n] = m0 + n * 8 + g < p.M;
        xr[n] = x + (m0 + n * 8 + g) * p.N;
    }
    const uint32_t lane4 = lane * 4;
    const float *sa = p.scales ? p.scales + ra * p.ngroups : nullptr, *sb = p.scales ? p.scales + rb * p.ngroups : nullptr;
    for (int blk = warp; blk < p.blocks; blk += kMmaWarps) {
        const int n0 = blk * (4 * CH) + chunk0;
        const Codes<CH> a = ca, b = cb;
        if (in_row(blk + kMmaWarps)) {
            ca = load_codes<CH>(pa + (static_cast<int64_t>(blk + kMmaWarps) * (4 * CH) + chunk0) / 2);
            cb = load_codes<CH>(pb + (static_cast<int64_t>(blk + kMmaWarps) * (4 * CH) + chunk0) / 2);
        }
        float s0 = 1.f, s1 = 1.f;
        if (sa) {
            const int gi = fd_div(p.bpg, blk);
            s0 = sa[gi];
            s1 = sb[gi];
        }
        const bool whole = (blk + 1) * (4 * CH) <= p.N;      // the same for the whole warp
        float acc[NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[n][i] = 0.f;
#pragma unroll
        for (int h = 0; h < CH / 8; ++h) {       // eight codes, two instructions
            uint32_t xb[NT][4];
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const int at = n0 + h * 8;
#pragma unroll
                for (int i = 0; i < 4; ++i) xb[n][i] = 0;
                if (xin[n]) {
                    if (whole && p.xvec) {
                        const uint4 v = __ldg(reinterpret_cast<const uint4 *>(xr[n] + at));
                        xb[n][0] = v.x, xb[n][1] = v.y, xb[n][2] = v.z, xb[n][3] = v.w;
                    } else {
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            if (at + 2 * i < p.N) xb[n][i] = bits16(xr[n][at + 2 * i]);
                            if (at + 2 * i + 1 < p.N) xb[n][i] |= bits16(xr[n][at + 2 * i + 1]) << 16;
                        }
                    }
                }
            }
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                uint32_t f[4];
                // table offset of a byte: the byte as bits 8-15, the lane's word below it
                f[0] = *reinterpret_cast<const uint32_t *>(tab + __byte_perm(a.w[h], lane4, 0x7704 | (2 * j) << 4));
                f[1] = *reinterpret_cast<const uint32_t *>(tab + 128 + __byte_perm(b.w[h], lane4, 0x7704 | (2 * j) << 4));
                f[2] = *reinterpret_cast<const uint32_t *>(tab + __byte_perm(a.w[h], lane4, 0x7704 | (2 * j + 1) << 4));
                f[3] = *reinterpret_cast<const uint32_t *>(tab + 128 + __byte_perm(b.w[h], lane4, 0x7704 | (2 * j + 1) << 4));
                if (!whole) {
                    // codes behind the row's end are no weights (a codebook value may be infinite)
                    const int at = n0 + h * 8 + 4 * j;
                    if (at >= p.N) f[0] = f[1] = 0;
                    else if (at + 1 >= p.N) f[0] &= 0xffff, f[1] &= 0xffff;
                    if (at + 2 >= p.N) f[2] = f[3] = 0;
                    else if (at + 3 >= p.N) f[2] &= 0xffff, f[3] &= 0xffff;
                }
#pragma unroll
                for (int n = 0; n < NT; ++n) mma16816<T>(acc[n], f, xb[n][2 * j], xb[n][2 * j + 1]);
            }
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            tot[n][0] = fmaf(s0, acc[n][0], tot[n][0]);
            tot[n][1] = fmaf(s0, acc[n][1], tot[n][1]);
            tot[n][2] = fmaf(s1, acc[n][2], tot[n][2]);
            tot[n][3] = fmaf(s1, acc[n][3], tot[n][3]);
        }
    }
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        red[warp][g][n * 8 + 2 * t] = tot[n][0];
        red[warp][g][n * 8 + 2 * t + 1] = tot[n][1];
        red[warp][g + 8][n * 8 + 2 * t] = tot[n][2];
        red[warp][g + 8][n * 8 + 2 * t + 1] = tot[n][3];
    }
    __syncthreads();
    for (int i = threadIdx.x; i < 16 * 8 * NT; i += kMmaThreads) {
        const int r = i & 15, m = i >> 4;
        float v = 0.f;
#pragma unroll
        for (int w = 0; w < kMmaWarps; ++w) v += red[w][r][m];
        if (r0 + r < p.R && m0 + m < p.M) y[(m0 + m) * p.R + r0 + r] = Cvt<T>::from_f(v);
    }
}

}  // namespace mv4
}  // namespace km

namespace {

using namespace km::mv4;

inline int64_t pitch_of(int64_t N) { return ceil_div(N, 32) * 16; }

template <typename T>
km_status matvec4_simt(const void *xv, int64_t M, const uint8_t *packed, const float *C, int64_t R, int64_t N,
                       int64_t K, const float *scales, int64_t group, void *yv, cudaStream_t st) {
    const T *x = static_cast<const T *>(xv);
    T *y = static_cast<T *>(yv);
    const int ng = scales ? static_cast<int>(ceil_div(N, group)) : 0;
    const bool xvec = N % 4 == 0 && aligned(x, 4 * sizeof(T));
    const unsigned grid = static_cast<unsigned>(ceil_div(R, kSimtWarps));
    const int g = static_cast<int>(group), Ni = static_cast<int>(N), Ki = static_cast<int>(K);
    if (M == 1)
        matvec4_simt_kernel<T, 1><<<grid, 32 * kSimtWarps, 0, st>>>(x, M, packed, pitch_of(N), C, R, Ni, Ki, scales, g, ng, xvec, y);
    else
        matvec4_simt_kernel<T, 4><<<grid, 32 * kSimtWarps, 0, st>>>(x, M, packed, pitch_of(N), C, R, Ni, Ki, scales, g, ng, xvec, y);
    return launch_status();
}

template <typename T, int CH, int NT>
km_status mma_launch(const T *x, MmaParams p, T *y, cudaStream_t st) {
    auto kernel = matvec4_mma_kernel<T, CH, NT>;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kTabBytes)) !=
        cudaSuccess)
        return KM_ERR_CUDA;
    // token tiles beyond the grid's y extent in further launches
    const int64_t per = static_cast<int64_t>(kMaxGridY) * 8 * NT, M = p.M;
    for (int64_t m0 = 0; m0 < M; m0 += per) {
        p.M = std::min(per, M - m0);
        const dim3 grid(static_cast<unsigned>(ceil_div(p.R, 16)), static_cast<unsigned>(ceil_div(p.M, 8 * NT)));
        kernel<<<grid, kMmaThreads, kTabBytes, st>>>(x + m0 * p.N, p, y + m0 * p.R);
        if (launch_status() != KM_OK) return KM_ERR_CUDA;
    }
    return KM_OK;
}
template <typename T, int CH>
km_status mma_tokens(const T *x, MmaParams p, T *y, cudaStream_t st) {
    p.blocks = static_cast<int>(ceil_div(p.N, 4 * CH));
    if (p.M <= 8) return mma_launch<T, CH, 1>(x, p, y, st);
    if (p.M <= 16) return mma_launch<T, CH, 2>(x, p, y, st);
    return mma_launch<T, CH, 4>(x, p, y, st);
}
template <typename T>
km_status matvec4_mma(const void *xv, int64_t M, const uint8_t *packed, const float *C, int64_t R, int64_t N,
                      int64_t K, const float *scales, int64_t group, void *yv, cudaStream_t st) {
    const T *x = static_cast<const T *>(xv);
    T *y = static_cast<T *>(yv);
    MmaParams p = {};
    p.packed = packed;
    p.C = C;
    p.scales = scales;
    p.pitch = pitch_of(N);
    p.R = R;
    p.M = M;
    p.N = static_cast<int>(N);
    p.K = static_cast<int>(K);
    p.ngroups = scales ? static_cast<int>(ceil_div(N, group)) : 0;
    p.xvec = N % 8 == 0 && aligned(x, 16) ? 1 : 0;
    const int ch = !scales || group % 128 == 0 ? 32 : group % 64 == 0 ? 16 : 8;
    p.bpg = km::make_fastdiv(static_cast<uint32_t>(scales ? group / (4 * ch) : 1));
    switch (ch) {
        case 32: return mma_tokens<T, 32>(x, p, y, st);
        case 16: return mma_tokens<T, 16>(x, p, y, st);
        default: return mma_tokens<T, 8>(x, p, y, st);
    }
}

}  // namespace

extern "C" {

km_status km_pack4(const uint8_t *codes, int64_t R, int64_t N, uint8_t *packed, void *stream) {
    if (!codes || !packed || !sizes_ok(R, N, 1, 1) || N > kMaxIndex - 256 || !aligned(packed, 16)) return KM_ERR_INVALID_ARG;
    const int64_t chunks = ceil_div(N, 32), blocks = ceil_div(R * chunks, 256);
    if (blocks > kMaxIndex) return KM_ERR_UNSUPPORTED;
    pack4_kernel<<<static_cast<unsigned>(blocks), 256, 0, S(stream)>>>(codes, R, N, chunks,
                                                                       reinterpret_cast<uint4 *>(packed));
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
        case KM_F32: return matvec4_simt<float>(x, M, packed, C, R, N, K, scales, group, y, S(stream));
        case KM_F16: return matvec4_mma<__half>(x, M, packed, C, R, N, K, scales, group, y, S(stream));
        default: return matvec4_mma<__nv_bfloat16>(x, M, packed, C, R, N, K, scales, group, y, S(stream));
    }
}

}  // extern "C"
