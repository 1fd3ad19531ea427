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

}  // namespace mv4
}  // namespace km

namespace {

using namespace km::mv4;

inline int64_t pitch_of(int64_t N) { return ceil_div(N, 32) * 16; }

template <typename T>
km_status matvec4_typed(const void *xv, int64_t M, const uint8_t *packed, const float *C, int64_t R, int64_t N,
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
        case KM_F32: return matvec4_typed<float>(x, M, packed, C, R, N, K, scales, group, y, S(stream));
        case KM_F16: return matvec4_typed<__half>(x, M, packed, C, R, N, K, scales, group, y, S(stream));
        default: return matvec4_typed<__nv_bfloat16>(x, M, packed, C, R, N, K, scales, group, y, S(stream));
    }
}

}  // extern "C"
