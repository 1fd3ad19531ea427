// km_host.h -- host helpers shared by the translation units of libkmeans_b200: argument checks,
// workspace carving, device queries, the tensor-map encoder.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cstddef>
#include <cstdint>

#include "kmeans_b200.h"

// Test-only switch of the codebook operators (km_debug_inject(3)): handed to their kernels as a parameter, so that
// it costs nothing where it is off.
namespace km {
inline std::atomic<int> g_withhold{0};
}  // namespace km

// The device error word and the wait limit of km_common.cuh exist once per translation unit; the
// other units that wait export theirs for km_device_error and km_debug_wait_limit.
namespace km {
namespace xe {
cudaError_t take_device_error(unsigned int *bits);            // reads and clears
cudaError_t set_wait_limit(unsigned long long limit_ns);
}  // namespace xe
namespace mv4 {
cudaError_t take_device_error(unsigned int *bits);
cudaError_t set_wait_limit(unsigned long long limit_ns);
}  // namespace mv4
}  // namespace km

namespace {

constexpr size_t kAlign = 256;
constexpr int64_t kMaxIndex = (int64_t{1} << 31) - 1;
constexpr int64_t kMaxD = int64_t{1} << 20;
constexpr int kMaxGridY = 65535;

inline size_t align_up(size_t x) { return (x + kAlign - 1) & ~(kAlign - 1); }
inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
inline cudaStream_t S(void *s) { return reinterpret_cast<cudaStream_t>(s); }

inline bool valid_dtype(km_dtype dt) { return dt == KM_F32 || dt == KM_F16 || dt == KM_BF16; }
inline size_t dtype_size(km_dtype dt) { return dt == KM_F32 ? 4 : 2; }

inline bool sizes_ok(int64_t B, int64_t N, int64_t K, int64_t d) {
    return B >= 1 && N >= 1 && K >= 1 && d >= 1 && B <= kMaxIndex && N <= kMaxIndex &&
           K <= kMaxIndex && d <= kMaxD && B * N <= (int64_t{1} << 40) &&
           B * K <= (int64_t{1} << 40);
}

struct Carver {
    uint8_t *base;
    size_t off = 0;
    explicit Carver(void *b) : base(static_cast<uint8_t *>(b)) {}
    template <typename P> P *take(size_t bytes) {
        P *p = base ? reinterpret_cast<P *>(base + off) : nullptr;
        off += align_up(bytes);
        return p;
    }
};

inline int num_sms() {
    static int cache[64] = {0};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 148;
    if (dev >= 0 && dev < 64 && cache[dev]) return cache[dev];
    int n = 148;
    cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
    if (dev >= 0 && dev < 64) cache[dev] = n;
    return n;
}

typedef CUresult (*EncodeTiledFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                                  const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                                  const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline EncodeTiledFn encode_fn() {
    static EncodeTiledFn fn = nullptr;
    if (!fn) {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeTiledFn>(p);
    }
    return fn;
}

// Raises a kernel's limit of dynamic shared memory, once per kernel and device (`done` is a static of
// the kernel's launcher: one bit per device).
template <typename Kernel> inline bool allow_smem(Kernel kernel, size_t bytes, std::atomic<uint64_t> &done) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return false;
    const uint64_t bit = dev >= 0 && dev < 64 ? uint64_t{1} << dev : 0;
    if (bit && (done.load(std::memory_order_relaxed) & bit)) return true;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(bytes)) != cudaSuccess)
        return false;
    done.fetch_or(bit, std::memory_order_relaxed);
    return true;
}

inline km_status launch_status() {
    return cudaGetLastError() == cudaSuccess ? KM_OK : KM_ERR_CUDA;
}

}  // namespace
