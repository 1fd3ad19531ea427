// km_lookup.cu -- reading a table back by ids, and the table's gradient.
//
//   km_lookup       Y[b,n,:]  = scale * C[b, ids[b,n], :]
//   km_lookup_grad  dC[b,k,:] = scale * sum over the n with ids[b,n] = k of dY[b,n,:]
//
// Both move memory and compute next to nothing. The gradient is the transposed access: instead of
// one atomic per token and coordinate, whose order would change the rounding from run to run, the
// tokens are sorted by id (stable, so equal ids keep their order) and every row is the sum of one
// contiguous run of the sorted order, always added in the same order.
#include "km_common.cuh"
#include "km_host.h"

namespace km {
namespace lk {

// V consecutive elements of T as one access.
template <typename T, int V> struct alignas(sizeof(T) * V) Vec {
    T v[V];
};
template <typename T, int V> __device__ __forceinline__ Vec<T, V> load_ro(const Vec<T, V> *p) {
    constexpr int kBytes = sizeof(T) * V;
    Vec<T, V> r;
    if constexpr (kBytes == 16) *reinterpret_cast<uint4 *>(&r) = __ldg(reinterpret_cast<const uint4 *>(p));
    else if constexpr (kBytes == 8) *reinterpret_cast<uint2 *>(&r) = __ldg(reinterpret_cast<const uint2 *>(p));
    else if constexpr (kBytes == 4) *reinterpret_cast<uint32_t *>(&r) = __ldg(reinterpret_cast<const uint32_t *>(p));
    else *reinterpret_cast<uint16_t *>(&r) = __ldg(reinterpret_cast<const uint16_t *>(p));
    return r;
}

// Streaming store: the result is written once and would only push the table out of L2.
template <typename T, int V> __device__ __forceinline__ void store_cs(Vec<T, V> *p, Vec<T, V> r) {
    constexpr int kBytes = sizeof(T) * V;
    if constexpr (kBytes == 16) __stcs(reinterpret_cast<uint4 *>(p), *reinterpret_cast<uint4 *>(&r));
    else if constexpr (kBytes == 8) __stcs(reinterpret_cast<uint2 *>(p), *reinterpret_cast<uint2 *>(&r));
    else if constexpr (kBytes == 4) __stcs(reinterpret_cast<uint32_t *>(p), *reinterpret_cast<uint32_t *>(&r));
    else __stcs(reinterpret_cast<uint16_t *>(p), *reinterpret_cast<uint16_t *>(&r));
}

// ------------------------------------------------------------------ lookup

constexpr int kLookupThreads = 256;

// A warp serves `rpw` consecutive rows (at most 32): each lane finds one row's source once, then
// the rows are moved 32 / TPR at a time, TPR lanes (a power of two) per row and V elements per lane,
// with 2 rows (4 pieces of a wide row) in flight
// per lane: more registers per thread cost more in resident warps than they hide (8: 122 us, 4: 91,
// 2: 87 for 2M rows of 256 bytes). Off is the type of offsets counted in units of V elements: 32 bits
// wherever table and output have fewer units than 2^32, which halves the address arithmetic that
// otherwise costs more than the conversion of the values.
template <typename T, int V, int TPR, typename Off>
__global__ void __launch_bounds__(kLookupThreads)
    lookup_kernel(const T *__restrict__ C, const int32_t *__restrict__ ids, uint32_t rows, FastDiv divN,
                  uint32_t K, uint32_t units, int rpw, float scale, T *__restrict__ Y) {
    constexpr int RS = 32 / TPR, U = 2, UW = 4;
    constexpr Off kNone = ~Off(0);
    using Unit = Vec<T, V>;
    const int lane = threadIdx.x & 31, sub = lane / TPR, t = lane % TPR;
    const uint32_t row0 = (blockIdx.x * (kLookupThreads / 32) + (threadIdx.x >> 5)) * static_cast<uint32_t>(rpw);
    if (row0 >= rows) return;
    const int n = min(static_cast<uint32_t>(rpw), rows - row0);
    Off src = kNone;
    if (lane < n) {
        const uint32_t id = static_cast<uint32_t>(ids[row0 + lane]);
        if (id < K) src = (static_cast<Off>(fd_div(divN, row0 + lane)) * K + id) * units;
    }
    const Unit *Cu = reinterpret_cast<const Unit *>(C);
    Unit *Yu = reinterpret_cast<Unit *>(Y) + static_cast<Off>(row0) * units;
    auto scaled = [&](Unit v) {
#pragma unroll
        for (int i = 0; i < V; ++i) v.v[i] = Cvt<T>::from_f(scale * Cvt<T>::to_f(v.v[i]));
        return v;
    };
    Unit zero;
#pragma unroll
    for (int i = 0; i < V; ++i) zero.v[i] = Cvt<T>::from_f(0.f);
    if (TPR < 32 || units <= 32) {
        const bool in = t < static_cast<int>(units);
        for (int j = 0; j < n; j += RS * U) {
            Unit v[U];
            Off s[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                s[u] = __shfl_sync(0xffffffffu, src, (j + u * RS + sub) & 31);
                if (j + u * RS + sub < n && in && s[u] != kNone) v[u] = load_ro(Cu + s[u] + t);
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int r = j + u * RS + sub;
                if (r < n && in) store_cs(Yu + static_cast<Off>(r) * units + t, s[u] != kNone ? scaled(v[u]) : zero);
            }
        }
    } else {
        for (int j = 0; j < n; ++j) {
            const Off s = __shfl_sync(0xffffffffu, src, j);
            Unit *out = Yu + static_cast<Off>(j) * units;
            for (uint32_t c = t; c < units; c += 32 * UW) {
                Unit v[UW];
#pragma unroll
                for (int u = 0; u < UW; ++u)
                    if (c + u * 32 < units && s != kNone) v[u] = load_ro(Cu + s + c + u * 32);
#pragma unroll
                for (int u = 0; u < UW; ++u)
                    if (c + u * 32 < units) store_cs(out + c + u * 32, s != kNone ? scaled(v[u]) : zero);
            }
        }
    }
}

// ------------------------------------------------------------------ stable radix sort by id

constexpr int kSortThreads = 256;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kSortItems = 16;
constexpr int kSortTile = kSortThreads * kSortItems;
constexpr int kBins = 256;

struct SortIn {
    const int32_t *ids;      // first pass: the ids themselves (else null)
    FastDiv divN;
    int K;
    const uint32_t *keys, *pos;   // later passes
    const uint32_t *nvalid;       // later passes: number of sorted entries
    uint32_t n;
};

// Entry i: its key (b K + id) and position; false past the end or for an id outside [0, K).
__device__ __forceinline__ bool sort_load(const SortIn &s, uint32_t n, uint32_t i, uint32_t &key,
                                          uint32_t &pos) {
    if (i >= n) return false;
    if (s.ids) {
        const int id = s.ids[i];
        pos = i;
        key = fd_div(s.divN, i) * static_cast<uint32_t>(s.K) + static_cast<uint32_t>(id);
        return id >= 0 && id < s.K;
    }
    key = s.keys[i];
    pos = s.pos[i];
    return true;
}

// Digit counts of each tile: counts[bin * tiles + tile].
__global__ void __launch_bounds__(kSortThreads)
    sort_hist_kernel(SortIn in, int shift, uint32_t tiles, uint32_t *__restrict__ counts) {
    __shared__ uint32_t bins[kBins];
    bins[threadIdx.x] = 0;
    __syncthreads();
    const uint32_t n = in.nvalid ? *in.nvalid : in.n;
    const uint32_t t0 = blockIdx.x * static_cast<uint32_t>(kSortTile);
    for (int i = 0; i < kSortItems; ++i) {
        uint32_t key, pos;
        if (sort_load(in, n, t0 + i * kSortThreads + threadIdx.x, key, pos))
            atomicAdd(&bins[(key >> shift) & (kBins - 1)], 1u);
    }
    __syncthreads();
    counts[threadIdx.x * static_cast<size_t>(tiles) + blockIdx.x] = bins[threadIdx.x];
}

// Inclusive scan over the block; *total receives the sum.
__device__ __forceinline__ uint32_t block_scan(uint32_t v, uint32_t *warp_sums, uint32_t *total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
    uint32_t x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) warp_sums[warp] = x;
    __syncthreads();
    uint32_t before = 0, all = 0;
    for (int w = 0; w < nw; ++w) {
        const uint32_t s = warp_sums[w];
        if (w < warp) before += s;
        all += s;
    }
    __syncthreads();
    *total = all;
    return x + before;
}

// One block per bin: exclusive scan of the bin's tile counts in place, its total in totals[bin].
__global__ void __launch_bounds__(kSortThreads)
    sort_scan_kernel(uint32_t tiles, uint32_t *__restrict__ counts, uint32_t *__restrict__ totals) {
    __shared__ uint32_t ws[kSortWarps];
    uint32_t *c = counts + blockIdx.x * static_cast<size_t>(tiles);
    uint32_t run = 0;
    for (uint32_t t = 0; t < tiles; t += kSortThreads) {
        const uint32_t i = t + threadIdx.x;
        const uint32_t v = i < tiles ? c[i] : 0;
        uint32_t tot;
        const uint32_t x = block_scan(v, ws, &tot);
        if (i < tiles) c[i] = run + x - v;
        run += tot;
    }
    if (threadIdx.x == 0) totals[blockIdx.x] = run;
}

// Places every entry of a tile at (bin start) + (entries of the bin in earlier tiles) + (earlier
// entries of the bin in this tile). Within a warp the rank among equal digits comes from a
// match over 32 consecutive entries, so the order of equal digits is kept.
__global__ void __launch_bounds__(kSortThreads)
    sort_scatter_kernel(SortIn in, int shift, uint32_t tiles, const uint32_t *__restrict__ counts,
                        const uint32_t *__restrict__ totals, uint32_t *__restrict__ keys_out,
                        uint32_t *__restrict__ pos_out, uint32_t *__restrict__ nvalid_out) {
    __shared__ uint32_t ws[kSortWarps];
    __shared__ uint32_t wcount[kSortWarps][kBins];
    __shared__ uint32_t base[kBins];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int w = 0; w < kSortWarps; ++w) wcount[w][threadIdx.x] = 0;
    uint32_t all;
    const uint32_t v = totals[threadIdx.x];
    const uint32_t x = block_scan(v, ws, &all);
    base[threadIdx.x] = x - v + counts[threadIdx.x * static_cast<size_t>(tiles) + blockIdx.x];
    if (nvalid_out && blockIdx.x == 0 && threadIdx.x == 0) *nvalid_out = all;
    __syncthreads();
    const uint32_t n = in.nvalid ? *in.nvalid : in.n;
    const uint32_t i0 = blockIdx.x * static_cast<uint32_t>(kSortTile) + warp * (32 * kSortItems) + lane;
    uint32_t key[kSortItems], pos[kSortItems], rank[kSortItems];
    bool ok[kSortItems];
#pragma unroll
    for (int i = 0; i < kSortItems; ++i) ok[i] = sort_load(in, n, i0 + i * 32, key[i], pos[i]);
#pragma unroll
    for (int i = 0; i < kSortItems; ++i) {
        const uint32_t digit = ok[i] ? (key[i] >> shift) & (kBins - 1) : kBins;
        const uint32_t peers = __match_any_sync(0xffffffffu, digit);
        uint32_t prior = 0;
        if (ok[i]) prior = wcount[warp][digit];
        __syncwarp();
        rank[i] = prior + __popc(peers & ((1u << lane) - 1));
        if (ok[i] && lane == __ffs(peers) - 1) wcount[warp][digit] = prior + __popc(peers);
        __syncwarp();
    }
    __syncthreads();
    {
        uint32_t run = base[threadIdx.x];
        for (int w = 0; w < kSortWarps; ++w) {
            const uint32_t c = wcount[w][threadIdx.x];
            wcount[w][threadIdx.x] = run;
            run += c;
        }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kSortItems; ++i)
        if (ok[i]) {
            const uint32_t at = wcount[warp][(key[i] >> shift) & (kBins - 1)] + rank[i];
            keys_out[at] = key[i];
            pos_out[at] = pos[i];
        }
}

// ------------------------------------------------------------------ sums over the sorted order

struct GradParams {
    const uint32_t *keys, *pos, *nvalid;
    uint32_t range;   // sorted entries per range
    int d;
    float scale;
    int accumulate;
    float *slots;     // [ranges][2][d] fp32: the range's first and last run where they go on
                      // in a neighbouring range
};

template <typename O, int V>
__device__ __forceinline__ void write_row(O *out, const float (&acc)[V], float scale, int accumulate) {
    Vec<O, V> o;
    if (accumulate) o = *reinterpret_cast<const Vec<O, V> *>(out);
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const float s = scale * acc[i];
        o.v[i] = Cvt<O>::from_f(accumulate ? Cvt<O>::to_f(o.v[i]) + s : s);
    }
    *reinterpret_cast<Vec<O, V> *>(out) = o;
}

constexpr int kGradThreads = 256;

// LPR lanes per range and column block of LPR * V columns. A range adds up the rows of its runs
// of equal keys one after the other in fp32; a run that begins and ends inside the range is
// written to its table row, the others to the range's slots.
template <typename T, typename O, int V, int LPR>
__global__ void __launch_bounds__(kGradThreads)
    grad_ranges_kernel(const T *__restrict__ dY, GradParams p, O *__restrict__ dC) {
    constexpr int GROUPS = kGradThreads / LPR;
    constexpr int U = 8;   // rows in flight per group
    const int g = threadIdx.x / LPR, t = threadIdx.x % LPR;
    const uint32_t n = *p.nvalid;
    const uint32_t r = blockIdx.x * static_cast<uint32_t>(GROUPS) + g;
    const uint64_t s64 = static_cast<uint64_t>(r) * p.range;
    if (s64 >= n) return;
    const uint32_t s = static_cast<uint32_t>(s64);
    const uint32_t e = static_cast<uint32_t>(min(static_cast<uint64_t>(n), s64 + p.range));
    const int c = (blockIdx.y * LPR + t) * V;
    if (c >= p.d) return;
    float acc[V];
#pragma unroll
    for (int i = 0; i < V; ++i) acc[i] = 0.f;
    uint32_t cur = p.keys[s];
    bool head = s > 0 && p.keys[s - 1] == cur;
    auto flush = [&](bool tail) {
        if (head || tail) {
            float *slot = p.slots + (static_cast<size_t>(r) * 2 + (head ? 0 : 1)) * p.d + c;
#pragma unroll
            for (int i = 0; i < V; ++i) slot[i] = acc[i];
        } else {
            write_row<O, V>(dC + static_cast<int64_t>(cur) * p.d + c, acc, p.scale, p.accumulate);
        }
    };
    for (uint32_t i = s; i < e; i += U) {
        uint32_t key[U];
        Vec<T, V> v[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (i + u < e) {
                key[u] = p.keys[i + u];
                v[u] = *reinterpret_cast<const Vec<T, V> *>(dY + static_cast<int64_t>(p.pos[i + u]) * p.d + c);
            }
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (i + u < e) {
                if (key[u] != cur) {
                    flush(false);
                    cur = key[u];
                    head = false;
#pragma unroll
                    for (int k = 0; k < V; ++k) acc[k] = 0.f;
                }
#pragma unroll
                for (int k = 0; k < V; ++k) acc[k] += Cvt<T>::to_f(v[u].v[k]);
            }
    }
    flush(e < n && p.keys[e] == cur);
}

// One block per range: joins, in range order, the pieces of the run that begins in this range
// and goes on in the next ones.
template <typename O, int V, int LPR>
__global__ void __launch_bounds__(kGradThreads)
    grad_join_kernel(GradParams p, O *__restrict__ dC) {
    constexpr int GROUPS = kGradThreads / LPR;
    __shared__ float part[GROUPS][LPR * V];
    const uint32_t n = *p.nvalid;
    const uint64_t s64 = static_cast<uint64_t>(blockIdx.x) * p.range;
    if (s64 + p.range >= n) return;                       // nothing follows this range
    const uint32_t s = static_cast<uint32_t>(s64), e = s + p.range;
    const uint32_t key = p.keys[e - 1];
    if (p.keys[e] != key) return;                         // its last run ends with it
    if (p.keys[s] == key && s > 0 && p.keys[s - 1] == key) return;   // the run began earlier
    uint32_t lo = e, hi = n;                              // first entry behind the run
    while (lo < hi) {
        const uint32_t mid = lo + (hi - lo) / 2;
        if (p.keys[mid] == key) lo = mid + 1; else hi = mid;
    }
    const uint32_t r0 = blockIdx.x, r1 = (lo - 1) / p.range;   // first and last range of the run
    const uint32_t len = r1 - r0 + 1, per = (len + GROUPS - 1) / GROUPS;
    const int g = threadIdx.x / LPR, t = threadIdx.x % LPR;
    for (int c0 = 0; c0 < p.d; c0 += LPR * V) {
        const int c = c0 + t * V;
        float acc[V];
#pragma unroll
        for (int i = 0; i < V; ++i) acc[i] = 0.f;
        if (c < p.d) {
            const uint32_t a = min(len, g * per), b = min(len, a + per);
#pragma unroll 4
            for (uint32_t j = a; j < b; ++j) {
                const float *slot = p.slots + (static_cast<size_t>(r0 + j) * 2 + (j == 0 ? 1 : 0)) * p.d + c;
#pragma unroll
                for (int i = 0; i < V; ++i) acc[i] += slot[i];
            }
        }
#pragma unroll
        for (int i = 0; i < V; ++i) part[g][t * V + i] = acc[i];
        __syncthreads();
        if (g == 0 && c < p.d) {
            for (int q = 1; q < GROUPS; ++q)
#pragma unroll
                for (int i = 0; i < V; ++i) acc[i] += part[q][t * V + i];
            write_row<O, V>(dC + static_cast<int64_t>(key) * p.d + c, acc, p.scale, p.accumulate);
        }
        __syncthreads();
    }
}

}  // namespace lk
}  // namespace km

namespace {

using namespace km::lk;
using km::FastDiv;
using km::make_fastdiv;

inline bool elem_ok(const void *p, km_dtype dt) { return aligned(p, dtype_size(dt)); }

// Elements per access: the widest of 16, 8, 4 bytes (or one element) that divides every row.
inline int vec_elems(int64_t d, size_t es, const void *a, const void *b) {
    for (size_t bytes = 16; bytes > es; bytes /= 2) {
        const int64_t v = static_cast<int64_t>(bytes / es);
        if (d % v == 0 && aligned(a, bytes) && aligned(b, bytes)) return static_cast<int>(v);
    }
    return 1;
}
inline int pow2_at_least(int64_t x, int cap) {
    int p = 1;
    while (p < cap && p < x) p *= 2;
    return p;
}

template <typename T, int V, int TPR>
km_status lookup_launch(const T *C, const int32_t *ids, uint32_t rows, FastDiv dv, int64_t table_rows, int K, int d,
                        float scale, T *Y, cudaStream_t st) {
    // rows per warp: 32 lets every lane look one id up, fewer where that would leave SMs without
    // warps (16 warps per SM wanted)
    int rpw = 32;
    while (rpw > 32 / TPR && ceil_div(rows, rpw) < 148 * 16) rpw /= 2;
    const unsigned grid = static_cast<unsigned>(ceil_div(ceil_div(rows, rpw), kLookupThreads / 32));
    const uint32_t units = static_cast<uint32_t>(d / V);
    constexpr int64_t kMax32 = (int64_t{1} << 32) - 1;
    if (table_rows * units < kMax32 && static_cast<int64_t>(rows) * units < kMax32)
        lookup_kernel<T, V, TPR, uint32_t><<<grid, kLookupThreads, 0, st>>>(C, ids, rows, dv, static_cast<uint32_t>(K),
                                                                            units, rpw, scale, Y);
    else
        lookup_kernel<T, V, TPR, uint64_t><<<grid, kLookupThreads, 0, st>>>(C, ids, rows, dv, static_cast<uint32_t>(K),
                                                                            units, rpw, scale, Y);
    return launch_status();
}
template <typename T, int V>
km_status lookup_tpr(const T *C, const int32_t *ids, uint32_t rows, FastDiv dv, int64_t tr, int K, int d, float scale,
                     T *Y, cudaStream_t st) {
    switch (pow2_at_least(ceil_div(d, V), 32)) {
        case 1: return lookup_launch<T, V, 1>(C, ids, rows, dv, tr, K, d, scale, Y, st);
        case 2: return lookup_launch<T, V, 2>(C, ids, rows, dv, tr, K, d, scale, Y, st);
        case 4: return lookup_launch<T, V, 4>(C, ids, rows, dv, tr, K, d, scale, Y, st);
        case 8: return lookup_launch<T, V, 8>(C, ids, rows, dv, tr, K, d, scale, Y, st);
        case 16: return lookup_launch<T, V, 16>(C, ids, rows, dv, tr, K, d, scale, Y, st);
        default: return lookup_launch<T, V, 32>(C, ids, rows, dv, tr, K, d, scale, Y, st);
    }
}
template <typename T>
km_status lookup_typed(const void *Cv, const int32_t *ids, int64_t B, int64_t N, int64_t K, int64_t d,
                       float scale, void *Yv, cudaStream_t st) {
    const T *C = static_cast<const T *>(Cv);
    T *Y = static_cast<T *>(Yv);
    const int v = vec_elems(d, sizeof(T), C, Y);
    const FastDiv dv = make_fastdiv(static_cast<uint32_t>(N));
    const int64_t nb_max = std::max<int64_t>(1, ((int64_t{1} << 31) - 1) / N);   // rows per launch < 2^31
    for (int64_t b0 = 0; b0 < B; b0 += nb_max) {
        const uint32_t rows = static_cast<uint32_t>(std::min(nb_max, B - b0) * N);
        const T *Cb = C + b0 * K * d;
        const int32_t *ib = ids + b0 * N;
        T *Yb = Y + b0 * N * d;
        const int Ki = static_cast<int>(K), di = static_cast<int>(d);
        km_status s;
        switch (v * sizeof(T)) {
            case 16: s = lookup_tpr<T, 16 / sizeof(T)>(Cb, ib, rows, dv, std::min(nb_max, B - b0) * K, Ki, di, scale, Yb, st); break;
            case 8: s = lookup_tpr<T, 8 / sizeof(T)>(Cb, ib, rows, dv, std::min(nb_max, B - b0) * K, Ki, di, scale, Yb, st); break;
            case 4: s = lookup_tpr<T, 4 / sizeof(T)>(Cb, ib, rows, dv, std::min(nb_max, B - b0) * K, Ki, di, scale, Yb, st); break;
            default: s = lookup_tpr<T, 1>(Cb, ib, rows, dv, std::min(nb_max, B - b0) * K, Ki, di, scale, Yb, st); break;
        }
        if (s != KM_OK) return s;
    }
    return KM_OK;
}

// ------------------------------------------------------------------ gradient

struct GradWs {
    uint32_t *keys[2], *pos[2], *counts, *totals, *nvalid;
    float *slots;
};
// Entries per range: enough ranges to fill the device (32 groups per SM on 148 SMs), never
// shorter than 16 entries.
inline int64_t grad_range(int64_t T) { return std::max<int64_t>(16, ceil_div(T, 148 * 32)); }
inline GradWs carve_grad(Carver &c, int64_t T, int64_t d) {
    GradWs g;
    const int64_t tiles = ceil_div(T, kSortTile);
    for (int i = 0; i < 2; ++i) {
        g.keys[i] = c.take<uint32_t>(static_cast<size_t>(T) * 4);
        g.pos[i] = c.take<uint32_t>(static_cast<size_t>(T) * 4);
    }
    g.counts = c.take<uint32_t>(static_cast<size_t>(kBins * tiles) * 4);
    g.totals = c.take<uint32_t>(kBins * 4);
    g.nvalid = c.take<uint32_t>(4);
    g.slots = c.take<float>(static_cast<size_t>(ceil_div(T, grad_range(T)) * 2 * d) * 4);
    return g;
}
inline bool grad_sizes_ok(int64_t B, int64_t N, int64_t K, int64_t d) {
    return sizes_ok(B, N, K, d) && B * N <= kMaxIndex && B * K <= kMaxIndex;
}

template <typename T, typename O, int V, int LPR>
km_status grad_sum(const T *dY, const GradParams &p, int64_t ranges, O *dC, cudaStream_t st) {
    constexpr int GROUPS = kGradThreads / LPR;
    dim3 grid(static_cast<unsigned>(ceil_div(ranges, GROUPS)), static_cast<unsigned>(ceil_div(p.d, LPR * V)));
    if (grid.y > kMaxGridY) return KM_ERR_UNSUPPORTED;   // never: d <= 2^20 and 32 lanes per block
    grad_ranges_kernel<T, O, V, LPR><<<grid, kGradThreads, 0, st>>>(dY, p, dC);
    if (launch_status() != KM_OK) return KM_ERR_CUDA;
    if (ranges > 1) grad_join_kernel<O, V, LPR><<<static_cast<unsigned>(ranges), kGradThreads, 0, st>>>(p, dC);
    return launch_status();
}
template <typename T, typename O, int V>
km_status grad_lpr(const T *dY, const GradParams &p, int64_t ranges, O *dC, cudaStream_t st) {
    switch (pow2_at_least(ceil_div(p.d, V), 32)) {
        case 1: return grad_sum<T, O, V, 1>(dY, p, ranges, dC, st);
        case 2:
        case 4: return grad_sum<T, O, V, 4>(dY, p, ranges, dC, st);
        case 8: return grad_sum<T, O, V, 8>(dY, p, ranges, dC, st);
        case 16: return grad_sum<T, O, V, 16>(dY, p, ranges, dC, st);
        default: return grad_sum<T, O, V, 32>(dY, p, ranges, dC, st);
    }
}
template <typename T, typename O>
km_status grad_typed(const void *dYv, const GradParams &p, int64_t ranges, void *dCv, cudaStream_t st) {
    const T *dY = static_cast<const T *>(dYv);
    O *dC = static_cast<O *>(dCv);
    // 8 bytes a lane for 16-bit rows and 16 for fp32: four columns, one vector access on either side
    const int v = std::min(vec_elems(p.d, sizeof(T), dY, dY), vec_elems(p.d, sizeof(O), dC, dC));
    if (v >= 4) return grad_lpr<T, O, 4>(dY, p, ranges, dC, st);
    if (v >= 2) return grad_lpr<T, O, 2>(dY, p, ranges, dC, st);
    return grad_lpr<T, O, 1>(dY, p, ranges, dC, st);
}

}  // namespace

extern "C" {

km_status km_lookup(const void *C, km_dtype dtype, const int32_t *ids, int64_t B, int64_t N, int64_t K,
                    int64_t d, float scale, void *Y, void *stream) {
    if (!C || !ids || !Y || !valid_dtype(dtype) || !sizes_ok(B, N, K, d) || !elem_ok(C, dtype) ||
        !elem_ok(Y, dtype) || !aligned(ids, 4))
        return KM_ERR_INVALID_ARG;
    switch (dtype) {
        case KM_F32: return lookup_typed<float>(C, ids, B, N, K, d, scale, Y, S(stream));
        case KM_F16: return lookup_typed<__half>(C, ids, B, N, K, d, scale, Y, S(stream));
        default: return lookup_typed<__nv_bfloat16>(C, ids, B, N, K, d, scale, Y, S(stream));
    }
}

size_t km_lookup_grad_workspace_size(int64_t B, int64_t N, int64_t K, int64_t d) {
    if (!grad_sizes_ok(B, N, K, d)) return 0;
    Carver c(nullptr);
    carve_grad(c, B * N, d);
    return c.off;
}

km_status km_lookup_grad(const void *dY, km_dtype dtype, const int32_t *ids, int64_t B, int64_t N, int64_t K,
                         int64_t d, float scale, void *dC, km_dtype out_dtype, int accumulate, void *ws,
                         size_t ws_bytes, void *stream) {
    if (!dY || !ids || !dC || !valid_dtype(dtype) || !valid_dtype(out_dtype) || !sizes_ok(B, N, K, d) ||
        !elem_ok(dY, dtype) || !elem_ok(dC, out_dtype) || !aligned(ids, 4) || (ws && !aligned(ws, kAlign)))
        return KM_ERR_INVALID_ARG;
    if (!grad_sizes_ok(B, N, K, d)) return KM_ERR_UNSUPPORTED;
    if (out_dtype != KM_F32 && out_dtype != dtype) return KM_ERR_UNSUPPORTED;
    if (!ws || ws_bytes < km_lookup_grad_workspace_size(B, N, K, d)) return KM_ERR_WORKSPACE;
    cudaStream_t st = S(stream);
    const int64_t T = B * N;
    Carver c(ws);
    const GradWs w = carve_grad(c, T, d);
    if (!accumulate &&
        cudaMemsetAsync(dC, 0, static_cast<size_t>(B * K * d) * dtype_size(out_dtype), st) != cudaSuccess)
        return KM_ERR_CUDA;
    const uint32_t tiles = static_cast<uint32_t>(ceil_div(T, kSortTile));
    int bits = 1;
    while ((int64_t{1} << bits) < B * K) ++bits;
    int side = 0;
    for (int shift = 0; shift < bits; shift += 8) {
        SortIn in = {};
        in.n = static_cast<uint32_t>(T);
        in.K = static_cast<int>(K);
        in.divN = make_fastdiv(static_cast<uint32_t>(N));
        if (shift == 0) {
            in.ids = ids;
        } else {
            in.keys = w.keys[side ^ 1];
            in.pos = w.pos[side ^ 1];
            in.nvalid = w.nvalid;
        }
        sort_hist_kernel<<<tiles, kSortThreads, 0, st>>>(in, shift, tiles, w.counts);
        if (launch_status() != KM_OK) return KM_ERR_CUDA;
        sort_scan_kernel<<<kBins, kSortThreads, 0, st>>>(tiles, w.counts, w.totals);
        if (launch_status() != KM_OK) return KM_ERR_CUDA;
        sort_scatter_kernel<<<tiles, kSortThreads, 0, st>>>(in, shift, tiles, w.counts, w.totals, w.keys[side],
                                                            w.pos[side], shift == 0 ? w.nvalid : nullptr);
        if (launch_status() != KM_OK) return KM_ERR_CUDA;
        side ^= 1;
    }
    GradParams p = {};
    p.keys = w.keys[side ^ 1];
    p.pos = w.pos[side ^ 1];
    p.nvalid = w.nvalid;
    p.range = static_cast<uint32_t>(grad_range(T));
    p.d = static_cast<int>(d);
    p.scale = scale;
    p.accumulate = accumulate ? 1 : 0;
    p.slots = w.slots;
    const int64_t ranges = ceil_div(T, p.range);
    if (dtype == KM_F32) return grad_typed<float, float>(dY, p, ranges, dC, st);
    if (dtype == KM_F16)
        return out_dtype == KM_F32 ? grad_typed<__half, float>(dY, p, ranges, dC, st)
                                   : grad_typed<__half, __half>(dY, p, ranges, dC, st);
    return out_dtype == KM_F32 ? grad_typed<__nv_bfloat16, float>(dY, p, ranges, dC, st)
                               : grad_typed<__nv_bfloat16, __nv_bfloat16>(dY, p, ranges, dC, st);
}

}  // extern "C"
