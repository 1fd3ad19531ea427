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
// with 2 rows (4 pieces of a wide row) in flight per lane: more registers per thread cost more in
// resident warps than they hide (8: 122 us, 4: 91, 2: 87 for 2M rows of 256 bytes, 6.3 TB/s). Off is the type of offsets counted in units of V elements: 32 bits
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

// ------------------------------------------------------------------ stable sort by id
//
// Tokens are sorted by (batch, id), equal ids in token order; ids outside [0, K) are dropped. A
// least-significant-digit radix sort over the id's bits, digits of up to 10 bits. Where every
// batch is long, batches are segments that are sorted side by side on the id alone (their order
// is already that of the keys); where batches are short, all tokens are one segment with keys
// b K + id. Up to kSmallMax tokens a cluster of blocks sorts everything in its shared memory.

struct SortSpec {
    const int32_t *ids;
    FastDiv divN;            // batch of a token
    uint32_t K;              // per batch
    uint32_t n;              // tokens of a segment (at most)
    uint32_t segs, tps;      // segments, tiles per segment
    int width, shift;        // digit of this pass
    int by_batch;            // segments are batches: the digit is taken of the id, not of b K + id
    int scanned;             // counts hold scans over the tiles, totals the bins' sums
    const uint32_t *keys, *pos;   // entries of the pass before (first pass: null)
    uint32_t *segtotal;      // [segs] valid tokens
    uint32_t *segstart;      // [segs + 1] their exclusive sums (written by the first scatter)
    FastDiv divE;            // entries per block of the sorting cluster
};

constexpr int kSortThreads = 512;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kSortItems = 16;
constexpr int kSortTile = kSortThreads * kSortItems;
constexpr int kMaxWidth = 10;                  // bits of a digit
constexpr int kMaxBins = 1 << kMaxWidth;
constexpr int kScanTiles = 64;                 // above this many tiles a kernel of its own scans them
constexpr int kCluster = 8;
constexpr int kSmallMax = kCluster * kSortTile;
constexpr size_t kSortSmem = kSortTile * 6 + kSortWarps * kMaxBins * 2 + kMaxBins * 4;

// Entry i of segment `seg`: its key (b K + id) and token; false past the segment's end or for an id
// outside [0, K).
__device__ __forceinline__ bool sort_load(const SortSpec &s, uint32_t seg, uint32_t i, uint32_t &key, uint32_t &pos) {
    if (!s.keys) {
        if (i >= s.n) return false;
        pos = seg * s.n + i;
        const uint32_t id = static_cast<uint32_t>(s.ids[pos]);
        key = fd_div(s.divN, pos) * s.K + id;
        return id < s.K;
    }
    const uint32_t a = s.segstart[seg], e = s.segstart[seg + 1];
    if (i >= e - a) return false;
    key = s.keys[a + i];
    pos = s.pos[a + i];
    return true;
}
__device__ __forceinline__ uint32_t sort_digit(const SortSpec &s, uint32_t seg, uint32_t key) {
    return ((s.by_batch ? key - seg * s.K : key) >> s.shift) & ((1u << s.width) - 1);
}

// Digit counts of each tile: counts[(seg * tps + tile) * bins + bin]; the first pass also counts the
// valid tokens of the segments (segtotal zeroed beforehand; integer sums do not depend on order).
__global__ void __launch_bounds__(kSortThreads)
    sort_hist_kernel(const SortSpec s, uint32_t *__restrict__ counts) {
    __shared__ uint32_t bins[kMaxBins];
    const int nb = 1 << s.width;
    for (int b = threadIdx.x; b < nb; b += kSortThreads) bins[b] = 0;
    __syncthreads();
    const uint32_t seg = blockIdx.x / s.tps, tile = blockIdx.x - seg * s.tps;
    uint32_t key[kSortItems], pos;
    bool ok[kSortItems];
#pragma unroll
    for (int i = 0; i < kSortItems; ++i)
        ok[i] = sort_load(s, seg, tile * kSortTile + i * kSortThreads + threadIdx.x, key[i], pos);
#pragma unroll
    for (int i = 0; i < kSortItems; ++i)
        if (ok[i]) atomicAdd(&bins[sort_digit(s, seg, key[i])], 1u);
    int valid = 0;
#pragma unroll
    for (int i = 0; i < kSortItems; ++i) valid += ok[i];
    __syncthreads();
    if (!s.keys) {
        valid = __reduce_add_sync(0xffffffffu, valid);
        if ((threadIdx.x & 31) == 0 && valid) atomicAdd(s.segtotal + seg, static_cast<uint32_t>(valid));
    }
    for (int b = threadIdx.x; b < nb; b += kSortThreads) counts[static_cast<size_t>(blockIdx.x) * nb + b] = bins[b];
}

// Exclusive scan of one value per thread over the block; *total receives the sum.
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
    uint32_t w = lane < nw ? warp_sums[lane] : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, w, o);
        if (lane >= o) w += y;
    }
    const uint32_t before = __shfl_sync(0xffffffffu, w, warp ? warp - 1 : 0);
    *total = __shfl_sync(0xffffffffu, w, 31);
    __syncthreads();
    return x - v + (warp ? before : 0);
}

// Many tiles: tile counts -> exclusive scan over a segment's tiles, in place, and the bins' sums. A
// block covers 32 bins of a segment, its 32 warps a slice of the tiles each.
__global__ void __launch_bounds__(1024)
    sort_scan_kernel(const SortSpec s, uint32_t *__restrict__ counts, uint32_t *__restrict__ totals) {
    __shared__ uint32_t slice[32][33];
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const uint32_t nb = 1u << s.width, bpb = (nb + 31) / 32;
    const uint32_t seg = blockIdx.x / bpb, bin = (blockIdx.x - seg * bpb) * 32 + lane;
    uint32_t *c = counts + static_cast<size_t>(seg) * s.tps * nb + bin;
    const uint32_t per = (s.tps + 31) / 32, a = min(s.tps, w * per), e = min(s.tps, a + per);
    uint32_t sum = 0;
    if (bin < nb)
        for (uint32_t t = a; t < e; ++t) sum += c[static_cast<size_t>(t) * nb];
    slice[w][lane] = sum;
    __syncthreads();
    uint32_t run = 0;
    for (int k = 0; k < w; ++k) run += slice[k][lane];
    if (bin < nb) {
        for (uint32_t t = a; t < e; ++t) {
            const uint32_t v = c[static_cast<size_t>(t) * nb];
            c[static_cast<size_t>(t) * nb] = run;
            run += v;
        }
        if (w == 31) totals[seg * nb + bin] = run;
    }
}

// Stable ranks of a warp's entries among equal digits: entry i of a lane (there if bit i of ok is set) is
// number i * 32 + lane of the warp's. The lanes with an equal digit are found by a ballot per digit bit
// (a warp match has a far lower rate), for all entries first: the ballots do not depend on one another,
// the counting that follows does. mine[bin] counts the warp's entries.
template <typename Digit>
__device__ __forceinline__ void rank_digits(const Digit &digit, uint32_t ok, int per, uint16_t *mine, uint32_t (&rank)[kSortItems]) {
    const uint32_t below = (1u << (threadIdx.x & 31)) - 1;
#pragma unroll
    for (int i = 0; i < kSortItems; ++i) {
        if (i >= per) break;
        const uint32_t d = digit(i);
        uint32_t p = __ballot_sync(0xffffffffu, (ok >> i) & 1);
#pragma unroll
        for (int b = 0; b < kMaxWidth; ++b) {
            const bool bit = (d >> b) & 1;
            const uint32_t v = __ballot_sync(0xffffffffu, bit);
            p &= bit ? v : ~v;
        }
        rank[i] = __popc(p & below) | __popc(p) << 8;       // equal digits in lower lanes, in all
    }
#pragma unroll
    for (int i = 0; i < kSortItems; ++i) {
        if (i >= per) break;
        const bool has = (ok >> i) & 1;
        const uint32_t d = digit(i), lower = rank[i] & 255, all = rank[i] >> 8;
        uint32_t prior = 0;
        if (has) prior = mine[d];
        __syncwarp();
        rank[i] = prior + lower;
        if (has && lower == 0) mine[d] = static_cast<uint16_t>(prior + all);
        __syncwarp();
    }
}

// The warps' counts of one bin: their sum, each replaced by the sum of the ones before it plus `add`.
__device__ __forceinline__ uint32_t scan_warps(uint16_t *wcount, int nb, int bin, uint32_t add) {
    uint32_t v[kSortWarps];
#pragma unroll
    for (int w = 0; w < kSortWarps; ++w) v[w] = wcount[w * nb + bin];
    uint32_t sum = 0;
#pragma unroll
    for (int w = 0; w < kSortWarps; ++w) {
        wcount[w * nb + bin] = static_cast<uint16_t>(sum + add);
        sum += v[w];
    }
    return sum;
}
__device__ __forceinline__ uint32_t sum_warps(const uint16_t *wcount, int nb, int bin) {
    uint32_t sum = 0;
#pragma unroll
    for (int w = 0; w < kSortWarps; ++w) sum += wcount[w * nb + bin];
    return sum;
}
constexpr int kBinsPerThread = kMaxBins / kSortThreads;
// Exclusive sums over all bins of one value per bin; thread t holds bins 2 t and 2 t + 1.
static_assert(kBinsPerThread == 2, "block_scan_bins pairs the bins");
__device__ __forceinline__ void block_scan_bins(uint32_t (&v)[2], uint32_t *ws, uint32_t *total) {
    const uint32_t a = v[0], x = block_scan(v[0] + v[1], ws, total);
    v[0] = x;
    v[1] = x + a;
}

// Sorts a tile by the pass's digit in shared memory and writes its runs to (start of the bin) +
// (entries of the bin in earlier tiles): consecutive threads write consecutive entries of a run.
// Two blocks to an SM (64 registers, some spilled) hide more of the chain load, rank, scan, store than one
// with all it asks for: gradient of 1024 rows x 32 batches over 65536 tokens each 172 to 165 us.
__global__ void __launch_bounds__(kSortThreads, 2)
    sort_scatter_kernel(const SortSpec s, const uint32_t *__restrict__ counts, const uint32_t *__restrict__ totals,
                        uint32_t *__restrict__ keys_out, uint32_t *__restrict__ pos_out) {
    extern __shared__ uint32_t dyn[];
    __shared__ uint32_t ws[32];
    uint32_t *skeys = dyn;                                                   // [tile]
    uint16_t *sloc = reinterpret_cast<uint16_t *>(dyn + kSortTile);          // [tile]: number in the tile
    uint16_t *wcount = sloc + kSortTile;                                     // [warps][bins]
    uint32_t *shift_of = reinterpret_cast<uint32_t *>(wcount + kSortWarps * kMaxBins);   // [bins]
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nb = 1 << s.width;
    const uint32_t seg = blockIdx.x / s.tps, tile = blockIdx.x - seg * s.tps;
    const uint32_t i0 = warp * (32 * kSortItems) + lane;
    uint32_t key[kSortItems], rank[kSortItems], pos, ok = 0;
#pragma unroll
    for (int i = 0; i < kSortItems; ++i) ok |= static_cast<uint32_t>(sort_load(s, seg, tile * kSortTile + i0 + i * 32, key[i], pos)) << i;
    auto digit = [&](int i) { return sort_digit(s, seg, key[i]); };
    for (int k = threadIdx.x; k < kSortWarps * nb / 2; k += kSortThreads) reinterpret_cast<uint32_t *>(wcount)[k] = 0;
    // valid tokens of earlier segments
    uint32_t before = 0, all = 0;
    for (uint32_t k = threadIdx.x; k < s.segs; k += kSortThreads) {
        const uint32_t v = s.segtotal[k];
        all += v;
        if (k < seg) before += v;
    }
    uint32_t segbase, sum;
    block_scan(before, ws, &segbase);
    block_scan(all, ws, &sum);
    if (!s.keys && tile == 0 && threadIdx.x == 0) {
        s.segstart[seg] = segbase;
        if (seg == 0) s.segstart[s.segs] = sum;
    }
    // this thread's bins: entries in earlier tiles and in all of the segment
    uint32_t early[2] = {0, 0}, whole[2] = {0, 0};
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int bin = threadIdx.x * 2 + h;
        if (bin >= nb) continue;
        const uint32_t *c = counts + static_cast<size_t>(seg) * s.tps * nb + bin;
        if (s.scanned) {
            early[h] = c[static_cast<size_t>(tile) * nb];
            whole[h] = totals[seg * nb + bin];
        } else {
#pragma unroll 8
            for (uint32_t t = 0; t < s.tps; ++t) {
                const uint32_t v = c[static_cast<size_t>(t) * nb];
                if (t < tile) early[h] += v;
                whole[h] += v;
            }
        }
    }
    block_scan_bins(whole, ws, &sum);            // (its barriers also cover the zeroed counters)
    uint16_t *mine = wcount + warp * nb;
    rank_digits(digit, ok, kSortItems, mine, rank);
    __syncthreads();
    uint32_t local[2] = {0, 0}, entries;         // the bins' places in the sorted tile
#pragma unroll
    for (int h = 0; h < 2; ++h)
        if (threadIdx.x * 2 + h < nb) local[h] = sum_warps(wcount, nb, threadIdx.x * 2 + h);
    block_scan_bins(local, ws, &entries);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int bin = threadIdx.x * 2 + h;
        if (bin >= nb) continue;
        scan_warps(wcount, nb, bin, local[h]);
        shift_of[bin] = segbase + whole[h] + early[h] - local[h];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kSortItems; ++i)
        if ((ok >> i) & 1) {
            const uint32_t at = mine[digit(i)] + rank[i];
            skeys[at] = key[i];
            sloc[at] = static_cast<uint16_t>(i0 + i * 32);
        }
    __syncthreads();
    const uint32_t from = s.keys ? s.segstart[seg] + tile * kSortTile : seg * s.n + tile * kSortTile;
    for (uint32_t at = threadIdx.x; at < entries; at += kSortThreads) {
        const uint32_t k = skeys[at], to = at + shift_of[sort_digit(s, seg, k)];
        keys_out[to] = k;
        pos_out[to] = s.keys ? s.pos[from + sloc[at]] : from + sloc[at];
    }
}

// Zeros over [p, p + bytes), spread over `threads` threads of which this is number i.
__device__ __forceinline__ void zero_fill(uint8_t *p, size_t bytes, size_t i, size_t threads) {
    size_t head = (16 - (reinterpret_cast<uintptr_t>(p) & 15)) & 15;
    if (head > bytes) head = bytes;
    if (i < head) p[i] = 0;
    uint4 *v = reinterpret_cast<uint4 *>(p + head);
    const size_t units = (bytes - head) / 16;
    const uint4 z = make_uint4(0u, 0u, 0u, 0u);
    size_t u = i;
    for (; u + 3 * threads < units; u += 4 * threads) {
        v[u] = z;
        v[u + threads] = z;
        v[u + 2 * threads] = z;
        v[u + 3 * threads] = z;
    }
    for (; u < units; u += threads) v[u] = z;
    const size_t tail = head + units * 16;
    if (tail + i < bytes) p[tail + i] = 0;
}

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    __syncwarp();          // .aligned: the whole warp at once
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t cluster_addr(const void *p, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_u32(p)), "r"(rank));
    return r;
}
__device__ __forceinline__ uint32_t cluster_load(uint32_t a) {
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ void cluster_store2(uint32_t a, uint32_t x, uint32_t y) {
    asm volatile("st.shared::cluster.v2.u32 [%0], {%1, %2};" ::"r"(a), "r"(x), "r"(y) : "memory");
}

constexpr size_t kSmallSmem = kSortTile * 8 + kSortWarps * kMaxBins * 2 + kMaxBins * 4;

// Up to kSmallMax tokens in one launch: the first cluster of eight blocks sorts, exchanging digit
// counts and entries through its blocks' shared memory (dropped tokens carry the key B K and end up
// behind the others); the other blocks zero the table's gradient, which for a large table takes
// longer than the sort. Block c of the cluster holds entries [c E, (c + 1) E).
__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kSortThreads, 1)
    sort_small_kernel(const SortSpec s, uint32_t tokens, uint32_t keys_total, int passes,
                      uint32_t *__restrict__ keys_out, uint32_t *__restrict__ pos_out, uint32_t *__restrict__ nvalid,
                      unsigned int *__restrict__ jobs, uint8_t *zero, size_t zero_bytes) {
    if (blockIdx.x >= kCluster) {
        if (zero)
            zero_fill(zero, zero_bytes, static_cast<size_t>(blockIdx.x - kCluster) * kSortThreads + threadIdx.x,
                      static_cast<size_t>(gridDim.x - kCluster) * kSortThreads);
        return;
    }
    extern __shared__ uint32_t dyn[];
    __shared__ uint32_t ws[32];
    __shared__ uint32_t nvalid_mine;
    uint2 *entries = reinterpret_cast<uint2 *>(dyn);                                 // [E]: key, token
    uint16_t *wcount = reinterpret_cast<uint16_t *>(dyn + 2 * kSortTile);            // [warps][bins]
    uint32_t *bincount = reinterpret_cast<uint32_t *>(wcount + kSortWarps * kMaxBins);   // [bins], this block's
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nb = 1 << s.width;
    const uint32_t rank_c = cluster_rank();
    const int per = static_cast<int>((tokens + kCluster * kSortThreads - 1) / (kCluster * kSortThreads));
    const uint32_t E = static_cast<uint32_t>(per) * kSortThreads, e0 = rank_c * E;
    const FastDiv div_e = s.divE;
    const uint32_t i0 = static_cast<uint32_t>(warp * 32 * per + lane);
    uint32_t key[kSortItems], pos[kSortItems];
    uint32_t rank[kSortItems], ok = 0, valid = 0;
#pragma unroll
    for (int i = 0; i < kSortItems; ++i) {
        const uint32_t at = e0 + i0 + i * 32;
        pos[i] = at;
        if (i < per && at < tokens) {
            ok |= 1u << i;
            const uint32_t id = static_cast<uint32_t>(s.ids[at]);
            key[i] = id < s.K ? fd_div(s.divN, at) * s.K + id : keys_total;
            valid += id < s.K;
        }
    }
    uint32_t tot;
    block_scan(valid, ws, &tot);
    if (threadIdx.x == 0) nvalid_mine = tot;
    uint16_t *mine = wcount + warp * nb;
    for (int pass = 0; pass < passes; ++pass) {
        for (int k = threadIdx.x; k < kSortWarps * nb / 2; k += kSortThreads) reinterpret_cast<uint32_t *>(wcount)[k] = 0;
        __syncthreads();
        auto digit = [&](int i) { return (key[i] >> (pass * s.width)) & (nb - 1); };
        rank_digits(digit, ok, per, mine, rank);
        __syncthreads();
        for (int b = threadIdx.x; b < nb; b += kSortThreads) bincount[b] = sum_warps(wcount, nb, b);
        cluster_sync();
        // entries of this thread's bins in earlier blocks and in all
        uint32_t early[2] = {0, 0}, whole[2] = {0, 0};
#pragma unroll
        for (int c = 0; c < kCluster; ++c) {
            const uint32_t base = cluster_addr(bincount, c);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int bin = threadIdx.x * 2 + h;
                const uint32_t v = bin < nb ? cluster_load(base + bin * 4) : 0;
                if (c < static_cast<int>(rank_c)) early[h] += v;
                whole[h] += v;
            }
        }
        if (pass == 0 && rank_c == 0 && threadIdx.x < 32) {
            const uint32_t v = lane < kCluster ? cluster_load(cluster_addr(&nvalid_mine, lane)) : 0;
            const uint32_t sum = __reduce_add_sync(0xffffffffu, v);
            if (lane == 0) {
                *nvalid = sum;
                *jobs = 0;
            }
        }
        block_scan_bins(whole, ws, &tot);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int bin = threadIdx.x * 2 + h;
            // the warps' places relative to the block's first entry of the bin (16 bits), and that
            if (bin < nb) scan_warps(wcount, nb, bin, 0);
        }
        // every block has read the counts; then they hold the bins' starts of this block
        cluster_sync();
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int bin = threadIdx.x * 2 + h;
            if (bin < nb) bincount[bin] = whole[h] + early[h];
        }
        __syncthreads();
        const bool final = pass + 1 == passes;
#pragma unroll
        for (int i = 0; i < kSortItems; ++i)
            if ((ok >> i) & 1) {
                const uint32_t at = bincount[digit(i)] + mine[digit(i)] + rank[i];
                if (final) {
                    keys_out[at] = key[i];
                    pos_out[at] = pos[i];
                } else {
                    const uint32_t c = fd_div(div_e, at);
                    cluster_store2(cluster_addr(entries + (at - c * E), c), key[i], pos[i]);
                }
            }
        cluster_sync();          // the entries have arrived; nobody leaves while others still read
        if (final) break;
#pragma unroll
        for (int i = 0; i < kSortItems; ++i)
            if ((ok >> i) & 1) {
                const uint2 v = entries[i0 + i * 32];
                key[i] = v.x;
                pos[i] = v.y;
            }
    }
}

// ------------------------------------------------------------------ sums over the sorted order

struct GradParams {
    const uint32_t *keys, *pos, *nvalid;
    uint32_t tokens;       // entries that keys and pos have room for
    uint32_t range;        // sorted entries per range, before its ends move to the ends of runs
    uint32_t units;        // per row
    float scale;
    int accumulate;
    float *slots;          // [ranges][2][d] fp32: the range's first and last run where they are cut
    uint32_t *jobs;        // [0] count, then the first range of every cut run
};

template <typename O, int V>
__device__ __forceinline__ void write_row(O *out, const float (&acc)[V], float scale, int accumulate) {
    constexpr int VO = 16 / sizeof(O) < V ? 16 / sizeof(O) : V;      // at most 16 bytes per access
#pragma unroll
    for (int h = 0; h < V; h += VO) {
        Vec<O, VO> o;
        if (accumulate) o = *reinterpret_cast<const Vec<O, VO> *>(out + h);
#pragma unroll
        for (int i = 0; i < VO; ++i) {
            const float s = scale * acc[h + i];
            o.v[i] = Cvt<O>::from_f(accumulate ? Cvt<O>::to_f(o.v[i]) + s : s);
        }
        *reinterpret_cast<Vec<O, VO> *>(out + h) = o;
    }
}

// V fp32 values of a slot, in 16-byte accesses where V allows.
template <int V> __device__ __forceinline__ void store_slot(float *p, const float (&v)[V]) {
    constexpr int W = V < 4 ? V : 4;
#pragma unroll
    for (int h = 0; h < V; h += W) {
        Vec<float, W> o;
#pragma unroll
        for (int i = 0; i < W; ++i) o.v[i] = v[h + i];
        *reinterpret_cast<Vec<float, W> *>(p + h) = o;
    }
}
template <int V> __device__ __forceinline__ void add_slot(const float *p, float (&v)[V]) {
    constexpr int W = V < 4 ? V : 4;
#pragma unroll
    for (int h = 0; h < V; h += W) {
        const Vec<float, W> o = *reinterpret_cast<const Vec<float, W> *>(p + h);
#pragma unroll
        for (int i = 0; i < W; ++i) v[h + i] += o.v[i];
    }
}

constexpr int kGradThreads = 256;

// Where range r begins: the first start of a run in [r L, (r + 1) L), so that a run is summed by
// one range; a run that covers all of it is cut at r L. The LPR lanes of a group search together;
// every lane of the warp takes part.
template <int LPR>
__device__ __forceinline__ uint32_t range_begin(const uint32_t *keys, uint32_t n, uint64_t at, uint32_t L, bool &cut) {
    const int t = threadIdx.x % LPR;
    const uint32_t gmask = LPR == 32 ? 0xffffffffu : ((1u << (LPR & 31)) - 1) << ((threadIdx.x & 31) / LPR * LPR);
    cut = false;
    const bool inside = at < n && at > 0;
    uint32_t found = at >= n ? n : static_cast<uint32_t>(at);
    bool open = inside;
    for (uint32_t o = 0; o < L; o += LPR) {
        if (!__any_sync(0xffffffffu, open)) break;
        const uint64_t i = at + o + t;
        bool start = false;
        if (open && o + t < L) start = i >= n || keys[i] != keys[i - 1];
        const uint32_t b = __ballot_sync(0xffffffffu, start) & gmask;
        if (open && b) {
            const uint64_t f = at + o + (__ffs(b) - 1) % LPR;
            found = f < n ? static_cast<uint32_t>(f) : n;
            open = false;
        }
    }
    cut = open;
    return found;
}

// LPR lanes per range and V columns per lane. A range adds up the rows of its runs of equal keys
// one after the other in fp32; a whole run goes to its table row, a cut one to the range's slots,
// and the range that a cut run begins in enters the run into the list of joins. SHORT: a range's
// possible entries are at most LPR, read in one go together with the search for its ends.
// Bound by memory: each row of dY is read once, in whole rows but in the order of the ids. 2M rows of 256
// bytes into 32 x 1024 rows: 112 us for 548 MB read, 4.9 TB/s (a plain copy moves 6.5). 16384 rows of
// 2 KB into 65536: 21 us under the profiler for 33 MB, the latency of short runs.
template <typename T, typename O, int V, int LPR, bool SHORT>
__global__ void __launch_bounds__(kGradThreads)
    grad_ranges_kernel(const T *__restrict__ dY, const GradParams p, O *__restrict__ dC) {
    constexpr int GROUPS = kGradThreads / LPR;
    constexpr int U = LPR < 8 ? LPR : (V * sizeof(T) >= 16 && !SHORT ? 4 : 8);   // rows in flight per group
    const int t = threadIdx.x % LPR;
    const uint32_t r = blockIdx.x * static_cast<uint32_t>(GROUPS) + threadIdx.x / LPR;
    const uint64_t first = static_cast<uint64_t>(r) * p.range;
    uint32_t key0 = 0, pos0 = 0, before = 0;
    if (SHORT) {      // read ahead of the number of entries: the arrays hold a value for every token
        const uint64_t i = first + t;
        if (i < p.tokens) {
            key0 = p.keys[i];
            pos0 = p.pos[i];
            if (t == 0 && i > 0) before = p.keys[i - 1];
        }
    }
    const uint32_t n = *p.nvalid;
    bool cut0, cut1;
    uint32_t s, len;
    if (SHORT) {
        const uint64_t i = first + t;
        uint32_t prev = __shfl_up_sync(0xffffffffu, key0, 1, LPR);
        if (t == 0) prev = before;
        const bool start = i >= n || i == 0 || key0 != prev;
        uint32_t m = __ballot_sync(0xffffffffu, start);
        if (LPR < 32) m = (m >> ((threadIdx.x & 31) / LPR * LPR)) & ((1u << (LPR & 31)) - 1);
        const uint32_t low = (1u << p.range) - 1;         // range <= LPR / 2 <= 16
        const uint32_t m0 = m & low, m1 = (m >> p.range) & low;
        const uint32_t left = first >= n ? 0 : static_cast<uint32_t>(min(static_cast<uint64_t>(n) - first, static_cast<uint64_t>(LPR)));
        const uint32_t so = min(left, m0 ? __ffs(m0) - 1u : 0u), eo = min(left, p.range + (m1 ? __ffs(m1) - 1u : 0u));
        cut0 = m0 == 0;
        cut1 = m1 == 0;
        // entries [so, eo) of the lanes' move to the front
        key0 = __shfl_sync(0xffffffffu, key0, (t + so) & (LPR - 1), LPR);
        pos0 = __shfl_sync(0xffffffffu, pos0, (t + so) & (LPR - 1), LPR);
        s = static_cast<uint32_t>(first) + so;
        len = eo - so;
    } else {
        s = range_begin<LPR>(p.keys, n, first, p.range, cut0);
        len = range_begin<LPR>(p.keys, n, first + p.range, p.range, cut1) - s;   // at most two ranges' entries
        if (t < len) {
            key0 = p.keys[s + t];
            pos0 = p.pos[s + t];
        }
    }
    const uint32_t c = blockIdx.y * LPR + t;
    const bool in = c < p.units;
    const int64_t d = static_cast<int64_t>(p.units) * V;
    const Vec<T, V> *src = reinterpret_cast<const Vec<T, V> *>(dY);
    float acc[V];
#pragma unroll
    for (int i = 0; i < V; ++i) acc[i] = 0.f;
    bool head = cut0;
    uint32_t cur = 0;
    auto flush = [&](bool tail) {
        if (!in) return;
        if (head || tail) {
            float *slot = p.slots + (static_cast<int64_t>(r) * 2 + (head ? 0 : 1)) * d + static_cast<int64_t>(c) * V;
            store_slot<V>(slot, acc);
        } else {
            write_row<O, V>(dC + static_cast<int64_t>(cur) * d + static_cast<int64_t>(c) * V, acc, p.scale, p.accumulate);
        }
    };
    for (uint32_t b = 0; __any_sync(0xffffffffu, b < len); b += LPR) {
        // this batch's entries were read while the one before was summed
        const uint32_t key = key0, pos = pos0;
        if (!SHORT && b + LPR + t < len) {
            key0 = p.keys[s + b + LPR + t];
            pos0 = p.pos[s + b + LPR + t];
        }
        if (b == 0) cur = __shfl_sync(0xffffffffu, key, 0, LPR);
#pragma unroll 1
        for (int u0 = 0; u0 < LPR; u0 += U) {
            if (!__any_sync(0xffffffffu, b + u0 < len)) break;
            Vec<T, V> v[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const uint32_t row = __shfl_sync(0xffffffffu, pos, u0 + u, LPR);
                if (b + u0 + u < len && in) v[u] = load_ro(src + static_cast<int64_t>(row) * p.units + c);
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const uint32_t k = __shfl_sync(0xffffffffu, key, u0 + u, LPR);
                if (b + u0 + u < len) {
                    if (k != cur) {
                        flush(false);
                        cur = k;
                        head = false;
#pragma unroll
                        for (int i = 0; i < V; ++i) acc[i] = 0.f;
                    }
                    if (in)
#pragma unroll
                        for (int i = 0; i < V; ++i) acc[i] += Cvt<T>::to_f(v[u].v[i]);
                }
            }
        }
    }
    if (len) {
        if (cut1 && !head && t == 0 && blockIdx.y == 0) p.jobs[1 + atomicAdd(p.jobs, 1u)] = r;
        flush(cut1);
    }
}

// Joins the pieces of the cut runs, each in range order: a block per run and 32 V columns takes the
// runs off the list (whose order does not matter: every run is a row of its own); its eight warps
// add up consecutive pieces, then the eight sums in order.
template <typename O, int V>
__global__ void __launch_bounds__(kGradThreads)
    grad_join_kernel(const GradParams p, O *__restrict__ dC) {
    constexpr int WARPS = kGradThreads / 32;
    __shared__ float part[WARPS][32 * V];
    const uint32_t n = *p.nvalid, njobs = p.jobs[0];
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int64_t d = static_cast<int64_t>(p.units) * V;
    const uint32_t c = blockIdx.y * 32 + lane;
    const bool in = c < p.units;
    for (uint32_t job = blockIdx.x; job < njobs; job += gridDim.x) {
        const uint32_t r0 = p.jobs[1 + job];
        const uint32_t cut = (r0 + 1) * p.range;            // an entry of the run, the first behind r0
        const uint32_t key = p.keys[cut];
        // the run's end, 32 probes at a time
        uint32_t lo = cut, hi = n;                           // keys[lo] == key; hi is behind the run
        while (hi - lo > 1) {
            const uint32_t step = (hi - lo + 31) / 32;
            const uint64_t at = static_cast<uint64_t>(lo) + static_cast<uint64_t>(lane) * step;
            const bool same = at < hi && p.keys[at] == key;
            const int k = 31 - __clz(__ballot_sync(0xffffffffu, same));
            const uint64_t nhi = static_cast<uint64_t>(lo) + static_cast<uint64_t>(k + 1) * step;
            lo += k * step;
            if (nhi < hi) hi = static_cast<uint32_t>(nhi);
        }
        // The last piece: the run ends at lo; it was cut at every multiple of the range whose whole
        // range it covers, i.e. up to the last r with r L + L <= lo + 1.
        const uint32_t r1 = (lo + 1) / p.range - 1;
        const uint32_t count = r1 - r0 + 1, per = (count + WARPS - 1) / WARPS;
        float acc[V];
#pragma unroll
        for (int i = 0; i < V; ++i) acc[i] = 0.f;
        if (in) {
            const uint32_t a = min(count, w * per), e = min(count, a + per);
            const float *slot = p.slots + static_cast<int64_t>(c) * V;
#pragma unroll 8
            for (uint32_t j = a; j < e; ++j) {
                add_slot<V>(slot + (static_cast<int64_t>(r0 + j) * 2 + (j == 0 ? 1 : 0)) * d, acc);
            }
        }
#pragma unroll
        for (int i = 0; i < V; ++i) part[w][i * 32 + lane] = acc[i];
        __syncthreads();
        if (w == 0 && in) {
            for (int q = 1; q < WARPS; ++q)
#pragma unroll
                for (int i = 0; i < V; ++i) acc[i] += part[q][i * 32 + lane];
            write_row<O, V>(dC + static_cast<int64_t>(key) * d + static_cast<int64_t>(c) * V, acc, p.scale, p.accumulate);
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

// How the tokens of a call are sorted.
struct SortPlan {
    bool small;              // one cluster, in shared memory
    int64_t segs, n, tps;    // otherwise: segments, their tokens, tiles per segment
    bool by_batch;
    int passes, width;       // digits
};
inline int bits_of(int64_t values) {     // bits that hold 0 .. values - 1
    int b = 1;
    while ((int64_t{1} << b) < values) ++b;
    return b;
}
inline SortPlan sort_plan(int64_t B, int64_t N, int64_t K) {
    SortPlan p = {};
    p.small = B * N <= kSmallMax;
    if (p.small) {
        const int bits = bits_of(B * K + 1);
        p.passes = static_cast<int>(ceil_div(bits, kMaxWidth));
        p.width = static_cast<int>(ceil_div(bits, p.passes));
        return p;
    }
    // Batches of at least half a tile are segments (their sort needs the bits of the id alone; every
    // block sums the sizes of the segments before its own).
    int bits = bits_of(K);
    p.passes = static_cast<int>(ceil_div(bits, kMaxWidth));
    p.width = static_cast<int>(ceil_div(bits, p.passes));
    p.by_batch = N >= kSortTile / 2 && B <= 65536;
    if (!p.by_batch) {
        bits = bits_of(B * K);
        p.passes = static_cast<int>(ceil_div(bits, kMaxWidth));
        p.width = static_cast<int>(ceil_div(bits, p.passes));
    }
    p.segs = p.by_batch ? B : 1;
    p.n = p.by_batch ? N : B * N;
    p.tps = ceil_div(p.n, kSortTile);
    return p;
}

// Entries per range: as many ranges as fill the device with their groups (64 per SM on 148 SMs), at
// least 16 entries each.
inline int64_t grad_range(int64_t T) { return std::max<int64_t>(16, ceil_div(T, 148 * 64)); }

struct GradWs {
    uint32_t *keys[2], *pos[2], *counts, *totals, *segtotal, *segstart, *jobs;
    float *slots;
};
inline GradWs carve_grad(Carver &c, int64_t B, int64_t N, int64_t K, int64_t d) {
    GradWs g = {};
    const int64_t T = B * N, ranges = ceil_div(T, grad_range(T));
    const SortPlan p = sort_plan(B, N, K);
    for (int i = 0; i < (p.passes > 1 && !p.small ? 2 : 1); ++i) {
        g.keys[i] = c.take<uint32_t>(static_cast<size_t>(T) * 4);
        g.pos[i] = c.take<uint32_t>(static_cast<size_t>(T) * 4);
    }
    if (!p.small) {
        g.counts = c.take<uint32_t>(static_cast<size_t>(p.segs * p.tps << p.width) * 4);
        if (p.tps > kScanTiles) g.totals = c.take<uint32_t>(static_cast<size_t>(p.segs << p.width) * 4);
        g.segtotal = c.take<uint32_t>(static_cast<size_t>(p.segs) * 4);
    }
    g.segstart = c.take<uint32_t>(static_cast<size_t>(p.segs + 1) * 4);
    g.jobs = c.take<uint32_t>(static_cast<size_t>(ranges + 1) * 4);
    g.slots = c.take<float>(static_cast<size_t>(ranges * 2 * d) * 4);
    return g;
}
inline bool grad_sizes_ok(int64_t B, int64_t N, int64_t K, int64_t d) {
    return sizes_ok(B, N, K, d) && B * N <= kMaxIndex && B * K < kMaxIndex;
}

// Sorts the tokens; *side is the buffer that holds them, *nvalid their number on the device. `zero`
// (or null) is set to zeros.
km_status grad_sort(const int32_t *ids, int64_t B, int64_t N, int64_t K, const GradWs &w, void *zero, size_t zero_bytes,
                    int *side, const uint32_t **nvalid, cudaStream_t st) {
    const SortPlan p = sort_plan(B, N, K);
    const int64_t T = B * N;
    SortSpec s = {};
    s.ids = ids;
    s.divN = make_fastdiv(static_cast<uint32_t>(N));
    s.K = static_cast<uint32_t>(K);
    s.width = p.width;
    if (p.small) {
        static std::atomic<uint64_t> ready{0};
        if (!allow_smem(sort_small_kernel, kSmallSmem, ready)) return KM_ERR_CUDA;
        s.divE = make_fastdiv(static_cast<uint32_t>(ceil_div(T, kCluster * kSortThreads) * kSortThreads));
        // A zeroing block per 64 KB, but no more clusters than can be resident beside the sorting one:
        // a second wave would double the time.
        static int resident[64] = {0};
        int dev = 0;
        cudaGetDevice(&dev);
        int clusters = (dev >= 0 && dev < 64) ? resident[dev] : 0;
        if (clusters <= 0) {
            cudaLaunchConfig_t cfg = {};
            cfg.gridDim = dim3(kCluster * 16);
            cfg.blockDim = dim3(kSortThreads);
            cfg.dynamicSmemBytes = kSmallSmem;
            cudaLaunchAttribute attr;
            attr.id = cudaLaunchAttributeClusterDimension;
            attr.val.clusterDim.x = kCluster;
            attr.val.clusterDim.y = 1;
            attr.val.clusterDim.z = 1;
            cfg.attrs = &attr;
            cfg.numAttrs = 1;
            if (cudaOccupancyMaxActiveClusters(&clusters, sort_small_kernel, &cfg) != cudaSuccess || clusters <= 1) {
                cudaGetLastError();
                clusters = 2;
            }
            if (dev >= 0 && dev < 64) resident[dev] = clusters;
        }
        const int64_t fill = zero ? std::min<int64_t>(clusters - 1, std::max<int64_t>(1, ceil_div(static_cast<int64_t>(zero_bytes), 65536 * kCluster))) * kCluster : 0;
        sort_small_kernel<<<static_cast<unsigned>(kCluster + fill), kSortThreads, kSmallSmem, st>>>(
            s, static_cast<uint32_t>(T), static_cast<uint32_t>(B * K), p.passes, w.keys[0], w.pos[0], w.segstart, w.jobs,
            static_cast<uint8_t *>(zero), zero_bytes);
        *side = 0;
        *nvalid = w.segstart;
        return launch_status();
    }
    if ((zero && cudaMemsetAsync(zero, 0, zero_bytes, st) != cudaSuccess) ||
        cudaMemsetAsync(w.segtotal, 0, static_cast<size_t>(p.segs) * 4, st) != cudaSuccess ||
        cudaMemsetAsync(w.jobs, 0, 4, st) != cudaSuccess)
        return KM_ERR_CUDA;
    static std::atomic<uint64_t> ready{0};
    if (!allow_smem(sort_scatter_kernel, kSortSmem, ready)) return KM_ERR_CUDA;
    s.n = static_cast<uint32_t>(p.n);
    s.segs = static_cast<uint32_t>(p.segs);
    s.tps = static_cast<uint32_t>(p.tps);
    s.by_batch = p.by_batch ? 1 : 0;
    s.scanned = p.tps > kScanTiles ? 1 : 0;
    s.segtotal = w.segtotal;
    s.segstart = w.segstart;
    const int64_t blocks = p.segs * p.tps, sblocks = p.segs * ceil_div(int64_t{1} << p.width, 32);
    if (blocks > kMaxIndex || sblocks > kMaxIndex) return KM_ERR_UNSUPPORTED;
    *side = 0;
    for (int pass = 0; pass < p.passes; ++pass) {
        s.shift = pass * p.width;
        if (pass) {
            s.keys = w.keys[*side];
            s.pos = w.pos[*side];
            *side ^= 1;
        }
        sort_hist_kernel<<<static_cast<unsigned>(blocks), kSortThreads, 0, st>>>(s, w.counts);
        if (launch_status() != KM_OK) return KM_ERR_CUDA;
        if (s.scanned) {
            sort_scan_kernel<<<static_cast<unsigned>(sblocks), 1024, 0, st>>>(s, w.counts, w.totals);
            if (launch_status() != KM_OK) return KM_ERR_CUDA;
        }
        sort_scatter_kernel<<<static_cast<unsigned>(blocks), kSortThreads, kSortSmem, st>>>(
            s, w.counts, w.totals, w.keys[*side], w.pos[*side]);
        if (launch_status() != KM_OK) return KM_ERR_CUDA;
    }
    *nvalid = w.segstart + p.segs;
    return KM_OK;
}

template <typename T, typename O, int V, int LPR>
km_status grad_sum(const T *dY, const GradParams &p, int64_t ranges, O *dC, cudaStream_t st) {
    const dim3 grid(static_cast<unsigned>(ceil_div(ranges, kGradThreads / LPR)), static_cast<unsigned>(ceil_div(p.units, LPR)));
    if (grid.y > kMaxGridY) return KM_ERR_UNSUPPORTED;   // never: d <= 2^20 and 32 lanes per block
    bool launched = false;
    if constexpr (LPR >= 32)
        if (2 * p.range <= LPR) {
            grad_ranges_kernel<T, O, V, LPR, true><<<grid, kGradThreads, 0, st>>>(dY, p, dC);
            launched = true;
        }
    if (!launched) grad_ranges_kernel<T, O, V, LPR, false><<<grid, kGradThreads, 0, st>>>(dY, p, dC);
    if (launch_status() != KM_OK) return KM_ERR_CUDA;
    if (ranges > 1) {
        const unsigned cols = static_cast<unsigned>(ceil_div(p.units, 32));
        const unsigned rows = static_cast<unsigned>(std::min<int64_t>(ranges, std::max<int64_t>(1, 148 * 4 / cols)));
        grad_join_kernel<O, V><<<dim3(rows, cols), kGradThreads, 0, st>>>(p, dC);
    }
    return launch_status();
}
template <typename T, typename O, int V>
km_status grad_lpr(const T *dY, GradParams p, int64_t d, int64_t ranges, O *dC, cudaStream_t st) {
    p.units = static_cast<uint32_t>(d / V);
    switch (pow2_at_least(p.units, 32)) {
        case 1: return grad_sum<T, O, V, 1>(dY, p, ranges, dC, st);
        case 2:
        case 4: return grad_sum<T, O, V, 4>(dY, p, ranges, dC, st);
        case 8: return grad_sum<T, O, V, 8>(dY, p, ranges, dC, st);
        case 16: return grad_sum<T, O, V, 16>(dY, p, ranges, dC, st);
        default: return grad_sum<T, O, V, 32>(dY, p, ranges, dC, st);
    }
}
template <typename T, typename O>
km_status grad_typed(const void *dYv, const GradParams &p, int64_t d, int64_t ranges, void *dCv, cudaStream_t st) {
    const T *dY = static_cast<const T *>(dYv);
    O *dC = static_cast<O *>(dCv);
    // the widest access that both sides' rows allow: 16 bytes of dY, and whole 16-byte pieces of dC
    const int vt = vec_elems(d, sizeof(T), dY, dY), vo = vec_elems(d, sizeof(O), dC, dC);
    const int v = vo * sizeof(O) >= 16 ? vt : std::min(vt, vo);
    if constexpr (sizeof(T) == 2)
        if (v >= 8) return grad_lpr<T, O, 8>(dY, p, d, ranges, dC, st);
    if (v >= 4) return grad_lpr<T, O, 4>(dY, p, d, ranges, dC, st);
    if (v >= 2) return grad_lpr<T, O, 2>(dY, p, d, ranges, dC, st);
    return grad_lpr<T, O, 1>(dY, p, d, ranges, dC, st);
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
    carve_grad(c, B, N, K, d);
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
    Carver c(ws);
    const GradWs w = carve_grad(c, B, N, K, d);
    GradParams p = {};
    int side = 0;
    const km_status s = grad_sort(ids, B, N, K, w, accumulate ? nullptr : dC,
                                  static_cast<size_t>(B * K * d) * dtype_size(out_dtype), &side, &p.nvalid, st);
    if (s != KM_OK) return s;
    p.keys = w.keys[side];
    p.pos = w.pos[side];
    p.tokens = static_cast<uint32_t>(B * N);
    p.range = static_cast<uint32_t>(grad_range(B * N));
    p.scale = scale;
    p.accumulate = accumulate ? 1 : 0;
    p.slots = w.slots;
    p.jobs = w.jobs;
    const int64_t ranges = ceil_div(B * N, p.range);
    if (dtype == KM_F32) return grad_typed<float, float>(dY, p, d, ranges, dC, st);
    if (dtype == KM_F16)
        return out_dtype == KM_F32 ? grad_typed<__half, float>(dY, p, d, ranges, dC, st)
                                   : grad_typed<__half, __half>(dY, p, d, ranges, dC, st);
    return out_dtype == KM_F32 ? grad_typed<__nv_bfloat16, float>(dY, p, d, ranges, dC, st)
                               : grad_typed<__nv_bfloat16, __nv_bfloat16>(dY, p, d, ranges, dC, st);
}

}  // extern "C"
