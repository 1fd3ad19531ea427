// km_xent.cu -- softmax cross entropy over a table: C entry points, workspaces and launches
// (kernels in km_xent.cuh).
#include <cmath>
#include <type_traits>

#include "km_host.h"
#include "km_xent.cuh"
#include "km_xent_tc.cuh"
#include "km_xent_fused.cuh"

namespace {

using namespace km::xe;

// Entries of P held at a time (256 MiB of 16-bit). Pieces that stay in L2 lose more to short launches
// than they save in traffic (8192 x 32768 points x rows at d = 1024, forward and backward: 2^25
// entries 1.77 ms, 2^26 1.60, 2^27 1.57).
constexpr int64_t kPieceElems = int64_t{1} << 27;
constexpr int kPieceStep = 256;

inline bool xent_sizes_ok(int64_t B, int64_t N, int64_t K, int64_t d) {
    return sizes_ok(B, N, K, d) && N <= kMaxIndex - 1024 && K <= kMaxIndex - 1024 && B * N <= kMaxIndex &&
           B * ceil_div(N, ST) * ceil_div(K, ST) <= kMaxIndex;
}

// Table rows per piece of the gradient.
inline int64_t piece_rows(int64_t B, int64_t N, int64_t K) {
    const int64_t all = ceil_div(K, kPieceStep) * kPieceStep;
    const int64_t fit = kPieceElems / (B * N) / kPieceStep * kPieceStep;
    return std::min(all, std::max<int64_t>(kPieceStep, fit));
}
// Splits of a product's reduction, each a multiple of 64 long. The tensor cores work on 256 x 256
// tiles, one SM pair each, of which 74 run at once: the split is the one with the shortest estimate of
// waves * (64-wide steps of a split + 4 to start and drain) at 0.3 us a step, plus the writing and
// reading of the splits' fp32 partials at 4 TB/s and a launch. (dC of a 4096-row table over 32768 points
// at d = 256, 16 tiles: 253 us unsplit, 161 in the chosen four; dX, 128 tiles: 152 unsplit as chosen, 189 in
// two.) No split is longer than 256 steps, kMaxChain products: its additions truncate, and the splits are joined
// in fp32 (65536 points, 2048 rows, d = 1024: one-signed sums 2.1e-4 too small in splits of 512 steps, 1.0e-4
// in these). The CUDA cores work on 128 x 128 tiles and split where those leave SMs idle, each split at least
// 512 long.
inline int64_t product_splits(int64_t B, int64_t M, int64_t N, int64_t Kk, km_dtype dt) {
    const int64_t steps = ceil_div(Kk, TKC);
    if (dt == KM_F32) {
        const int64_t tiles = B * ceil_div(M, ST) * ceil_div(N, ST);
        if (tiles >= 148) return 1;
        const int64_t want = std::max<int64_t>(1, std::min(ceil_div(148, tiles), Kk / 512));
        return ceil_div(steps, ceil_div(steps, want));
    }
    const int64_t tiles = B * ceil_div(M, 2 * TBM) * ceil_div(N, TBN);
    const int64_t least = ceil_div(steps, kMaxChain / 4);
    int64_t best = least;
    double best_us = 0;
    for (int64_t s = least; s <= std::max<int64_t>(64, least) && s <= steps; ++s) {
        const int64_t per = ceil_div(steps, s), splits = ceil_div(steps, per);
        if (splits != s) continue;      // the same pieces as with fewer splits
        const double us = 0.3 * static_cast<double>(ceil_div(tiles * s, 74)) * static_cast<double>(per + 4) +
                          (s > 1 ? 3.0 + 8e-6 / 4 * static_cast<double>(s * B * M * N) : 0.0);
        if (s == least || us < best_us) {
            best = s;
            best_us = us;
        }
    }
    return best;
}

// fp16 and bf16 run on the tensor cores. Rows that are no multiple of 16 bytes are copied to padded
// ones first; rows that are, but in a buffer that does not start on 16 bytes, take the CUDA cores.
inline int64_t padded(int64_t d, km_dtype dt) { return dt == KM_F32 ? d : ceil_div(d, 8) * 8; }
// (A scale of zero takes them too: the tensor-core epilogue keeps its maximum before the scaling.)
inline bool use_tc(km_dtype dt, int64_t d, float scale, const void *X, const void *C) {
    return dt != KM_F32 && scale != 0.f && (d % 8 != 0 || (aligned(X, 16) && aligned(C, 16))) && encode_fn() != nullptr;
}

// A logit is one chain of truncating additions (loss at d = 1024, 8192 and 65536 off by 5e-7, 4e-6 and 4e-5 of itself,
// in terms of both signs): rows of more than kMaxChain products are summed on the CUDA cores, rounded to nearest.
inline bool logits_on_tc(int64_t d) { return d <= kMaxChain * 16; }

struct LossWs {
    float2 *pairs;
    float *zt;
    void *X, *C;    // padded copies, or null
};
inline LossWs carve_loss(Carver &c, int64_t B, int64_t N, int64_t K, int64_t d, km_dtype dt) {
    LossWs w;
    const int64_t dp = padded(d, dt);
    w.X = dp != d ? c.take<uint8_t>(static_cast<size_t>(B * N * dp) * 2) : nullptr;
    w.C = dp != d ? c.take<uint8_t>(static_cast<size_t>(B * K * dp) * 2) : nullptr;
    w.pairs = c.take<float2>(static_cast<size_t>(B * ceil_div(K, ST) * N) * 8);
    w.zt = c.take<float>(static_cast<size_t>(B * N) * 4);
    return w;
}

// Gradients of rows of up to 128 16-bit values take the fused form (three tiles of S and one of O fill
// TMEM; longer rows leave the exponentials the smaller part). 32768 points x 8192 rows at d = 128: dX
// 146 us against 270 through P in memory, dC 155 against 268; 20000 x 300: dX 31 against 27, dC 31 against
// 36; 100000 x 64 at d = 32: dX 38 against 39, dC 48 against 50.
inline bool fused_shape(km_dtype dt, int64_t d) { return dt != KM_F32 && d <= 128; }
// Blocks of one gradient: all SMs, but two tiles at least for each.
// (The tiles of both directions number the same, below 2^31 by xent_sizes_ok.)
inline int fused_tiles(int64_t B, int64_t M, int64_t cols) {
    static_assert(FR == ST, "xent_sizes_ok counts tiles of ST");
    return static_cast<int>(B * ceil_div(M, FR) * ceil_div(cols, FR));
}
inline int fused_blocks(int tiles) { return std::min(num_sms(), tiles / 2 + tiles % 2); }
struct FusedWs {
    void *X, *C;
    float *w, *parts;
    unsigned int *wmax;
    PointTile *points;
    PointRow *rows;
    int64_t ptiles;
};
inline FusedWs carve_fused(Carver &c, int64_t B, int64_t N, int64_t K, int64_t d, km_dtype dt) {
    FusedWs f;
    const int64_t dp = padded(d, dt);
    f.ptiles = ceil_div(N, FR);
    f.X = c.take<uint8_t>(static_cast<size_t>(B * N * dp) * 2);
    f.C = c.take<uint8_t>(static_cast<size_t>(B * K * dp) * 2);
    f.w = c.take<float>(static_cast<size_t>(B * N) * 4);
    f.wmax = c.take<unsigned int>(kStats * 4);
    f.points = c.take<PointTile>(static_cast<size_t>(B * f.ptiles) * sizeof(PointTile));
    f.rows = c.take<PointRow>(static_cast<size_t>(B * f.ptiles) * FR * sizeof(PointRow));
    f.parts = c.take<float>(static_cast<size_t>(fused_blocks(fused_tiles(B, N, K))) * 2 * FR * (d > 64 ? 128 : 64) * 4);
    return f;
}

struct GradWs {
    void *P, *X, *C;
    void *Xs;       // (fp16) the points as dC sums them, where X is a padded copy already
    float *w, *parts, *dxacc;
    unsigned int *wmax;
};
inline GradWs carve_grad(Carver &c, int64_t B, int64_t N, int64_t K, int64_t d, km_dtype dt) {
    GradWs g;
    const int64_t kc = piece_rows(B, N, K);
    g.P = c.take<uint8_t>(static_cast<size_t>(B * N * kc) * dtype_size(dt));
    const int64_t dp = padded(d, dt);
    g.X = c.take<uint8_t>(static_cast<size_t>(B * N * dp) * dtype_size(dt));
    g.C = dp != d ? c.take<uint8_t>(static_cast<size_t>(B * K * dp) * 2) : nullptr;
    g.Xs = dp != d && dt == KM_F16 ? c.take<uint8_t>(static_cast<size_t>(B * N * dp) * 2) : g.X;
    g.w = c.take<float>(static_cast<size_t>(B * N) * 4);
    g.wmax = c.take<unsigned int>(kStats * 4);
    int64_t parts = 0;
    for (int64_t k0 = 0; k0 < K; k0 += kc) {
        const int64_t kn = std::min(kc, K - k0);
        const int64_t sx = product_splits(B, N, d, kn, dt), nb = kn == K ? B : 1;
        const int64_t sc = product_splits(nb, kn, d, N, dt);
        if (sx > 1) parts = std::max(parts, sx * B * N * d);
        if (sc > 1) parts = std::max(parts, sc * nb * kn * d);
        if (k0 == 0 && K - k0 > 2 * kc) k0 += (K - k0 - 2 * kc) / kc * kc;   // whole pieces are alike
    }
    g.parts = c.take<float>(static_cast<size_t>(parts) * 4);
    g.dxacc = c.take<float>(kc < K ? static_cast<size_t>(B * N * d) * 4 : 0);
    return g;
}

template <typename T, int MODE>
km_status simt_product(const Operand &A, const Operand &Bo, int64_t B, int64_t M, int64_t N, int64_t Kk, Epi p,
                       int64_t splits, cudaStream_t st) {
    const int64_t mt = ceil_div(M, ST), nt = ceil_div(N, ST);
    const int64_t kper = ceil_div(ceil_div(Kk, TKC), splits) * TKC;
    p.splits = static_cast<int>(splits);
    const int64_t blocks = mt * nt * splits * B;
    if (blocks > kMaxIndex) return KM_ERR_UNSUPPORTED;
    simt_product_kernel<T, MODE><<<static_cast<unsigned>(blocks), kSimtThreads, 0, st>>>(
        A, Bo, static_cast<int>(M), static_cast<int>(N), Kk, static_cast<int>(mt), static_cast<int>(nt), kper, p);
    return launch_status();
}

// Tensor map of an operand: K-major boxes of 64 reduction steps x `rows`, MN-major boxes of 64 rows
// x 64 reduction steps. Every box starts on a multiple of 64 elements of its contiguous index.
inline bool encode_operand(CUtensorMap *tm, CUtensorMapDataType tdt, const Operand &o, int64_t rows_total, int64_t Kk,
                           int64_t B, int rows) {
    const bool mn = o.k_s != 1;
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(mn ? rows_total : Kk),
                                static_cast<cuuint64_t>(mn ? Kk : rows_total), static_cast<cuuint64_t>(B)};
    const int64_t ld = mn ? o.k_s : o.row_s;
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(ld * 2), static_cast<cuuint64_t>(o.batch * 2)};
    const cuuint32_t box[3] = {TKC, static_cast<cuuint32_t>(mn ? TKC : rows), 1};
    const cuuint32_t estr[3] = {1, 1, 1};
    return encode_fn()(tm, tdt, 3, const_cast<void *>(o.base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                       CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                       CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename T, int MODE, bool AMN, bool BMN>
km_status tc_launch(const Operand &A, const Operand &Bo, int64_t B, int64_t M, int64_t N, int64_t Kk, Epi e,
                    int64_t splits, cudaStream_t st) {
    using Sh = TcShape<MODE>;
    const bool bf16 = std::is_same<T, __nv_bfloat16>::value;
    const CUtensorMapDataType tdt = bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
    CUtensorMap tmA, tmB;
    if (!encode_operand(&tmA, tdt, A, M, Kk, B, TBM) || !encode_operand(&tmB, tdt, Bo, N, Kk, B, TBN / 2))
        return KM_ERR_CUDA;
    CUtensorMap tmP = tmA;      // (read where P is written only)
    if (MODE == kProb) {
        const cuuint64_t dims[3] = {static_cast<cuuint64_t>(e.ldp), static_cast<cuuint64_t>(M), static_cast<cuuint64_t>(B)};
        const cuuint64_t strides[2] = {static_cast<cuuint64_t>(e.ldp * 2), static_cast<cuuint64_t>(M * e.ldp * 2)};
        const cuuint32_t box[3] = {64, 32, 1}, estr[3] = {1, 1, 1};
        if (encode_fn()(&tmP, tdt, 3, e.P, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                        CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
            return KM_ERR_CUDA;
    }
    auto kernel = tc_product_kernel<T, MODE, AMN, BMN>;
    static std::atomic<uint64_t> ready{0};
    if (!allow_smem(kernel, Sh::kTotal, ready)) return KM_ERR_CUDA;
    // persistent SM pairs: as many as can be resident (a pair needs two SMs of one GPC)
    static int resident[64] = {0};
    int dev = 0;
    cudaGetDevice(&dev);
    int clusters = (dev >= 0 && dev < 64) ? resident[dev] : 0;
    if (clusters <= 0) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(static_cast<unsigned>(2 * std::max(1, num_sms() / 2)));
        cfg.blockDim = dim3(T_THREADS);
        cfg.dynamicSmemBytes = Sh::kTotal;
        cudaLaunchAttribute attr;
        attr.id = cudaLaunchAttributeClusterDimension;
        attr.val.clusterDim.x = 2;
        attr.val.clusterDim.y = 1;
        attr.val.clusterDim.z = 1;
        cfg.attrs = &attr;
        cfg.numAttrs = 1;
        if (cudaOccupancyMaxActiveClusters(&clusters, kernel, &cfg) != cudaSuccess || clusters <= 0) {
            cudaGetLastError();
            clusters = std::max(1, num_sms() / 2);
        }
        if (dev >= 0 && dev < 64) resident[dev] = clusters;
    }
    TcParams p = {};
    p.M = static_cast<int>(M);
    p.N = static_cast<int>(N);
    p.mt = static_cast<int>(ceil_div(M, 2 * TBM));
    p.nt = static_cast<int>(ceil_div(N, TBN));
    p.nb = static_cast<int>(B);
    p.Kk = static_cast<int>(Kk);
    p.kchunks = static_cast<int>(ceil_div(Kk, TKC));
    p.kper = static_cast<int>(ceil_div(p.kchunks, splits));
    p.idesc = km::mma_idesc_f16(bf16 ? 1u : 0u, 2 * TBM, TBN) | (AMN ? 1u << 15 : 0u) | (BMN ? 1u << 16 : 0u) |
              (MODE != kOut && e.scale < 0.f ? 1u << 13 : 0u);   // bit 13 negates A
    p.vec = N % 8 == 0 && (!e.outT || aligned(e.outT, 16)) ? 1 : 0;
    p.withhold = km::g_withhold;
    e.splits = static_cast<int>(splits);
    const int64_t items = static_cast<int64_t>(p.mt) * p.nt * splits * B;
    if (items > kMaxIndex) return KM_ERR_UNSUPPORTED;
    p.div_split = km::make_fastdiv(static_cast<uint32_t>(p.mt * p.nt));
    p.div_batch = km::make_fastdiv(static_cast<uint32_t>(p.mt * p.nt * splits));
    p.div_group = km::make_fastdiv(static_cast<uint32_t>(T_GROUP * p.nt));
    p.div_last = km::make_fastdiv(static_cast<uint32_t>(p.mt % T_GROUP ? p.mt % T_GROUP : T_GROUP));
    const unsigned grid = static_cast<unsigned>(2 * std::min<int64_t>(items, clusters));
    kernel<<<grid, T_THREADS, Sh::kTotal, st>>>(tmA, tmB, tmP, p, e);
    return launch_status();
}

template <typename T, int MODE>
km_status product(bool tc, const Operand &A, const Operand &Bo, int64_t B, int64_t M, int64_t N, int64_t Kk,
                  const Epi &p, int64_t splits, cudaStream_t st) {
    if constexpr (!std::is_same<T, float>::value) {
        if (tc) {
            if constexpr (MODE != kOut) {
                return tc_launch<T, MODE, false, false>(A, Bo, B, M, N, Kk, p, splits, st);
            } else {
                if (A.k_s == 1) return tc_launch<T, kOut, false, true>(A, Bo, B, M, N, Kk, p, splits, st);   // dX = P C
                return tc_launch<T, kOut, true, true>(A, Bo, B, M, N, Kk, p, splits, st);
            }
        }
    }
    return simt_product<T, MODE>(A, Bo, B, M, N, Kk, p, splits, st);
}

inline unsigned fill_blocks(int64_t n) {
    return static_cast<unsigned>(std::max<int64_t>(1, std::min<int64_t>(ceil_div(n, 256), 148 * 16)));
}

// out = A B (+ acc), through split partials where the reduction is split.
template <typename T>
km_status out_product(bool tc, km_dtype dt, const Operand &A, const Operand &Bo, int64_t B, int64_t M, int64_t N,
                      int64_t Kk, Epi p, float *parts, cudaStream_t st) {
    const int64_t splits = product_splits(B, M, N, Kk, dt);
    if (splits == 1) return product<T, kOut>(tc, A, Bo, B, M, N, Kk, p, 1, st);
    Epi q = p;
    q.out32 = parts;
    q.outT = nullptr;
    km_status s = product<T, kOut>(tc, A, Bo, B, M, N, Kk, q, splits, st);
    if (s != KM_OK) return s;
    const int64_t v = N % 4 == 0 && (!p.outT || aligned(p.outT, 4 * sizeof(T))) ? 4 : 1, units = B * M * N / v;
    const km::FastDiv per_row = km::make_fastdiv(static_cast<uint32_t>(N / v));
    auto kernel = v == 4 ? split_join_kernel<T, 4> : split_join_kernel<T, 1>;
    kernel<<<fill_blocks(units), 256, 0, st>>>(parts, static_cast<int>(splits), units, per_row, p);
    return launch_status();
}

template <typename T>
km_status copy_rows(const void *src, const int32_t *ids, int64_t rows, int64_t d, int64_t dp, int64_t K, void *dst,
                    cudaStream_t st) {
    const int64_t v = 16 / sizeof(T);
    if (d == dp && d % v == 0 && aligned(src, 16) && aligned(dst, 16))
        copy_rows_kernel<uint4><<<fill_blocks(rows * d / v), 256, 0, st>>>(
            static_cast<const uint4 *>(src), ids, rows, static_cast<int>(d / v),
            km::make_fastdiv(static_cast<uint32_t>(d / v)), static_cast<int>(K), static_cast<uint4 *>(dst));
    else
        copy_rows_kernel<T><<<fill_blocks(rows * dp), 256, 0, st>>>(
            static_cast<const T *>(src), ids, rows, static_cast<int>(d), km::make_fastdiv(static_cast<uint32_t>(dp)),
            static_cast<int>(K), static_cast<T *>(dst));
    return launch_status();
}

template <typename T>
km_status loss_typed(const void *X, km_dtype dt, const void *C, const int32_t *ids, int64_t B, int64_t N, int64_t K,
                     int64_t d, float scale, float *loss, float *lse, const LossWs &w, cudaStream_t st) {
    const bool tc = use_tc(dt, d, scale, X, C) && logits_on_tc(d);
    const int64_t dp = tc ? padded(d, dt) : d;
    km_status s;
    if (dp != d) {
        if ((s = copy_rows<T>(X, nullptr, B * N, d, dp, K, w.X, st)) != KM_OK) return s;
        if ((s = copy_rows<T>(C, nullptr, B * K, d, dp, K, w.C, st)) != KM_OK) return s;
        X = w.X;
        C = w.C;
    }
    Epi p = {};
    p.scale = scale;
    p.pairs = w.pairs;
    p.zt = w.zt;
    p.ids = ids;
    p.K = static_cast<int>(K);
    s = product<T, kLse>(tc, Operand{X, N * dp, dp, 1}, Operand{C, K * dp, dp, 1}, B, N, K, dp, p, 1, st);
    if (s != KM_OK) return s;
    lse_join_kernel<<<static_cast<unsigned>(B * ceil_div(N, 32)), 256, 0, st>>>(
        w.pairs, w.zt, ids, B, static_cast<int>(N), static_cast<int>(K), static_cast<int>(ceil_div(K, ST)), loss, lse);
    return launch_status();
}

// One gradient of the fused form: rows of A against all rows of B.
template <typename T, int DN, bool COL, bool LO>
km_status fused_launch(const void *A, const void *Bo, int64_t B, int64_t M, int64_t cols, int64_t d, int64_t dp, float scale,
                       const FusedWs &w, float pscale, void *out, cudaStream_t st) {
    using Sh = FShape<DN, COL>;
    const bool bf16 = std::is_same<T, __nv_bfloat16>::value;
    const CUtensorMapDataType tdt = bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
    CUtensorMap tmA, tmB;
    if (!encode_operand(&tmA, tdt, Operand{A, M * dp, dp, 1}, M, dp, B, FR) ||
        !encode_operand(&tmB, tdt, Operand{Bo, cols * dp, dp, 1}, cols, dp, B, FR))
        return KM_ERR_CUDA;
    auto kernel = fused_grad_kernel<T, DN, COL, LO>;
    static std::atomic<uint64_t> ready{0};
    if (!allow_smem(kernel, Sh::kTotal, ready)) return KM_ERR_CUDA;
    FParams p = {};
    p.M = static_cast<int>(M);
    p.cols = static_cast<int>(cols);
    p.d = static_cast<int>(d);
    p.mt = static_cast<int>(ceil_div(M, FR));
    p.ct = static_cast<int>(ceil_div(cols, FR));
    p.tiles = fused_tiles(B, M, cols);
    p.scale = std::fabs(scale);
    p.idesc_s = km::mma_idesc_f16(bf16 ? 1u : 0u, FR, FR) | (scale < 0.f ? 1u << 13 : 0u);   // bit 13 negates A
    p.idesc_o = km::mma_idesc_f16(bf16 ? 1u : 0u, FR, DN) | (1u << 16);                      // B MN-major
    p.points = w.points;
    p.rows = w.rows;
    p.wmax = w.wmax;
    p.pscale = pscale;
    p.withhold = km::g_withhold;
    p.parts = w.parts;
    p.out = out;
    p.vec = d % 8 == 0 && aligned(out, 16) ? 1 : 0;
    const int blocks = fused_blocks(p.tiles);
    kernel<<<blocks, F_THREADS, Sh::kTotal, st>>>(tmA, tmB, p);
    const km_status launched = launch_status();      // (reading the error clears it)
    if (launched != KM_OK || blocks == 1) return launched;
    // (nothing to join where the blocks' shares are whole row tiles)
    if (p.tiles % blocks == 0 && p.tiles / blocks % p.ct == 0) return KM_OK;
    const int rows = p.tiles / p.ct;
    auto join = [&](auto parts, int units) {
        constexpr int PARTS = decltype(parts)::value;
        fused_join_kernel<T, DN, PARTS><<<static_cast<unsigned>(units) * (FR * PARTS / 4), DN, 0, st>>>(
            w.parts, p.tiles, blocks, p.M, p.d, p.mt, p.ct, COL ? nullptr : w.rows, w.wmax, pscale,
            static_cast<T *>(out));
    };
    // (from 16 blocks to a row tile on, its partials are worth sharing out)
    if (blocks >= 16 * rows) join(std::integral_constant<int, 4>(), rows);
    else join(std::integral_constant<int, 1>(), blocks - 1);
    return launch_status();
}

template <typename T, bool LO>
km_status fused_both(const void *X, const void *C, int64_t B, int64_t N, int64_t K, int64_t d, int64_t dp, float scale,
                     const FusedWs &w, float pscale, void *dX, void *dC, cudaStream_t st) {
    if (dX) {
        const km_status s = d > 64 ? fused_launch<T, 128, false, LO>(X, C, B, N, K, d, dp, scale, w, pscale, dX, st)
                                   : fused_launch<T, 64, false, LO>(X, C, B, N, K, d, dp, scale, w, pscale, dX, st);
        if (s != KM_OK) return s;
    }
    if (!dC) return KM_OK;
    return d > 64 ? fused_launch<T, 128, true, LO>(C, X, B, K, N, d, dp, scale, w, pscale, dC, st)
                  : fused_launch<T, 64, true, LO>(C, X, B, K, N, d, dp, scale, w, pscale, dC, st);
}

template <typename T>
km_status fused_grads(const void *X, km_dtype dt, const void *C, const int32_t *ids, const float *lse, const float *g,
                      int64_t B, int64_t N, int64_t K, int64_t d, float scale, void *dX, void *dC, void *ws,
                      cudaStream_t st) {
    if (!encode_fn()) return KM_ERR_CUDA;
    Carver cv(ws);
    const FusedWs w = carve_fused(cv, B, N, K, d, dt);
    const int64_t dp = padded(d, dt);
    const float pscale = dt == KM_F16 ? 16384.f : 1.f;
    km_status s;
    if (cudaMemsetAsync(w.wmax, 0, kStats * 4, st) != cudaSuccess) return KM_ERR_CUDA;
    km::xe::weight_kernel<<<static_cast<unsigned>(ceil_div(B * N, 256)), 256, 0, st>>>(
        g, ids, B * N, static_cast<int>(K), scale, w.w, w.wmax, false);
    if (launch_status() != KM_OK) return KM_ERR_CUDA;
    point_param_kernel<<<fill_blocks(B * w.ptiles * FR), 256, 0, st>>>(w.w, lse, ids, B, static_cast<int>(N), w.ptiles,
                                                                static_cast<int>(K), w.wmax, pscale, w.points, w.rows);
    if (launch_status() != KM_OK) return KM_ERR_CUDA;
    // points without a label become zeros, so that nothing they hold reaches a sum
    if ((s = copy_rows<T>(X, ids, B * N, d, dp, K, w.X, st)) != KM_OK) return s;
    X = w.X;
    if (dp != d || !aligned(C, 16)) {
        if ((s = copy_rows<T>(C, nullptr, B * K, d, dp, K, w.C, st)) != KM_OK) return s;
        C = w.C;
    }
    // Few table rows: P in two parts. The gradients' errors against 64 bits are then the rounding of the
    // result alone (with one part 1.2 to 1.5 times that); 100000 x 64 at d = 32: dX 40 us, dC 37, in one
    // part 37 and 46; 30000 x 8 at d = 64: 23 and 25, in one 21 and 35.
    if (K <= FR) return fused_both<T, true>(X, C, B, N, K, d, dp, scale, w, pscale, dX, dC, st);
    return fused_both<T, false>(X, C, B, N, K, d, dp, scale, w, pscale, dX, dC, st);
}

template <typename T>
km_status grad_typed(const void *X, km_dtype dt, const void *C, const int32_t *ids, const float *lse, const float *g,
                     int64_t B, int64_t N, int64_t K, int64_t d, float scale, void *dX, void *dC, void *ws,
                     cudaStream_t st) {
    if constexpr (!std::is_same<T, float>::value)
        if (fused_shape(dt, d)) return fused_grads<T>(X, dt, C, ids, lse, g, B, N, K, d, scale, dX, dC, ws, st);
    Carver cv(ws);
    const GradWs w = carve_grad(cv, B, N, K, d, dt);
    const bool tc = use_tc(dt, d, scale, X, C);
    const int64_t dp = tc ? padded(d, dt) : d;
    km_status s;
    unsigned int *wmax = dt != KM_F32 ? w.wmax : nullptr;
    const float pscale = dt == KM_F16 ? 16384.f : 1.f;
    if (wmax && cudaMemsetAsync(wmax, 0, kStats * 4, st) != cudaSuccess) return KM_ERR_CUDA;
    km::xe::weight_kernel<<<static_cast<unsigned>(ceil_div(B * N, 256)), 256, 0, st>>>(
        g, ids, B * N, static_cast<int>(K), scale, w.w, wmax, kShifts<T>);
    if (launch_status() != KM_OK) return KM_ERR_CUDA;
    // points without a label become zeros here, so that nothing they hold reaches dC
    const void *Xc = w.X;         // the points as dC sums them
    if constexpr (kShifts<T>) {
        if (dC) {
            Xc = w.Xs;
            max_point_kernel<<<static_cast<unsigned>(std::min<int64_t>(B * N, 148 * 8)), 256, 0, st>>>(
                static_cast<const __half *>(X), ids, B * N, static_cast<int>(d), static_cast<int>(K), wmax);
            if (launch_status() != KM_OK) return KM_ERR_CUDA;
            const bool whole = d % 8 == 0 && aligned(X, 16);
            auto kernel = whole ? shift_points_kernel<8> : shift_points_kernel<1>;
            const int64_t per = whole ? dp / 8 : dp;
            kernel<<<fill_blocks(B * N * per), 256, 0, st>>>(
                static_cast<const __half *>(X), ids, w.w, B * N, static_cast<int>(d),
                km::make_fastdiv(static_cast<uint32_t>(per)), static_cast<int>(K), wmax, static_cast<__half *>(w.Xs));
            if (launch_status() != KM_OK) return KM_ERR_CUDA;
        }
        if (dp != d) {
            if ((s = copy_rows<T>(X, ids, B * N, d, dp, K, w.X, st)) != KM_OK) return s;
            X = w.X;
        }
    } else if (dC || dp != d) {
        if ((s = copy_rows<T>(X, ids, B * N, d, dp, K, w.X, st)) != KM_OK) return s;
        X = w.X;
    }
    if (dp != d) {
        if ((s = copy_rows<T>(C, nullptr, B * K, d, dp, K, w.C, st)) != KM_OK) return s;
        C = w.C;
    }
    const int64_t kc = piece_rows(B, N, K);
    for (int64_t k0 = 0; k0 < K; k0 += kc) {
        const int64_t kn = std::min(kc, K - k0);
        const T *Ck = static_cast<const T *>(C) + k0 * dp;
        Epi p = {};
        p.scale = scale;
        p.ids = ids;
        p.k0 = static_cast<int>(k0);
        p.K = static_cast<int>(K);
        p.lse = lse;
        p.w = w.w;
        p.P = w.P;
        p.ldp = kc;
        p.wmax = wmax;
        p.pscale = pscale;
        s = product<T, kProb>(tc && logits_on_tc(d), Operand{X, N * dp, dp, 1}, Operand{Ck, K * dp, dp, 1}, B, N, kn, dp, p, 1, st);
        if (s != KM_OK) return s;
        if (dX) {
            Epi q = {};
            q.wmax = wmax;
            q.pscale = pscale;
            q.rows = true;
            q.w = w.w;
            q.acc = k0 ? w.dxacc : nullptr;
            if (k0 + kc < K) q.out32 = w.dxacc;
            else q.outT = dX;
            s = out_product<T>(tc, dt, Operand{w.P, N * kc, kc, 1}, Operand{Ck, K * dp, 1, dp}, B, N, d, kn, q, w.parts,
                               st);
            if (s != KM_OK) return s;
        }
        if (dC) {
            // the pieces of dC are K * d apart between batches: one product per batch unless the
            // piece is the whole table
            Epi q = {};
            q.wmax = wmax;
            q.pscale = pscale;
            const int64_t nb = kn == K ? B : 1;
            for (int64_t b = 0; b < B; b += nb) {
                q.outT = static_cast<T *>(dC) + (b * K + k0) * d;
                s = out_product<T>(tc, dt, Operand{static_cast<const T *>(w.P) + b * N * kc, N * kc, 1, kc},
                                   Operand{static_cast<const T *>(Xc) + b * N * dp, N * dp, 1, dp}, nb, kn, d, N, q,
                                   w.parts, st);
                if (s != KM_OK) return s;
            }
        }
    }
    return KM_OK;
}

}  // namespace

namespace km {
namespace xe {

cudaError_t take_device_error(unsigned int *bits) {
    const unsigned int zero = 0;
    const cudaError_t e = cudaMemcpyFromSymbol(bits, g_km_dev_error, sizeof(*bits));
    return e != cudaSuccess ? e : cudaMemcpyToSymbol(g_km_dev_error, &zero, sizeof(zero));
}
cudaError_t set_wait_limit(unsigned long long limit_ns) {
    return cudaMemcpyToSymbol(g_km_wait_limit_ns, &limit_ns, sizeof(limit_ns));
}

}  // namespace xe
}  // namespace km

extern "C" {

size_t km_xent_workspace_size(int64_t B, int64_t N, int64_t K, int64_t d, km_dtype dtype) {
    if (!valid_dtype(dtype) || !xent_sizes_ok(B, N, K, d)) return 0;
    Carver c(nullptr);
    carve_loss(c, B, N, K, d, dtype);
    return c.off;
}

km_status km_xent(const void *X, km_dtype dtype, const void *C, const int32_t *ids, int64_t B, int64_t N, int64_t K,
                  int64_t d, float scale, float *loss, float *lse, void *ws, size_t ws_bytes, void *stream) {
    if (!X || !C || !ids || (!loss && !lse) || !valid_dtype(dtype) || !sizes_ok(B, N, K, d) ||
        !aligned(X, dtype_size(dtype)) || !aligned(C, dtype_size(dtype)) || !aligned(ids, 4) ||
        (loss && !aligned(loss, 4)) || (lse && !aligned(lse, 4)) || (ws && !aligned(ws, kAlign)))
        return KM_ERR_INVALID_ARG;
    if (!xent_sizes_ok(B, N, K, d)) return KM_ERR_UNSUPPORTED;
    if (!ws || ws_bytes < km_xent_workspace_size(B, N, K, d, dtype)) return KM_ERR_WORKSPACE;
    Carver c(ws);
    const LossWs w = carve_loss(c, B, N, K, d, dtype);
    switch (dtype) {
        case KM_F32: return loss_typed<float>(X, dtype, C, ids, B, N, K, d, scale, loss, lse, w, S(stream));
        case KM_F16: return loss_typed<__half>(X, dtype, C, ids, B, N, K, d, scale, loss, lse, w, S(stream));
        default: return loss_typed<__nv_bfloat16>(X, dtype, C, ids, B, N, K, d, scale, loss, lse, w, S(stream));
    }
}

size_t km_xent_grad_workspace_size(int64_t B, int64_t N, int64_t K, int64_t d, km_dtype dtype) {
    if (!valid_dtype(dtype) || !xent_sizes_ok(B, N, K, d)) return 0;
    Carver c(nullptr);
    if (fused_shape(dtype, d)) carve_fused(c, B, N, K, d, dtype);
    else carve_grad(c, B, N, K, d, dtype);
    return c.off;
}

km_status km_xent_grad(const void *X, km_dtype dtype, const void *C, const int32_t *ids, const float *lse,
                       const float *g, int64_t B, int64_t N, int64_t K, int64_t d, float scale, void *dX, void *dC,
                       void *ws, size_t ws_bytes, void *stream) {
    if (!X || !C || !ids || !lse || (!dX && !dC) || !valid_dtype(dtype) || !sizes_ok(B, N, K, d) ||
        !aligned(X, dtype_size(dtype)) || !aligned(C, dtype_size(dtype)) || !aligned(ids, 4) || !aligned(lse, 4) ||
        (g && !aligned(g, 4)) || (dX && !aligned(dX, dtype_size(dtype))) ||
        (dC && !aligned(dC, dtype_size(dtype))) || (ws && !aligned(ws, kAlign)))
        return KM_ERR_INVALID_ARG;
    if (!xent_sizes_ok(B, N, K, d)) return KM_ERR_UNSUPPORTED;
    if (!ws || ws_bytes < km_xent_grad_workspace_size(B, N, K, d, dtype)) return KM_ERR_WORKSPACE;
    switch (dtype) {
        case KM_F32: return grad_typed<float>(X, dtype, C, ids, lse, g, B, N, K, d, scale, dX, dC, ws, S(stream));
        case KM_F16: return grad_typed<__half>(X, dtype, C, ids, lse, g, B, N, K, d, scale, dX, dC, ws, S(stream));
        default: return grad_typed<__nv_bfloat16>(X, dtype, C, ids, lse, g, B, N, K, d, scale, dX, dC, ws, S(stream));
    }
}

}  // extern "C"
