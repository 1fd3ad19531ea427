// km_xent.cu -- softmax cross entropy over a table: C entry points, workspaces and launches
// (kernels in km_xent.cuh).
#include "km_host.h"
#include "km_xent.cuh"

namespace {

using namespace km::xe;

constexpr int64_t kPieceElems = int64_t{1} << 27;   // entries of P held at a time (256 MiB of 16-bit)
constexpr int kPieceStep = 256;

inline bool xent_sizes_ok(int64_t B, int64_t N, int64_t K, int64_t d) {
    return sizes_ok(B, N, K, d) && N <= kMaxIndex - 1024 && K <= kMaxIndex - 1024 && B * N <= kMaxIndex &&
           B * ceil_div(N, ST) * ceil_div(K, ST) <= kMaxIndex;
}

struct LossWs {
    float2 *pairs;
    float *zt;
};
inline LossWs carve_loss(Carver &c, int64_t B, int64_t N, int64_t K) {
    LossWs w;
    w.pairs = c.take<float2>(static_cast<size_t>(B * ceil_div(K, ST) * N) * 8);
    w.zt = c.take<float>(static_cast<size_t>(B * N) * 4);
    return w;
}

// Table rows per piece of the gradient.
inline int64_t piece_rows(int64_t B, int64_t N, int64_t K) {
    const int64_t all = ceil_div(K, kPieceStep) * kPieceStep;
    const int64_t fit = kPieceElems / (B * N) / kPieceStep * kPieceStep;
    return std::min(all, std::max<int64_t>(kPieceStep, fit));
}
// Splits of a product's reduction: only where the output tiles alone leave SMs idle, each split
// at least 512 long.
inline int64_t product_splits(int64_t B, int64_t M, int64_t N, int64_t Kk) {
    const int64_t tiles = B * ceil_div(M, ST) * ceil_div(N, ST);
    if (tiles >= 148) return 1;
    return std::max<int64_t>(1, std::min(ceil_div(2 * 148, tiles), Kk / 512));
}

struct GradWs {
    void *P, *X;
    float *w, *parts, *dxacc;
    unsigned int *wmax;
};
inline GradWs carve_grad(Carver &c, int64_t B, int64_t N, int64_t K, int64_t d, km_dtype dt) {
    GradWs g;
    const int64_t kc = piece_rows(B, N, K);
    g.P = c.take<uint8_t>(static_cast<size_t>(B * N * kc) * dtype_size(dt));
    g.X = c.take<uint8_t>(static_cast<size_t>(B * N * d) * dtype_size(dt));
    g.w = c.take<float>(static_cast<size_t>(B * N) * 4);
    g.wmax = c.take<unsigned int>(4);
    int64_t parts = 0;
    for (int64_t k0 = 0; k0 < K; k0 += kc) {
        const int64_t kn = std::min(kc, K - k0);
        const int64_t sx = product_splits(B, N, d, kn), nb = kn == K ? B : 1;
        const int64_t sc = product_splits(nb, kn, d, N);
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
    const int64_t kper = ceil_div(ceil_div(Kk, splits), SK) * SK;
    p.splits = static_cast<int>(splits);
    const int64_t blocks = mt * nt * splits * B;
    if (blocks > kMaxIndex) return KM_ERR_UNSUPPORTED;
    simt_product_kernel<T, MODE><<<static_cast<unsigned>(blocks), kSimtThreads, 0, st>>>(
        A, Bo, static_cast<int>(M), static_cast<int>(N), Kk, static_cast<int>(mt), static_cast<int>(nt), kper, p);
    return launch_status();
}

inline unsigned fill_blocks(int64_t n) {
    return static_cast<unsigned>(std::max<int64_t>(1, std::min<int64_t>(ceil_div(n, 256), 148 * 16)));
}

// out = A B (+ acc), through split partials where the reduction is split.
template <typename T>
km_status out_product(const Operand &A, const Operand &Bo, int64_t B, int64_t M, int64_t N, int64_t Kk, Epi p,
                      float *parts, cudaStream_t st) {
    const int64_t splits = product_splits(B, M, N, Kk);
    if (splits == 1) return simt_product<T, kOut>(A, Bo, B, M, N, Kk, p, 1, st);
    Epi q = p;
    q.out32 = parts;
    km_status s = simt_product<T, kOut>(A, Bo, B, M, N, Kk, q, splits, st);
    if (s != KM_OK) return s;
    split_join_kernel<T><<<fill_blocks(B * M * N), 256, 0, st>>>(parts, static_cast<int>(splits), B * M * N, p);
    return launch_status();
}

template <typename T>
km_status loss_typed(const void *X, const void *C, const int32_t *ids, int64_t B, int64_t N, int64_t K, int64_t d,
                     float scale, float *loss, float *lse, const LossWs &w, cudaStream_t st) {
    Epi p = {};
    p.scale = scale;
    p.pairs = w.pairs;
    p.zt = w.zt;
    p.ids = ids;
    p.K = static_cast<int>(K);
    const Operand A = {X, N * d, d, 1}, Bo = {C, K * d, d, 1};
    km_status s = simt_product<T, kLse>(A, Bo, B, N, K, d, p, 1, st);
    if (s != KM_OK) return s;
    lse_join_kernel<<<static_cast<unsigned>(B * ceil_div(N, 32)), 256, 0, st>>>(
        w.pairs, w.zt, ids, B, static_cast<int>(N), static_cast<int>(K), static_cast<int>(ceil_div(K, ST)), loss, lse);
    return launch_status();
}

template <typename T>
km_status grad_typed(const void *X, km_dtype dt, const void *C, const int32_t *ids, const float *lse, const float *g,
                     int64_t B, int64_t N, int64_t K, int64_t d, float scale, void *dX, void *dC, void *ws,
                     cudaStream_t st) {
    Carver cv(ws);
    const GradWs w = carve_grad(cv, B, N, K, d, dt);
    unsigned int *wmax = dt == KM_F16 ? w.wmax : nullptr;
    if (wmax && cudaMemsetAsync(wmax, 0, 4, st) != cudaSuccess) return KM_ERR_CUDA;
    km::xe::weight_kernel<<<static_cast<unsigned>(ceil_div(B * N, 256)), 256, 0, st>>>(
        g, ids, B * N, static_cast<int>(K), scale, w.w, wmax);
    if (launch_status() != KM_OK) return KM_ERR_CUDA;
    if (dC) {
        copy_rows_kernel<T><<<fill_blocks(B * N * d), 256, 0, st>>>(
            static_cast<const T *>(X), ids, B * N, static_cast<int>(d), static_cast<int>(d), static_cast<int>(K),
            static_cast<T *>(w.X));
        if (launch_status() != KM_OK) return KM_ERR_CUDA;
    }
    const int64_t kc = piece_rows(B, N, K);
    for (int64_t k0 = 0; k0 < K; k0 += kc) {
        const int64_t kn = std::min(kc, K - k0);
        const T *Ck = static_cast<const T *>(C) + k0 * d;
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
        km_status s = simt_product<T, kProb>(Operand{X, N * d, d, 1}, Operand{Ck, K * d, d, 1}, B, N, kn, d, p, 1, st);
        if (s != KM_OK) return s;
        if (dX) {
            Epi q = {};
            q.wmax = wmax;
            q.acc = k0 ? w.dxacc : nullptr;
            if (k0 + kc < K) q.out32 = w.dxacc;
            else q.outT = dX;
            s = out_product<T>(Operand{w.P, N * kc, kc, 1}, Operand{Ck, K * d, 1, d}, B, N, d, kn, q, w.parts, st);
            if (s != KM_OK) return s;
        }
        if (dC) {
            // the pieces of dC are K * d apart between batches: one product per batch unless the
            // piece is the whole table
            Epi q = {};
            q.wmax = wmax;
            const int64_t nb = kn == K ? B : 1;
            for (int64_t b = 0; b < B; b += nb) {
                q.outT = static_cast<T *>(dC) + (b * K + k0) * d;
                s = out_product<T>(Operand{static_cast<const T *>(w.P) + b * N * kc, N * kc, 1, kc},
                                   Operand{static_cast<const T *>(w.X) + b * N * d, N * d, 1, d}, nb, kn, d, N, q,
                                   w.parts, st);
                if (s != KM_OK) return s;
            }
        }
    }
    return KM_OK;
}

}  // namespace

extern "C" {

size_t km_xent_workspace_size(int64_t B, int64_t N, int64_t K, int64_t d, km_dtype dtype) {
    if (!valid_dtype(dtype) || !xent_sizes_ok(B, N, K, d)) return 0;
    Carver c(nullptr);
    carve_loss(c, B, N, K);
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
    const LossWs w = carve_loss(c, B, N, K);
    switch (dtype) {
        case KM_F32: return loss_typed<float>(X, C, ids, B, N, K, d, scale, loss, lse, w, S(stream));
        case KM_F16: return loss_typed<__half>(X, C, ids, B, N, K, d, scale, loss, lse, w, S(stream));
        default: return loss_typed<__nv_bfloat16>(X, C, ids, B, N, K, d, scale, loss, lse, w, S(stream));
    }
}

size_t km_xent_grad_workspace_size(int64_t B, int64_t N, int64_t K, int64_t d, km_dtype dtype) {
    if (!valid_dtype(dtype) || !xent_sizes_ok(B, N, K, d)) return 0;
    Carver c(nullptr);
    carve_grad(c, B, N, K, d, dtype);
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
