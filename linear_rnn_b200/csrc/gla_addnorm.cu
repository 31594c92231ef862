// Residual sum and the norm before a block, over rows of D channels:
//   r = res + alpha rscale x,  y = norm(r) w
// and its gradient at the stored r:
//   dres = dr + d norm(r) (dy w),  dx = alpha rscale dres,  dw = sum dy n,  drscale = sum alpha x dres.
// gla_norm_common.cuh describes the layout and the row sums.
#include "gla_norm_common.cuh"

namespace gla {
namespace {

using namespace norm;

// Blocks of 256 threads per SM that the registers leave room for, 16384 x 4096: 4 with an fp32 residual (2: 139 us,
// 3: 143, 4: 135), 2 with everything in bf16 (2: 100 us, 3: 104, 4: 105).
template <typename T, typename R, int VEC, int NV, int S, int KIND, int MAXT, bool ODD>
__global__ void __launch_bounds__(MAXT, ODD || (MAXT == 256 && VEC == 8) ? (MAXT == 256 ? 2 : 1) : 1024 / MAXT)
    k_addnorm_fwd(const T* __restrict__ x, const R* res, const float* __restrict__ rscale,
                  const float* __restrict__ w, R* r_out, T* __restrict__ y, int rows, int D, int G, float alpha,
                  float eps) {
    extern __shared__ __align__(128) uint8_t smem[];
    constexpr int NP = kPairs<VEC>;
    using F = std::conditional_t<ODD, RowFeed<S>, Feed<S>>;
    constexpr int XOFF = F::template bytes<R, VEC, NV>();   // res first, then x
    constexpr int ROW = XOFF + F::template bytes<T, VEC, NV>();
    RowSum sum{reinterpret_cast<float*>(smem), G, 0};
    F feed = make_feed<S, ODD>(smem + kHead, ROW, G);
    const int grp = threadIdx.x / G, ngrp = blockDim.x / G;
    const Place P{(int)threadIdx.x - grp * G, G, ODD ? (D + 1) / 2 : D / VEC, D};
    const float inv_d = 1.f / D;
    uint64_t wv[NV][NP], sv[NV][NP];   // this thread's columns of w and alpha rscale
    load_columns<VEC, NV, ODD>(wv, w, P, 1.f);
    load_columns<VEC, NV, ODD>(sv, rscale, P, alpha);
    const long long step = (long long)gridDim.x * ngrp;
    long long row = (long long)blockIdx.x * ngrp + grp;
    auto copy = [&](long long to, int stage) {
        if constexpr (S > 0) {
            if constexpr (ODD) {
                if (to < rows) {
                    const size_t e0 = (size_t)to * D, n = (size_t)rows * D;
                    if (res) feed.copy_row(stage, 0, res, e0, n, P);
                    feed.copy_row(stage, XOFF, x, e0, n, P);
                }
            } else if (to < rows) {
#pragma unroll
                for (int j = 0; j < NV; ++j)
                    if (P.has(j)) {
                        const size_t c = (size_t)to * D + P.col<VEC>(j);
                        if (res) feed.template copy<R, VEC>(stage, 0, j, res + c);
                        feed.template copy<T, VEC>(stage, XOFF, j, x + c);
                    }
            }
            feed.commit();
        }
    };
#pragma unroll
    for (int k = 0; k + 1 < S; ++k) copy(row + k * step, k);
    // every group of a block takes as many turns: the row sums are the block's business
    for (long long first = (long long)blockIdx.x * ngrp; first < rows; first += step, row += step) {
        const bool live = row < rows;
        const size_t off = (size_t)row * D;
        if (S > 0) {
            feed.wait();
            copy(row + (S - 1) * step, feed.ahead());
        }
        uint64_t r[NV][NP];
#pragma unroll
        for (int j = 0; j < NV; ++j) {
#pragma unroll
            for (int i = 0; i < NP; ++i) r[j][i] = 0;
            if (live && P.has(j)) {
                uint64_t xv[NP];
                if constexpr (S > 0) {
                    feed.template read<T, VEC>(XOFF, j, xv, off, P);
                    if (res) feed.template read<R, VEC>(0, j, r[j], off, P);
                } else {
                    load_piece<VEC>(x + off + P.col<VEC>(j), xv);
                    if (res) load_piece<VEC>(res + off + P.col<VEC>(j), r[j]);
                }
#pragma unroll
                for (int i = 0; i < NP; ++i) r[j][i] = f2_fma(sv[j][i], xv[i], r[j][i]);
                if (r_out) put_piece<VEC, ODD>(r_out + off, P, j, r[j]);
            }
        }
        center<KIND, VEC, NV, ODD>(sum, r, P, inv_d);
        float s[1] = {square_sum<VEC, NV>(r)};
        sum(s);
        const uint64_t rstd = f2_all(rsqrtf(fmaf(s[0], inv_d, eps)));
#pragma unroll
        for (int j = 0; j < NV; ++j)
            if (live && P.has(j)) {
#pragma unroll
                for (int i = 0; i < NP; ++i) r[j][i] = f2_mul(f2_mul(r[j][i], rstd), wv[j][i]);
                put_piece<VEC, ODD>(y + off, P, j, r[j]);
            }
        feed.next();
    }
}

// The kernels of blocks of up to 256 threads, which the bound in their launch bounds tunes: 448 and 512 threads both
// leave a thread 128 registers (14 warps too are four to one of the schedulers), spent in another order. us at 512 and
// at 448, 16384 rows: all in bf16, RMS x 768 38 / 43, x 2048 73 / 85, x 4096 136 / 158, layer x 768 44 / 44, x 2048
// 80 / 79, x 4096 151 / 148; fp32 x 2048 RMS 132 / 143, layer 149 / 140; fp32 residual, layer x 3000 187 / 210 (60
// bytes of spills); pairs, RMS x 2002 121 / 115.
template <typename T, int VEC, int KIND>
constexpr int bwd_bound = VEC >= 4 && (KIND == GLA_NORM_RMS || (VEC == 4 && sizeof(T) == 2)) ? 512 : 448;
template <typename T, typename R, int VEC, int NV, int S, int KIND, int MAXT, bool ODD>
__global__ void __launch_bounds__(MAXT >= 512 ? MAXT : bwd_bound<T, VEC, KIND>)
    k_addnorm_bwd(const T* __restrict__ x, const R* __restrict__ r_in, const float* __restrict__ rscale,
                  const float* __restrict__ w, const T* __restrict__ dy, const R* dr, R* dres, T* __restrict__ dx,
                  float* __restrict__ pdw, float* __restrict__ pds, int rows, int D, int G, float alpha, float eps) {
    extern __shared__ __align__(128) uint8_t smem[];
    constexpr int NP = kPairs<VEC>;
    using F = std::conditional_t<ODD, RowFeed<S>, Feed<S>>;
    constexpr int BR = F::template bytes<R, VEC, NV>(), BT = F::template bytes<T, VEC, NV>();
    constexpr int DROFF = BR, DYOFF = 2 * BR, XOFF = 2 * BR + BT, ROW = 2 * (BR + BT);   // r, dr, dy, x
    RowSum sum{reinterpret_cast<float*>(smem), G, 0};
    F feed = make_feed<S, ODD>(smem + kHead, ROW, G);
    const int grp = threadIdx.x / G, ngrp = blockDim.x / G;
    const Place P{(int)threadIdx.x - grp * G, G, ODD ? (D + 1) / 2 : D / VEC, D};
    const float inv_d = 1.f / D;
    uint64_t wv[NV][NP], sv[NV][NP], aw[NV][NP] = {}, as[NV][NP] = {};
    load_columns<VEC, NV, ODD>(wv, w, P, 1.f);
    load_columns<VEC, NV, ODD>(sv, rscale, P, alpha);
    const long long step = (long long)gridDim.x * ngrp;
    long long row = (long long)blockIdx.x * ngrp + grp;
    auto copy = [&](long long to, int stage) {
        if constexpr (S > 0) {
            if constexpr (ODD) {
                if (to < rows) {
                    const size_t e0 = (size_t)to * D, n = (size_t)rows * D;
                    feed.copy_row(stage, 0, r_in, e0, n, P);
                    feed.copy_row(stage, DYOFF, dy, e0, n, P);
                    if (dr) feed.copy_row(stage, DROFF, dr, e0, n, P);
                    if (pds) feed.copy_row(stage, XOFF, x, e0, n, P);
                }
            } else if (to < rows) {
#pragma unroll
                for (int j = 0; j < NV; ++j)
                    if (P.has(j)) {
                        const size_t c = (size_t)to * D + P.col<VEC>(j);
                        feed.template copy<R, VEC>(stage, 0, j, r_in + c);
                        feed.template copy<T, VEC>(stage, DYOFF, j, dy + c);
                        if (dr) feed.template copy<R, VEC>(stage, DROFF, j, dr + c);
                        if (pds) feed.template copy<T, VEC>(stage, XOFF, j, x + c);
                    }
            }
            feed.commit();
        }
    };
#pragma unroll
    for (int k = 0; k + 1 < S; ++k) copy(row + k * step, k);
    for (long long first = (long long)blockIdx.x * ngrp; first < rows; first += step, row += step) {
        const bool live = row < rows;
        const size_t off = (size_t)row * D;
        if (S > 0) {
            feed.wait();
            copy(row + (S - 1) * step, feed.ahead());
        }
        uint64_t r[NV][NP], d[NV][NP];   // r - mu, then n; dy, then d = dy w
#pragma unroll
        for (int j = 0; j < NV; ++j) {
#pragma unroll
            for (int i = 0; i < NP; ++i) r[j][i] = d[j][i] = 0;
            if (live && P.has(j)) {
                if constexpr (S > 0) {
                    feed.template read<R, VEC>(0, j, r[j], off, P);
                    feed.template read<T, VEC>(DYOFF, j, d[j], off, P);
                } else {
                    load_piece<VEC>(r_in + off + P.col<VEC>(j), r[j]);
                    load_piece<VEC>(dy + off + P.col<VEC>(j), d[j]);
                }
            }
        }
        center<KIND, VEC, NV, ODD>(sum, r, P, inv_d);
        // sums of (r - mu)^2, d (r - mu) and, for the layer norm, d
        uint64_t t0 = 0, t1 = 0, t2 = 0;
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int i = 0; i < NP; ++i) {
                const uint64_t dw = f2_mul(d[j][i], wv[j][i]);
                t0 = f2_fma(r[j][i], r[j][i], t0);
                t1 = f2_fma(dw, r[j][i], t1);
                if (KIND == GLA_NORM_LAYER) t2 = f2_add(t2, dw);
            }
        float s[KIND == GLA_NORM_LAYER ? 3 : 2];
        s[0] = f2_sum(t0);
        s[1] = f2_sum(t1);
        if (KIND == GLA_NORM_LAYER) s[KIND == GLA_NORM_LAYER ? 2 : 0] = f2_sum(t2);
        sum(s);
        const float rstd = rsqrtf(fmaf(s[0], inv_d, eps));
        const uint64_t rstd2 = f2_all(rstd);
        // dres = dr + rstd d - (rstd mean(d n)) n - rstd mean(d)
        const uint64_t mdn = f2_all(-rstd * rstd * s[1] * inv_d);
        const uint64_t md = f2_all(KIND == GLA_NORM_LAYER ? -rstd * s[KIND == GLA_NORM_LAYER ? 2 : 0] * inv_d : 0.f);
#pragma unroll
        for (int j = 0; j < NV; ++j)
            if (live && P.has(j)) {
                uint64_t t[NP], xv[NP];
#pragma unroll
                for (int i = 0; i < NP; ++i) t[i] = 0;
                if (dr) {
                    if constexpr (S > 0) {
                        feed.template read<R, VEC>(DROFF, j, t, off, P);
                    } else {
                        load_piece<VEC>(dr + off + P.col<VEC>(j), t);
                    }
                }
#pragma unroll
                for (int i = 0; i < NP; ++i) {
                    const uint64_t n = f2_mul(r[j][i], rstd2);
                    aw[j][i] = f2_fma(d[j][i], n, aw[j][i]);
                    t[i] = f2_fma(n, mdn, t[i]);
                    if (KIND == GLA_NORM_LAYER) t[i] = f2_add(t[i], md);
                    t[i] = f2_fma(f2_mul(d[j][i], wv[j][i]), rstd2, t[i]);
                }
                if (dres) put_piece<VEC, ODD>(dres + off, P, j, t);
                if (pds) {
                    if constexpr (S > 0) {
                        feed.template read<T, VEC>(XOFF, j, xv, off, P);
                    } else {
                        load_piece<VEC>(x + off + P.col<VEC>(j), xv);
                    }
#pragma unroll
                    for (int i = 0; i < NP; ++i) as[j][i] = f2_fma(t[i], xv[i], as[j][i]);
                }
                if (dx) {
#pragma unroll
                    for (int i = 0; i < NP; ++i) t[i] = f2_mul(t[i], sv[j][i]);
                    put_piece<VEC, ODD>(dx + off, P, j, t);
                }
            }
        feed.next();
    }
    grid_dep_launch();
    float* cols = reinterpret_cast<float*>(smem);
    if (pdw) write_partial<VEC, NV, ODD>(aw, cols, grp, P, pdw + (size_t)blockIdx.x * D);
    if (pds) {
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int i = 0; i < NP; ++i) as[j][i] = f2_mul(as[j][i], f2_all(alpha));
        write_partial<VEC, NV, ODD>(as, cols, grp, P, pds + (size_t)blockIdx.x * D);
    }
}

template <typename F>
cudaError_t by_dtypes(gla_dtype io, gla_dtype res, F&& f) {
    if (io == GLA_F32) return f(float{}, float{});
    return res == GLA_F32 ? f(__nv_bfloat16{}, float{}) : f(__nv_bfloat16{}, __nv_bfloat16{});
}

RowPlan plan(const gla_norm_problem* p, bool bwd) {
    return row_plan(p->D, p->io == GLA_BF16 && p->res == GLA_BF16, p->io == GLA_F32, bwd);
}

gla_status check(const gla_norm_problem* p) {
    const gla_status s = check_common(p);
    if (s != GLA_OK) return s;
    if (p->H != 1) return GLA_ERR_INVALID_ARG;
    if (p->res != GLA_F32 && p->res != GLA_BF16) return GLA_ERR_INVALID_ARG;
    if (p->io == GLA_F32 && p->res != GLA_F32) return GLA_ERR_UNSUPPORTED;
    return GLA_OK;
}

}  // namespace
}  // namespace gla

using namespace gla;

extern "C" {

size_t gla_addnorm_workspace_bytes(const gla_norm_problem* p) {
    if (check(p) != GLA_OK) return 0;
    const int P = row_blocks(plan(p, true), (long long)p->B * p->L, 1);
    return P > 1 ? 256 + 2 * align_up((size_t)P * p->D * 4, 256) : 256;
}

gla_status gla_addnorm_fwd(const gla_norm_problem* p, const void* x, const void* res, const float* rscale,
                           const float* w, void* r, void* y, void* stream) {
    const gla_status s = check(p);
    if (s != GLA_OK) return s;
    const void* const ptrs[] = {x, res, rscale, w, r, y};
    if (!all_aligned(ptrs)) return GLA_ERR_INVALID_ARG;
    const int rows = p->B * p->L;
    if (rows == 0) return GLA_OK;
    if (!x || !y) return GLA_ERR_INVALID_ARG;
    cudaStream_t st = (cudaStream_t)stream;
    const RowPlan rp = plan(p, false);
    const cudaError_t e = by_dtypes(p->io, p->res, [&](auto tv, auto rv) {
        using T = decltype(tv);
        using R = decltype(rv);
        const int thread_bytes = rp.nv * rp.vec * (int)(sizeof(T) + sizeof(R));
        const int stages = ring_stages(rp, thread_bytes, p->kind);
        return by_shape<sizeof(T) + sizeof(R) == 4, sizeof(T) == 4, false>(rp, stages, [&](auto sh) {
            return by_kind(p->kind, [&](auto kind) {
                using Sh = decltype(sh);
                auto kern = k_addnorm_fwd<T, R, Sh::vec, Sh::nv, Sh::stages, decltype(kind)::value, Sh::maxt, Sh::odd>;
                const size_t smem = block_smem(rp, Sh::stages, thread_bytes);
                static std::atomic<bool> seen[kMaxDevices];
                static Occupancy known;
                const cudaError_t e = smem_attr_once(kern, kSmSmem, seen);
                if (e != cudaSuccess) return e;
                const int blocks = fit_blocks(kern, rp, smem, row_blocks(rp, rows, 1), 1, known);
                GLA_LAUNCH("addnorm_fwd", st,
                           (kern<<<blocks, rp.threads, smem, st>>>(
                               static_cast<const T*>(x), static_cast<const R*>(res), rscale, w, static_cast<R*>(r),
                               static_cast<T*>(y), rows, p->D, rp.G, p->alpha, p->eps)));
                return cudaGetLastError();
            });
        });
    });
    return record_cuda(e, "addnorm forward");
}

gla_status gla_addnorm_bwd(const gla_norm_problem* p, const void* x, const void* r, const float* rscale,
                           const float* w, const void* dy, const void* dr, void* dres, void* dx, float* dw,
                           float* drscale, void* ws, size_t ws_bytes, void* stream) {
    const gla_status s = check(p);
    if (s != GLA_OK) return s;
    const void* const ptrs[] = {x, r, rscale, w, dy, dr, dres, dx, dw, drscale, ws};
    const int rows = p->B * p->L;
    const RowPlan rp = plan(p, true);
    int P = row_blocks(rp, rows, 1);
    const bool direct = P == 1;   // a single block's sums are the result
    if (!all_aligned(ptrs) || (!ws && P > 1)) return GLA_ERR_INVALID_ARG;
    if (drscale && !rscale) return GLA_ERR_INVALID_ARG;
    if (P > 1 && ws_bytes < gla_addnorm_workspace_bytes(p)) return GLA_ERR_WORKSPACE;
    cudaStream_t st = (cudaStream_t)stream;
    float* pdw = !dw || direct ? dw : static_cast<float*>(ws);
    float* pds = !drscale || direct
                     ? drscale
                     : reinterpret_cast<float*>(static_cast<char*>(ws) + align_up((size_t)P * p->D * 4, 256));
    cudaError_t e = cudaSuccess;
    if (rows > 0) {
        if (!r || !dy || (drscale && !x)) return GLA_ERR_INVALID_ARG;
        e = by_dtypes(p->io, p->res, [&](auto tv, auto rv) {
            using T = decltype(tv);
            using R = decltype(rv);
            const int thread_bytes = 2 * rp.nv * rp.vec * (int)(sizeof(T) + sizeof(R));
            const int stages = ring_stages(rp, thread_bytes, p->kind);
            return by_shape<sizeof(T) + sizeof(R) == 4, sizeof(T) == 4, true>(rp, stages, [&](auto sh) {
                return by_kind(p->kind, [&](auto kind) {
                    using Sh = decltype(sh);
                    auto kern = k_addnorm_bwd<T, R, Sh::vec, Sh::nv, Sh::stages, decltype(kind)::value, Sh::maxt,
                                              Sh::odd>;
                    const size_t smem = block_smem(rp, Sh::stages, thread_bytes);
                    static std::atomic<bool> seen[kMaxDevices];
                    static Occupancy known;
                    const cudaError_t e = smem_attr_once(kern, kSmSmem, seen);
                    if (e != cudaSuccess) return e;
                    P = fit_blocks(kern, rp, smem, P, 1, known);
                    GLA_LAUNCH("addnorm_bwd", st,
                               (kern<<<P, rp.threads, smem, st>>>(
                                   static_cast<const T*>(x), static_cast<const R*>(r), rscale, w,
                                   static_cast<const T*>(dy), static_cast<const R*>(dr), static_cast<R*>(dres),
                                   static_cast<T*>(dx), pdw, pds, rows, p->D, rp.G, p->alpha, p->eps)));
                    return cudaGetLastError();
                });
            });
        });
    }
    if (e == cudaSuccess && !direct) e = colsum(pdw, dw, pds, drscale, P, p->D, p->D, st);
    return record_cuda(e, "addnorm backward");
}

}  // extern "C"
