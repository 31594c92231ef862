// The norms before and after a block, forward and backward, with what stands next to them fused in:
//   addnorm   r = res + alpha rscale x,  y = norm(r) w          (rows of D channels)
//   headnorm  y = norm(o) w act(z)                              (D channels of a head; [B,H,L,D] in,
//                                                                [B,L,H,D] out)
//   norm(r) = n = (r - mu) rstd,  rstd = 1 / sqrt(mean((r - mu)^2) + eps);  mu = 0 for the RMS norm.
// Gradient of a norm, d the gradient of n:  dr = rstd (d - n mean(d n) - [layer] mean(d)).
// Both are bound by HBM: a row is read once, kept in registers by the G threads that share it, and
// its sums are exchanged by shuffles (G <= 32) or through shared memory.
#include <type_traits>

#include "gla_common.cuh"
#include "gla_plans.h"

namespace gla {
namespace {

// ------------------------------------------------------------------ vectors of a row
template <int VEC>
__device__ __forceinline__ void load_vec(const float* p, float (&v)[VEC]) {
    if constexpr (VEC == 1) {
        v[0] = *p;
    } else {
#pragma unroll
        for (int i = 0; i < VEC; i += 4) {
            const float4 f = *reinterpret_cast<const float4*>(p + i);
            v[i] = f.x; v[i + 1] = f.y; v[i + 2] = f.z; v[i + 3] = f.w;
        }
    }
}
template <int VEC>
__device__ __forceinline__ void load_vec(const __nv_bfloat16* p, float (&v)[VEC]) {
    if constexpr (VEC == 1) {
        v[0] = __bfloat162float(*p);
    } else {
        uint32_t w[VEC / 2];
        if constexpr (VEC == 8) {
            const uint4 u = *reinterpret_cast<const uint4*>(p);
            w[0] = u.x; w[1] = u.y; w[2] = u.z; w[3] = u.w;
        } else {
            const uint2 u = *reinterpret_cast<const uint2*>(p);
            w[0] = u.x; w[1] = u.y;
        }
#pragma unroll
        for (int i = 0; i < VEC / 2; ++i) {
            v[2 * i] = __uint_as_float(w[i] << 16);
            v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
}
template <int VEC>
__device__ __forceinline__ void store_vec(float* p, const float (&v)[VEC]) {
    if constexpr (VEC == 1) {
        *p = v[0];
    } else {
#pragma unroll
        for (int i = 0; i < VEC; i += 4)
            *reinterpret_cast<float4*>(p + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
    }
}
template <int VEC>
__device__ __forceinline__ void store_vec(__nv_bfloat16* p, const float (&v)[VEC]) {
    if constexpr (VEC == 1) {
        *p = __float2bfloat16_rn(v[0]);
    } else {
        uint32_t w[VEC / 2];
#pragma unroll
        for (int i = 0; i < VEC / 2; ++i) {
            const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t*>(&b);
        }
        if constexpr (VEC == 8)
            *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
        else
            *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
    }
}

// ------------------------------------------------------------------ sums over a row
// Sums of K values over the G threads of a row (G a power of two; every thread of the block calls).
// G <= 32: shuffles. Otherwise the block is one row: one value per warp through `buf`, which
// alternates between two halves so that one barrier per call is enough.
struct RowSum {
    float* buf;   // [2][32 * 4]
    int G, half;
    template <int K>
    __device__ __forceinline__ void operator()(float (&v)[K]) {
        const int lim = min(G, 32);
        for (int off = lim >> 1; off; off >>= 1)
#pragma unroll
            for (int k = 0; k < K; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], off);
        if (G <= 32) return;
        float* b = buf + half * 128;
        half ^= 1;
        const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nw = G >> 5;
        if (lane == 0)
#pragma unroll
            for (int k = 0; k < K; ++k) b[k * 32 + warp] = v[k];
        __syncthreads();
#pragma unroll
        for (int k = 0; k < K; ++k) {
            v[k] = lane < nw ? b[k * 32 + lane] : 0.f;
#pragma unroll
            for (int off = 16; off; off >>= 1) v[k] += __shfl_xor_sync(0xffffffffu, v[k], off);
        }
    }
};

// mean (0 for the RMS norm) and 1 / root of the row r, elements beyond D zero and not counted
template <int KIND, int VEC, int NV>
__device__ __forceinline__ void row_stats(RowSum& sum, const float (&r)[NV][VEC], int at, int G, int nvec, float inv_d,
                                          float eps, float& mu, float& rstd) {
    mu = 0.f;
    if (KIND == GLA_NORM_LAYER) {
        float s[1] = {0.f};
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int i = 0; i < VEC; ++i) s[0] += r[j][i];
        sum(s);
        mu = s[0] * inv_d;
    }
    float s[1] = {0.f};
#pragma unroll
    for (int j = 0; j < NV; ++j)
        if (at + j * G < nvec)
#pragma unroll
            for (int i = 0; i < VEC; ++i) s[0] = fmaf(r[j][i] - mu, r[j][i] - mu, s[0]);
    sum(s);
    rstd = 1.f / sqrtf(fmaf(s[0], inv_d, eps));
}

template <int ACT>
__device__ __forceinline__ void act_grad(float z, float& f, float& df) {
    const float p = 1.f / (1.f + expf(-z));
    f = ACT == GLA_ACT_SILU ? z * p : p;
    df = ACT == GLA_ACT_SILU ? p * fmaf(z, 1.f - p, 1.f) : p * (1.f - p);
}

// Sums a column accumulator over the row groups of a block and writes the block's partial row.
// acc: this thread's [NV][VEC] columns; smem: blockDim * NV * VEC floats.
template <int VEC, int NV>
__device__ __forceinline__ void write_partial(const float (&acc)[NV][VEC], float* smem, int grp, int at, int G,
                                              int nvec, float* out) {
    const int D = nvec * VEC, ngrp = blockDim.x / G;
    if (ngrp == 1) {
#pragma unroll
        for (int j = 0; j < NV; ++j)
            if (at + j * G < nvec) store_vec<VEC>(out + (size_t)(at + j * G) * VEC, acc[j]);
        return;
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < NV; ++j)
        if (at + j * G < nvec)
#pragma unroll
            for (int i = 0; i < VEC; ++i) smem[grp * D + (at + j * G) * VEC + i] = acc[j][i];
    __syncthreads();
    for (int c = threadIdx.x; c < D; c += blockDim.x) {
        float s = 0.f;
        for (int k = 0; k < ngrp; ++k) s += smem[k * D + c];
        out[c] = s;
    }
}

// ------------------------------------------------------------------ addnorm
template <typename T, typename R, int VEC, int NV, int KIND>
__global__ void __launch_bounds__(1024) k_addnorm_fwd(const T* __restrict__ x, const R* res, const float* __restrict__ rscale,
                              const float* __restrict__ w, R* r_out, T* __restrict__ y, int rows, int D, int G,
                              float alpha, float eps) {
    __shared__ float buf[256];
    RowSum sum{buf, G, 0};
    const int grp = threadIdx.x / G, at = threadIdx.x & (G - 1), ngrp = blockDim.x / G, nvec = D / VEC;
    const float inv_d = 1.f / D;
    for (long long row0 = (long long)blockIdx.x * ngrp; row0 < rows; row0 += (long long)gridDim.x * ngrp) {
        const long long row = row0 + grp;
        const bool live = row < rows;
        const size_t off = (size_t)row * D;
        float r[NV][VEC];
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = (at + j * G) * VEC;
#pragma unroll
            for (int i = 0; i < VEC; ++i) r[j][i] = 0.f;
            if (live && at + j * G < nvec) {
                float xv[VEC], sv[VEC];
                load_vec<VEC>(x + off + c, xv);
                if (res) load_vec<VEC>(res + off + c, r[j]);
                if (rscale) load_vec<VEC>(rscale + c, sv);
#pragma unroll
                for (int i = 0; i < VEC; ++i) r[j][i] = fmaf(rscale ? alpha * sv[i] : alpha, xv[i], r[j][i]);
                if (r_out) store_vec<VEC>(r_out + off + c, r[j]);
            }
        }
        float mu, rstd;
        row_stats<KIND, VEC, NV>(sum, r, at, G, nvec, inv_d, eps, mu, rstd);
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = (at + j * G) * VEC;
            if (live && at + j * G < nvec) {
                float wv[VEC], yv[VEC];
                if (w) load_vec<VEC>(w + c, wv);
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    const float n = (r[j][i] - mu) * rstd;
                    yv[i] = w ? n * wv[i] : n;
                }
                store_vec<VEC>(y + off + c, yv);
            }
        }
    }
}

template <typename T, typename R, int VEC, int NV, int KIND>
__global__ void __launch_bounds__(1024) k_addnorm_bwd(const T* __restrict__ x, const R* __restrict__ r_in, const float* __restrict__ rscale,
                              const float* __restrict__ w, const T* __restrict__ dy, const R* dr, R* dres,
                              T* __restrict__ dx, float* __restrict__ pdw, float* __restrict__ pds, int rows, int D,
                              int G, float alpha, float eps) {
    extern __shared__ float smem[];
    float* buf = smem;
    RowSum sum{buf, G, 0};
    const int grp = threadIdx.x / G, at = threadIdx.x & (G - 1), ngrp = blockDim.x / G, nvec = D / VEC;
    const float inv_d = 1.f / D;
    float aw[NV][VEC] = {}, as[NV][VEC] = {};
    for (long long row0 = (long long)blockIdx.x * ngrp; row0 < rows; row0 += (long long)gridDim.x * ngrp) {
        const long long row = row0 + grp;
        const bool live = row < rows;
        const size_t off = (size_t)row * D;
        float r[NV][VEC], d[NV][VEC];
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = (at + j * G) * VEC;
#pragma unroll
            for (int i = 0; i < VEC; ++i) r[j][i] = d[j][i] = 0.f;
            if (live && at + j * G < nvec) {
                load_vec<VEC>(r_in + off + c, r[j]);
                load_vec<VEC>(dy + off + c, d[j]);
            }
        }
        float mu, rstd;
        row_stats<KIND, VEC, NV>(sum, r, at, G, nvec, inv_d, eps, mu, rstd);
        float s[2] = {0.f, 0.f};   // sums of d n and d, d = dy w
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = (at + j * G) * VEC;
            if (live && at + j * G < nvec) {
                float wv[VEC];
                if (w) load_vec<VEC>(w + c, wv);
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    r[j][i] = (r[j][i] - mu) * rstd;
                    aw[j][i] = fmaf(d[j][i], r[j][i], aw[j][i]);
                    if (w) d[j][i] *= wv[i];
                    s[0] = fmaf(d[j][i], r[j][i], s[0]);
                    s[1] += d[j][i];
                }
            }
        }
        sum(s);
        const float mdn = s[0] * inv_d, md = KIND == GLA_NORM_LAYER ? s[1] * inv_d : 0.f;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = (at + j * G) * VEC;
            if (live && at + j * G < nvec) {
                float t[VEC], sv[VEC], xv[VEC];
#pragma unroll
                for (int i = 0; i < VEC; ++i) t[i] = 0.f;
                if (dr) load_vec<VEC>(dr + off + c, t);
#pragma unroll
                for (int i = 0; i < VEC; ++i) t[i] = fmaf(rstd, d[j][i] - md - r[j][i] * mdn, t[i]);
                if (dres) store_vec<VEC>(dres + off + c, t);
                if (pds) {
                    load_vec<VEC>(x + off + c, xv);
#pragma unroll
                    for (int i = 0; i < VEC; ++i) as[j][i] = fmaf(alpha * t[i], xv[i], as[j][i]);
                }
                if (dx) {
                    if (rscale) load_vec<VEC>(rscale + c, sv);
#pragma unroll
                    for (int i = 0; i < VEC; ++i) t[i] *= rscale ? alpha * sv[i] : alpha;
                    store_vec<VEC>(dx + off + c, t);
                }
            }
        }
    }
    if (pdw) write_partial<VEC, NV>(aw, smem, grp, at, G, nvec, pdw + (size_t)blockIdx.x * D);
    if (pds) write_partial<VEC, NV>(as, smem, grp, at, G, nvec, pds + (size_t)blockIdx.x * D);
}

// ------------------------------------------------------------------ headnorm
// blockIdx.y = head; a row of the block = one token of that head.
template <typename T, int VEC, int NV, int KIND, int ACT>
__global__ void __launch_bounds__(1024) k_headnorm_fwd(const T* __restrict__ o, const T* __restrict__ z, const float* __restrict__ w,
                               T* __restrict__ y, int tokens, int H, int L, int D, int G, int w_stride, float eps) {
    __shared__ float buf[256];
    RowSum sum{buf, G, 0};
    const int grp = threadIdx.x / G, at = threadIdx.x & (G - 1), ngrp = blockDim.x / G, nvec = D / VEC;
    const int h = blockIdx.y;
    const float inv_d = 1.f / D;
    for (long long row0 = (long long)blockIdx.x * ngrp; row0 < tokens; row0 += (long long)gridDim.x * ngrp) {
        const long long row = row0 + grp;
        const bool live = row < tokens;
        const int b = live ? (int)row / L : 0, l = live ? (int)row - b * L : 0;
        const size_t src = (((size_t)b * H + h) * L + l) * D, dst = ((size_t)row * H + h) * D;
        float r[NV][VEC];
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = (at + j * G) * VEC;
#pragma unroll
            for (int i = 0; i < VEC; ++i) r[j][i] = 0.f;
            if (live && at + j * G < nvec) load_vec<VEC>(o + src + c, r[j]);
        }
        float mu, rstd;
        row_stats<KIND, VEC, NV>(sum, r, at, G, nvec, inv_d, eps, mu, rstd);
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = (at + j * G) * VEC;
            if (live && at + j * G < nvec) {
                float wv[VEC], zv[VEC];
                if (w) load_vec<VEC>(w + (size_t)h * w_stride + c, wv);
                if (z) load_vec<VEC>(z + dst + c, zv);
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    float n = (r[j][i] - mu) * rstd, f, df;
                    if (w) n *= wv[i];
                    if (z) {
                        act_grad<ACT>(zv[i], f, df);
                        n *= f;
                    }
                    r[j][i] = n;
                }
                store_vec<VEC>(y + dst + c, r[j]);
            }
        }
    }
}

template <typename T, int VEC, int NV, int KIND, int ACT>
__global__ void __launch_bounds__(1024) k_headnorm_bwd(const T* __restrict__ o, const T* __restrict__ z, const float* __restrict__ w,
                               const T* __restrict__ dy, T* __restrict__ d_o, T* __restrict__ dz,
                               float* __restrict__ pdw, int tokens, int H, int L, int D, int G, int w_stride,
                               float eps) {
    extern __shared__ float smem[];
    float* buf = smem;
    RowSum sum{buf, G, 0};
    const int grp = threadIdx.x / G, at = threadIdx.x & (G - 1), ngrp = blockDim.x / G, nvec = D / VEC;
    const int h = blockIdx.y;
    const float inv_d = 1.f / D;
    float aw[NV][VEC] = {};
    for (long long row0 = (long long)blockIdx.x * ngrp; row0 < tokens; row0 += (long long)gridDim.x * ngrp) {
        const long long row = row0 + grp;
        const bool live = row < tokens;
        const int b = live ? (int)row / L : 0, l = live ? (int)row - b * L : 0;
        const size_t src = (((size_t)b * H + h) * L + l) * D, dst = ((size_t)row * H + h) * D;
        float r[NV][VEC], d[NV][VEC];
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = (at + j * G) * VEC;
#pragma unroll
            for (int i = 0; i < VEC; ++i) r[j][i] = d[j][i] = 0.f;
            if (live && at + j * G < nvec) {
                load_vec<VEC>(o + src + c, r[j]);
                load_vec<VEC>(dy + dst + c, d[j]);
            }
        }
        float mu, rstd;
        row_stats<KIND, VEC, NV>(sum, r, at, G, nvec, inv_d, eps, mu, rstd);
        float s[2] = {0.f, 0.f};
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = (at + j * G) * VEC;
            if (live && at + j * G < nvec) {
                float wv[VEC], zv[VEC];
                if (w) load_vec<VEC>(w + (size_t)h * w_stride + c, wv);
                if (z) load_vec<VEC>(z + dst + c, zv);
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    const float n = (r[j][i] - mu) * rstd, wi = w ? wv[i] : 1.f;
                    if (z) {
                        float f, df;
                        act_grad<ACT>(zv[i], f, df);
                        zv[i] = d[j][i] * n * wi * df;
                        d[j][i] *= f;
                    }
                    aw[j][i] = fmaf(d[j][i], n, aw[j][i]);
                    d[j][i] *= wi;
                    s[0] = fmaf(d[j][i], n, s[0]);
                    s[1] += d[j][i];
                    r[j][i] = n;
                }
                if (dz) store_vec<VEC>(dz + dst + c, zv);
            }
        }
        sum(s);
        const float mdn = s[0] * inv_d, md = KIND == GLA_NORM_LAYER ? s[1] * inv_d : 0.f;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = (at + j * G) * VEC;
            if (live && at + j * G < nvec) {
#pragma unroll
                for (int i = 0; i < VEC; ++i) d[j][i] = rstd * (d[j][i] - md - r[j][i] * mdn);
                store_vec<VEC>(d_o + src + c, d[j]);
            }
        }
    }
    if (pdw) write_partial<VEC, NV>(aw, smem, grp, at, G, nvec, pdw + ((size_t)blockIdx.x * H + h) * D);
}

// ------------------------------------------------------------------ partial rows -> dw
// out[c] = sum over i < n of part[i * stride + c]: 32 columns per block, 32 rows at a time.
__global__ void __launch_bounds__(1024) k_colsum(const float* __restrict__ part, float* __restrict__ out, int n,
                                                 size_t stride, int cols) {
    __shared__ float red[32][33];
    const int c = blockIdx.x * 32 + threadIdx.x;
    float s = 0.f;
    if (c < cols)
        for (int i = threadIdx.y; i < n; i += 32) s += part[(size_t)i * stride + c];
    red[threadIdx.y][threadIdx.x] = s;
    __syncthreads();
    s = red[threadIdx.x][threadIdx.y];
#pragma unroll
    for (int off = 16; off; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
    const int cc = blockIdx.x * 32 + threadIdx.y;
    if (threadIdx.x == 0 && cc < cols) out[cc] = s;
}

// ------------------------------------------------------------------ host side
struct RowPlan {
    int vec, nv, G, threads, smem;
};
int pow2_at_least(int n) {
    int p = 1;
    while (p < n) p *= 2;
    return p;
}
// Threads per row: vectors of 16 bytes of the narrow dtype where D allows, one element otherwise.
RowPlan row_plan(int D, gla_dtype io) {
    const int wide = io == GLA_BF16 ? 8 : 4;
    RowPlan p;
    p.vec = D % wide == 0 ? wide : 1;
    const int nvec = D / p.vec;
    const int most = 16 / p.vec;   // elements per thread: at most 16
    p.nv = nvec <= 32 ? 1 : most;
    if (p.vec > 1 && cdiv(nvec, 1024) == 1 && nvec > 32) p.nv = 1;
    p.G = pow2_at_least(cdiv(nvec, p.nv));
    p.threads = p.G <= 32 ? 256 : p.G;
    p.smem = 4 * (p.G <= 32 ? 256 * p.nv * p.vec : 256);
    return p;
}
constexpr int kMaxPartials = 148 * 4;
int row_blocks(const RowPlan& p, long long rows, int most) {
    const long long need = (rows + p.threads / p.G - 1) / (p.threads / p.G);
    return (int)(need < most ? need : most);
}
int partial_blocks(const RowPlan& p, long long rows, int heads) {
    int most = kMaxPartials * 512 / (p.threads < 512 ? 512 : p.threads) / heads;
    return row_blocks(p, rows, most < 1 ? 1 : most);
}

template <int V, int N> struct Shape {
    static constexpr int vec = V, nv = N;
};
template <typename T, typename F>
cudaError_t by_shape(const RowPlan& p, F&& f) {
    constexpr int W = std::is_same<T, float>::value ? 4 : 8;
    if (p.vec == 1) return p.nv == 1 ? f(Shape<1, 1>{}) : f(Shape<1, 16>{});
    return p.nv == 1 ? f(Shape<W, 1>{}) : f(Shape<W, 16 / W>{});
}
template <typename F>
cudaError_t by_dtypes(gla_dtype io, gla_dtype res, F&& f) {
    if (io == GLA_F32) return f(float{}, float{});
    return res == GLA_F32 ? f(__nv_bfloat16{}, float{}) : f(__nv_bfloat16{}, __nv_bfloat16{});
}
template <typename F>
cudaError_t by_kind(int kind, F&& f) {
    return kind == GLA_NORM_RMS ? f(std::integral_constant<int, GLA_NORM_RMS>{})
                                : f(std::integral_constant<int, GLA_NORM_LAYER>{});
}
template <typename F>
cudaError_t by_act(int act, F&& f) {
    return act == GLA_ACT_SILU ? f(std::integral_constant<int, GLA_ACT_SILU>{})
                               : f(std::integral_constant<int, GLA_ACT_SIGMOID>{});
}

cudaError_t colsum(const float* part, float* out, int n, size_t stride, int cols, cudaStream_t st) {
    GLA_LAUNCH("norm_colsum", st,
               (k_colsum<<<cdiv(cols, 32), dim3(32, 32), 0, st>>>(part, out, n, stride, cols)));
    return cudaGetLastError();
}

bool aligned16(const void* x) { return x == nullptr || (reinterpret_cast<uintptr_t>(x) & 15u) == 0; }
template <int N>
bool all_aligned(const void* const (&ptrs)[N]) {
    for (const void* q : ptrs)
        if (!aligned16(q)) return false;
    return true;
}

gla_status check(const gla_norm_problem* p, bool head) {
    if (!p || p->B < 0 || p->H < 0 || p->L < 0 || p->D < 1) return GLA_ERR_INVALID_ARG;
    if (p->io != GLA_F32 && p->io != GLA_BF16) return GLA_ERR_INVALID_ARG;
    if (p->kind != GLA_NORM_RMS && p->kind != GLA_NORM_LAYER) return GLA_ERR_INVALID_ARG;
    if (!(p->eps > 0.f) || p->eps > 3.4e38f) return GLA_ERR_INVALID_ARG;
    if (head) {
        if (p->act != GLA_ACT_SILU && p->act != GLA_ACT_SIGMOID) return GLA_ERR_INVALID_ARG;
        if (p->w_per_head != 0 && p->w_per_head != 1) return GLA_ERR_INVALID_ARG;
        if (p->H > 65535) return GLA_ERR_UNSUPPORTED;
    } else {
        if (p->H != 1) return GLA_ERR_INVALID_ARG;
        if (p->res != GLA_F32 && p->res != GLA_BF16) return GLA_ERR_INVALID_ARG;
        if (p->io == GLA_F32 && p->res != GLA_F32) return GLA_ERR_UNSUPPORTED;
    }
    if (p->D > 16384 || (long long)p->B * p->L > 2147483647LL) return GLA_ERR_UNSUPPORTED;
    return GLA_OK;
}

}  // namespace
}  // namespace gla

using namespace gla;

extern "C" {

size_t gla_addnorm_workspace_bytes(const gla_norm_problem* p) {
    if (check(p, false) != GLA_OK) return 0;
    const int P = partial_blocks(row_plan(p->D, p->io), (long long)p->B * p->L, 1);
    return 256 + 2 * align_up((size_t)P * p->D * 4, 256);
}

gla_status gla_addnorm_fwd(const gla_norm_problem* p, const void* x, const void* res, const float* rscale,
                           const float* w, void* r, void* y, void* stream) {
    const gla_status s = check(p, false);
    if (s != GLA_OK) return s;
    const void* const ptrs[] = {x, res, rscale, w, r, y};
    if (!all_aligned(ptrs)) return GLA_ERR_INVALID_ARG;
    const int rows = p->B * p->L;
    if (rows == 0) return GLA_OK;
    if (!x || !y) return GLA_ERR_INVALID_ARG;
    cudaStream_t st = (cudaStream_t)stream;
    const RowPlan rp = row_plan(p->D, p->io);
    const int blocks = row_blocks(rp, rows, 2147483647);
    const cudaError_t e = by_dtypes(p->io, p->res, [&](auto tv, auto rv) {
        using T = decltype(tv);
        using R = decltype(rv);
        return by_shape<T>(rp, [&](auto sh) {
            return by_kind(p->kind, [&](auto kind) {
                GLA_LAUNCH("addnorm_fwd", st,
                           (k_addnorm_fwd<T, R, decltype(sh)::vec, decltype(sh)::nv, decltype(kind)::value>
                            <<<blocks, rp.threads, 0, st>>>(static_cast<const T*>(x), static_cast<const R*>(res),
                                                            rscale, w, static_cast<R*>(r), static_cast<T*>(y), rows,
                                                            p->D, rp.G, p->alpha, p->eps)));
                return cudaGetLastError();
            });
        });
    });
    return record_cuda(e, "addnorm forward");
}

gla_status gla_addnorm_bwd(const gla_norm_problem* p, const void* x, const void* r, const float* rscale,
                           const float* w, const void* dy, const void* dr, void* dres, void* dx, float* dw,
                           float* drscale, void* ws, size_t ws_bytes, void* stream) {
    const gla_status s = check(p, false);
    if (s != GLA_OK) return s;
    const void* const ptrs[] = {x, r, rscale, w, dy, dr, dres, dx, dw, drscale, ws};
    if (!all_aligned(ptrs) || !ws) return GLA_ERR_INVALID_ARG;
    if (drscale && !rscale) return GLA_ERR_INVALID_ARG;
    if (ws_bytes < gla_addnorm_workspace_bytes(p)) return GLA_ERR_WORKSPACE;
    cudaStream_t st = (cudaStream_t)stream;
    const int rows = p->B * p->L;
    const RowPlan rp = row_plan(p->D, p->io);
    const int P = partial_blocks(rp, rows, 1);
    float* pdw = dw ? static_cast<float*>(ws) : nullptr;
    float* pds = drscale ? reinterpret_cast<float*>(static_cast<char*>(ws) + align_up((size_t)P * p->D * 4, 256))
                         : nullptr;
    cudaError_t e = cudaSuccess;
    if (rows > 0) {
        if (!r || !dy || (drscale && !x)) return GLA_ERR_INVALID_ARG;
        e = by_dtypes(p->io, p->res, [&](auto tv, auto rv) {
            using T = decltype(tv);
            using R = decltype(rv);
            return by_shape<T>(rp, [&](auto sh) {
                return by_kind(p->kind, [&](auto kind) {
                    GLA_LAUNCH("addnorm_bwd", st,
                               (k_addnorm_bwd<T, R, decltype(sh)::vec, decltype(sh)::nv, decltype(kind)::value>
                                <<<P, rp.threads, rp.smem, st>>>(
                                    static_cast<const T*>(x), static_cast<const R*>(r), rscale, w,
                                    static_cast<const T*>(dy), static_cast<const R*>(dr), static_cast<R*>(dres),
                                    static_cast<T*>(dx), pdw, pds, rows, p->D, rp.G, p->alpha, p->eps)));
                    return cudaGetLastError();
                });
            });
        });
    }
    if (e == cudaSuccess && dw) e = colsum(pdw, dw, P, p->D, p->D, st);
    if (e == cudaSuccess && drscale) e = colsum(pds, drscale, P, p->D, p->D, st);
    return record_cuda(e, "addnorm backward");
}

size_t gla_headnorm_workspace_bytes(const gla_norm_problem* p) {
    if (check(p, true) != GLA_OK) return 0;
    const int P = p->H ? partial_blocks(row_plan(p->D, p->io), (long long)p->B * p->L, p->H) : 0;
    return 256 + (size_t)P * p->H * p->D * 4;
}

gla_status gla_headnorm_fwd(const gla_norm_problem* p, const void* o, const void* z, const float* w, void* y,
                            void* stream) {
    const gla_status s = check(p, true);
    if (s != GLA_OK) return s;
    const void* const ptrs[] = {o, z, w, y};
    if (!all_aligned(ptrs)) return GLA_ERR_INVALID_ARG;
    const int tokens = p->B * p->L;
    if (tokens == 0 || p->H == 0) return GLA_OK;
    if (!o || !y) return GLA_ERR_INVALID_ARG;
    cudaStream_t st = (cudaStream_t)stream;
    const RowPlan rp = row_plan(p->D, p->io);
    const dim3 grid(row_blocks(rp, tokens, 2147483647), p->H);
    const cudaError_t e = by_dtypes(p->io, GLA_F32, [&](auto tv, auto) {
        using T = decltype(tv);
        return by_shape<T>(rp, [&](auto sh) {
            return by_kind(p->kind, [&](auto kind) {
                return by_act(p->act, [&](auto act) {
                    GLA_LAUNCH("headnorm_fwd", st,
                               (k_headnorm_fwd<T, decltype(sh)::vec, decltype(sh)::nv, decltype(kind)::value,
                                               decltype(act)::value><<<grid, rp.threads, 0, st>>>(
                                   static_cast<const T*>(o), static_cast<const T*>(z), w, static_cast<T*>(y), tokens,
                                   p->H, p->L, p->D, rp.G, p->w_per_head ? p->D : 0, p->eps)));
                    return cudaGetLastError();
                });
            });
        });
    });
    return record_cuda(e, "headnorm forward");
}

gla_status gla_headnorm_bwd(const gla_norm_problem* p, const void* o, const void* z, const float* w, const void* dy,
                            void* d_o, void* dz, float* dw, void* ws, size_t ws_bytes, void* stream) {
    const gla_status s = check(p, true);
    if (s != GLA_OK) return s;
    const void* const ptrs[] = {o, z, w, dy, d_o, dz, dw, ws};
    if (!all_aligned(ptrs) || !ws || (dz && !z)) return GLA_ERR_INVALID_ARG;
    if (ws_bytes < gla_headnorm_workspace_bytes(p)) return GLA_ERR_WORKSPACE;
    cudaStream_t st = (cudaStream_t)stream;
    const int tokens = p->B * p->L;
    if (p->H == 0 && (!dw || p->w_per_head)) return GLA_OK;
    const RowPlan rp = row_plan(p->D, p->io);
    const int P = p->H ? partial_blocks(rp, tokens, p->H) : 0;
    float* pdw = dw ? static_cast<float*>(ws) : nullptr;
    cudaError_t e = cudaSuccess;
    if (tokens > 0 && p->H > 0) {
        if (!o || !dy || !d_o) return GLA_ERR_INVALID_ARG;
        const dim3 grid(P, p->H);
        e = by_dtypes(p->io, GLA_F32, [&](auto tv, auto) {
            using T = decltype(tv);
            return by_shape<T>(rp, [&](auto sh) {
                return by_kind(p->kind, [&](auto kind) {
                    return by_act(p->act, [&](auto act) {
                        GLA_LAUNCH("headnorm_bwd", st,
                                   (k_headnorm_bwd<T, decltype(sh)::vec, decltype(sh)::nv, decltype(kind)::value,
                                                   decltype(act)::value><<<grid, rp.threads, rp.smem, st>>>(
                                       static_cast<const T*>(o), static_cast<const T*>(z), w,
                                       static_cast<const T*>(dy), static_cast<T*>(d_o), static_cast<T*>(dz), pdw,
                                       tokens, p->H, p->L, p->D, rp.G, p->w_per_head ? p->D : 0, p->eps)));
                        return cudaGetLastError();
                    });
                });
            });
        });
    }
    if (e == cudaSuccess && dw)
        e = p->w_per_head ? colsum(pdw, dw, P, (size_t)p->H * p->D, p->H * p->D, st)
                          : colsum(pdw, dw, P * p->H, p->D, p->D, st);
    return record_cuda(e, "headnorm backward");
}

}  // extern "C"
