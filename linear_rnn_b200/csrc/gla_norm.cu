// The norms before and after a block, forward and backward, with what stands next to them fused in:
//   addnorm   r = res + alpha rscale x,  y = norm(r) w          (rows of D channels)
//   headnorm  y = norm(o) w act(z)                              (D channels of a head; [B,H,L,D] in,
//                                                                [B,L,H,D] out)
//   norm(r) = n = (r - mu) rstd,  rstd = 1 / sqrt(mean((r - mu)^2) + eps);  mu = 0 for the RMS norm.
// Gradient of a norm, d the gradient of n:  dr = rstd (d - n mean(d n) - [layer] mean(d)).
// Both are bound by HBM: a row is read once, kept in registers by the G threads that share it, and
// its sums are exchanged by shuffles (G <= 32: D up to 512, several rows per block) or through shared
// memory (one row per block). Blocks walk many rows. The next row's loads are in flight while a row is
// worked on: in registers where a warp holds a row, as bulk copies into a ring of rows in
// shared memory where a block does.
#include <type_traits>

#include "gla_common.cuh"
#include "gla_plans.h"
#include "sm100.cuh"

namespace gla {
namespace {

using namespace sm100;

// ------------------------------------------------------------------ vectors of a row
// VEC elements as they are in memory (16-byte pieces at most).
template <typename T, int VEC>
struct alignas(VEC * sizeof(T) > 16 ? 16 : VEC * sizeof(T)) Raw {
    T v[VEC];
};
template <typename T, int VEC>
__device__ __forceinline__ Raw<T, VEC> load_raw(const T* p) {
    return *reinterpret_cast<const Raw<T, VEC>*>(p);
}
template <int VEC>
__device__ __forceinline__ void unpack(const Raw<float, VEC>& r, float (&v)[VEC]) {
#pragma unroll
    for (int i = 0; i < VEC; ++i) v[i] = r.v[i];
}
template <int VEC>
__device__ __forceinline__ void unpack(const Raw<__nv_bfloat16, VEC>& r, float (&v)[VEC]) {
#pragma unroll
    for (int i = 0; i < VEC; ++i) v[i] = __bfloat162float(r.v[i]);
}
template <int VEC, typename T>
__device__ __forceinline__ void load_vec(const T* p, float (&v)[VEC]) {
    unpack(load_raw<T, VEC>(p), v);
}
template <int VEC, typename T>
__device__ __forceinline__ void store_vec(T* p, const float (&v)[VEC]) {
    Raw<T, VEC> r;
    if constexpr (std::is_same<T, float>::value || VEC == 1) {
#pragma unroll
        for (int i = 0; i < VEC; ++i) r.v[i] = from_f<T>(v[i]);
    } else {
#pragma unroll
        for (int i = 0; i < VEC; i += 2) {
            const __nv_bfloat162 b = __floats2bfloat162_rn(v[i], v[i + 1]);
            r.v[i] = b.x;
            r.v[i + 1] = b.y;
        }
    }
    *reinterpret_cast<Raw<T, VEC>*>(p) = r;
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
        for (int k = 0; k < K; ++k) v[k] = lane < nw ? b[k * 32 + lane] : 0.f;
        for (int off = nw >> 1; off; off >>= 1)
#pragma unroll
            for (int k = 0; k < K; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], off);
#pragma unroll
        for (int k = 0; k < K; ++k) v[k] = __shfl_sync(0xffffffffu, v[k], 0);
    }
};

// Where a thread's pieces of a row are.
struct Place {
    int at, G, nvec;
    __device__ __forceinline__ bool has(int j) const { return at + j * G < nvec; }
    __device__ __forceinline__ int piece(int j) const { return at + j * G; }
};

// mean (0 for the RMS norm) and 1 / root of the row r, elements beyond D zero and not counted
template <int KIND, int VEC, int NV>
__device__ __forceinline__ void row_stats(RowSum& sum, const float (&r)[NV][VEC], const Place& P, float inv_d,
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
        if (P.has(j))
#pragma unroll
            for (int i = 0; i < VEC; ++i) s[0] = fmaf(r[j][i] - mu, r[j][i] - mu, s[0]);
    sum(s);
    rstd = rsqrtf(fmaf(s[0], inv_d, eps));
}

// act(z) and its derivative. With bf16 data the exponential is the hardware's (its error grows with |z|,
// 2^-19 at |z| = 25, below a hundredth of the data's rounding); fp32 takes the exact one.
template <typename T, int ACT>
__device__ __forceinline__ void act_grad(float z, float& f, float& df) {
    const float e = std::is_same<T, float>::value ? expf(-z) : __expf(-z);
    const float p = __fdividef(1.f, 1.f + e);   // 0 where e overflows
    f = ACT == GLA_ACT_SILU ? z * p : p;
    df = ACT == GLA_ACT_SILU ? p * fmaf(z, 1.f - p, 1.f) : p * (1.f - p);
}

// Sums a column accumulator over the row groups of a block and writes the block's partial row.
// acc: this thread's [NV][VEC] columns; smem: blockDim * NV * VEC floats.
template <int VEC, int NV>
__device__ __forceinline__ void write_partial(const float (&acc)[NV][VEC], float* smem, int grp, const Place& P,
                                              float* out) {
    const int D = P.nvec * VEC, ngrp = blockDim.x / P.G;
    if (ngrp == 1) {
#pragma unroll
        for (int j = 0; j < NV; ++j)
            if (P.has(j)) store_vec<VEC>(out + (size_t)P.piece(j) * VEC, acc[j]);
        return;
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < NV; ++j)
        if (P.has(j))
#pragma unroll
            for (int i = 0; i < VEC; ++i) smem[grp * D + P.piece(j) * VEC + i] = acc[j][i];
    __syncthreads();
    for (int c = threadIdx.x; c < D; c += blockDim.x) {
        float s = 0.f;
        for (int k = 0; k < ngrp; ++k) s += smem[k * D + c];
        out[c] = s;
    }
}

// Whether the next row's loads wait in registers while a row is worked on: with more than 8 elements per
// thread they would spill.
template <int VEC, int NV, bool RING>
constexpr bool kAhead = !RING && VEC * NV <= 8;

// ------------------------------------------------------------------ a ring of rows
// For blocks that hold one row (G = blockDim): thread 0 copies the rows that follow, all inputs
// of a row into one stage. A stage is refilled once every thread is past the row in it, which the first
// barrier of the next row's sums shows.
constexpr int kRingStages = 4;
struct Ring {
    uint8_t* base;
    uint64_t* full;
    int stage_bytes, stages;
    bool ok;
    __device__ __forceinline__ uint8_t* wait(int k) {
        const int s = k % stages;
        if (ok) ok = mbar_wait(&full[s], (k / stages) & 1);   // a wait that gave up is the last one
        return base + (size_t)s * stage_bytes;
    }
};

// ------------------------------------------------------------------ addnorm
template <typename T, typename R, int VEC, int NV, int KIND, bool RING, int MAXT>
__global__ void __launch_bounds__(MAXT)
    k_addnorm_fwd(const T* __restrict__ x, const R* res, const float* __restrict__ rscale,
                  const float* __restrict__ w, R* r_out, T* __restrict__ y, int rows, int D, int G, float alpha,
                  float eps, int stages) {
    extern __shared__ __align__(128) uint8_t smem[];
    RowSum sum{reinterpret_cast<float*>(smem), G, 0};
    const int grp = threadIdx.x / G, ngrp = blockDim.x / G, nvec = D / VEC;
    const Place P{(int)threadIdx.x & (G - 1), G, nvec};
    const float inv_d = 1.f / D;
    float wv[NV][VEC], sv[NV][VEC];   // this thread's columns of w and alpha rscale
#pragma unroll
    for (int j = 0; j < NV; ++j) {
#pragma unroll
        for (int i = 0; i < VEC; ++i) wv[j][i] = 1.f, sv[j][i] = 1.f;
        if (P.has(j)) {
            if (w) load_vec<VEC>(w + P.piece(j) * VEC, wv[j]);
            if (rscale) load_vec<VEC>(rscale + P.piece(j) * VEC, sv[j]);
        }
#pragma unroll
        for (int i = 0; i < VEC; ++i) sv[j][i] *= alpha;
    }
    const long long step = (long long)gridDim.x * ngrp, first = (long long)blockIdx.x * ngrp;
    Ring ring{smem + 2048, reinterpret_cast<uint64_t*>(smem + 1024), D * (int)(sizeof(T) + sizeof(R)), stages, true};
    auto copy = [&](int k) {   // thread 0: row k of this block
        const long long row = first + k * step;
        if (row >= rows) return;
        uint64_t* bar = &ring.full[k % stages];
        uint8_t* to = ring.base + (size_t)(k % stages) * ring.stage_bytes;
        mbar_arrive_expect_tx(bar, D * (uint32_t)(sizeof(T) + (res ? sizeof(R) : 0)));
        if (res) bulk_load_1d(to, res + (size_t)row * D, D * (uint32_t)sizeof(R), bar);
        bulk_load_1d(to + D * sizeof(R), x + (size_t)row * D, D * (uint32_t)sizeof(T), bar);
    };
    if (RING) {
        if (threadIdx.x == 0) {
            for (int s = 0; s < stages; ++s) mbar_init(&ring.full[s], 1);
            mbar_fence_init();
            for (int k = 0; k + 1 < stages; ++k) copy(k);
        }
        __syncthreads();
    }
    Raw<T, VEC> xn[NV] = {};
    Raw<R, VEC> rn[NV] = {};
    auto fetch = [&](long long row) {   // the next row into registers
        if (row < rows)
#pragma unroll
            for (int j = 0; j < NV; ++j)
                if (P.has(j)) {
                    const size_t c = (size_t)row * D + P.piece(j) * VEC;
                    xn[j] = load_raw<T, VEC>(x + c);
                    if (res) rn[j] = load_raw<R, VEC>(res + c);
                }
    };
    constexpr bool AHEAD = kAhead<VEC, NV, RING>;
    if (AHEAD) fetch(first + grp);
    int k = 0;
    for (long long row0 = first; row0 < rows; row0 += step, ++k) {
        const long long row = row0 + grp;
        const bool live = row < rows;
        const size_t off = (size_t)row * D;
        float r[NV][VEC];
        if (!RING && !AHEAD) fetch(row);
        const uint8_t* st = RING ? ring.wait(k) : nullptr;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
#pragma unroll
            for (int i = 0; i < VEC; ++i) r[j][i] = 0.f;
            if (live && P.has(j)) {
                float xv[VEC];
                if (RING) {
                    load_vec<VEC>(reinterpret_cast<const T*>(st + D * sizeof(R)) + P.piece(j) * VEC, xv);
                    if (res) load_vec<VEC>(reinterpret_cast<const R*>(st) + P.piece(j) * VEC, r[j]);
                } else {
                    unpack(xn[j], xv);
                    if (res) unpack(rn[j], r[j]);
                }
#pragma unroll
                for (int i = 0; i < VEC; ++i) r[j][i] = fmaf(sv[j][i], xv[i], r[j][i]);
                if (r_out) store_vec<VEC>(r_out + off + P.piece(j) * VEC, r[j]);
            }
        }
        if (AHEAD) fetch(row + step);
        float mu, rstd;
        row_stats<KIND, VEC, NV>(sum, r, P, inv_d, eps, mu, rstd);
        if (RING && threadIdx.x == 0) copy(k + stages - 1);
#pragma unroll
        for (int j = 0; j < NV; ++j)
            if (live && P.has(j)) {
#pragma unroll
                for (int i = 0; i < VEC; ++i) r[j][i] = (r[j][i] - mu) * rstd * wv[j][i];
                store_vec<VEC>(y + off + P.piece(j) * VEC, r[j]);
            }
    }
}

template <typename T, typename R, int VEC, int NV, int KIND, bool RING, int MAXT>
__global__ void __launch_bounds__(MAXT)
    k_addnorm_bwd(const T* __restrict__ x, const R* __restrict__ r_in, const float* __restrict__ rscale,
                  const float* __restrict__ w, const T* __restrict__ dy, const R* dr, R* dres, T* __restrict__ dx,
                  float* __restrict__ pdw, float* __restrict__ pds, int rows, int D, int G, float alpha, float eps,
                  int stages) {
    extern __shared__ __align__(128) uint8_t smem[];
    RowSum sum{reinterpret_cast<float*>(smem), G, 0};
    const int grp = threadIdx.x / G, ngrp = blockDim.x / G, nvec = D / VEC;
    const Place P{(int)threadIdx.x & (G - 1), G, nvec};
    const float inv_d = 1.f / D;
    float wv[NV][VEC], sv[NV][VEC], aw[NV][VEC] = {}, as[NV][VEC] = {};
#pragma unroll
    for (int j = 0; j < NV; ++j) {
#pragma unroll
        for (int i = 0; i < VEC; ++i) wv[j][i] = 1.f, sv[j][i] = 1.f;
        if (P.has(j)) {
            if (w) load_vec<VEC>(w + P.piece(j) * VEC, wv[j]);
            if (rscale) load_vec<VEC>(rscale + P.piece(j) * VEC, sv[j]);
        }
#pragma unroll
        for (int i = 0; i < VEC; ++i) sv[j][i] *= alpha;
    }
    const long long step = (long long)gridDim.x * ngrp, first = (long long)blockIdx.x * ngrp;
    Ring ring{smem + 2048, reinterpret_cast<uint64_t*>(smem + 1024), 2 * D * (int)(sizeof(T) + sizeof(R)), stages,
              true};
    auto copy = [&](int k) {
        const long long row = first + k * step;
        if (row >= rows) return;
        const size_t off = (size_t)row * D;
        uint64_t* bar = &ring.full[k % stages];
        uint8_t* to = ring.base + (size_t)(k % stages) * ring.stage_bytes;
        const uint32_t br = D * (uint32_t)sizeof(R), bt = D * (uint32_t)sizeof(T);
        mbar_arrive_expect_tx(bar, br + bt + (dr ? br : 0) + (pds ? bt : 0));
        bulk_load_1d(to, r_in + off, br, bar);
        bulk_load_1d(to + 2 * br, dy + off, bt, bar);
        if (dr) bulk_load_1d(to + br, dr + off, br, bar);
        if (pds) bulk_load_1d(to + 2 * br + bt, x + off, bt, bar);
    };
    if (RING) {
        if (threadIdx.x == 0) {
            for (int s = 0; s < stages; ++s) mbar_init(&ring.full[s], 1);
            mbar_fence_init();
            for (int k = 0; k + 1 < stages; ++k) copy(k);
        }
        __syncthreads();
    }
    constexpr bool AHEAD = kAhead<VEC, NV, RING>;
    Raw<R, VEC> rn[NV] = {}, drn[NV] = {};
    Raw<T, VEC> dn[NV] = {}, xn[NV] = {};
    auto fetch = [&](long long row) {
        if (row < rows)
#pragma unroll
            for (int j = 0; j < NV; ++j)
                if (P.has(j)) {
                    const size_t c = (size_t)row * D + P.piece(j) * VEC;
                    rn[j] = load_raw<R, VEC>(r_in + c);
                    dn[j] = load_raw<T, VEC>(dy + c);
                    if (AHEAD && dr) drn[j] = load_raw<R, VEC>(dr + c);
                    if (AHEAD && pds) xn[j] = load_raw<T, VEC>(x + c);
                }
    };
    if (AHEAD) fetch(first + grp);
    int k = 0;
    for (long long row0 = first; row0 < rows; row0 += step, ++k) {
        const long long row = row0 + grp;
        const bool live = row < rows;
        const size_t off = (size_t)row * D;
        float r[NV][VEC], d[NV][VEC];
        if (!RING && !AHEAD) fetch(row);
        const uint8_t* st = RING ? ring.wait(k) : nullptr;
        Raw<R, VEC> drc[NV];
        Raw<T, VEC> xc[NV];
#pragma unroll
        for (int j = 0; j < NV; ++j) {
#pragma unroll
            for (int i = 0; i < VEC; ++i) r[j][i] = d[j][i] = 0.f;
            if (live && P.has(j)) {
                if (RING) {
                    load_vec<VEC>(reinterpret_cast<const R*>(st) + P.piece(j) * VEC, r[j]);
                    load_vec<VEC>(reinterpret_cast<const T*>(st + 2 * D * sizeof(R)) + P.piece(j) * VEC, d[j]);
                } else {
                    unpack(rn[j], r[j]);
                    unpack(dn[j], d[j]);
                }
            }
            if (AHEAD) drc[j] = drn[j], xc[j] = xn[j];
        }
        if (AHEAD) fetch(row + step);
        float mu, rstd;
        row_stats<KIND, VEC, NV>(sum, r, P, inv_d, eps, mu, rstd);
        if (RING && threadIdx.x == 0) copy(k + stages - 1);
        float s[2] = {0.f, 0.f};   // sums of d n and d, d = dy w
#pragma unroll
        for (int j = 0; j < NV; ++j)
            if (live && P.has(j))
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    r[j][i] = (r[j][i] - mu) * rstd;
                    aw[j][i] = fmaf(d[j][i], r[j][i], aw[j][i]);
                    d[j][i] *= wv[j][i];
                    s[0] = fmaf(d[j][i], r[j][i], s[0]);
                    s[1] += d[j][i];
                }
        sum(s);
        const float mdn = s[0] * inv_d, md = KIND == GLA_NORM_LAYER ? s[1] * inv_d : 0.f;
#pragma unroll
        for (int j = 0; j < NV; ++j)
            if (live && P.has(j)) {
                float t[VEC], xv[VEC];
#pragma unroll
                for (int i = 0; i < VEC; ++i) t[i] = 0.f;
                if (dr) {
                    if (RING) load_vec<VEC>(reinterpret_cast<const R*>(st + D * sizeof(R)) + P.piece(j) * VEC, t);
                    else if (AHEAD) unpack(drc[j], t);
                    else load_vec<VEC>(dr + off + P.piece(j) * VEC, t);
                }
#pragma unroll
                for (int i = 0; i < VEC; ++i) t[i] = fmaf(rstd, d[j][i] - md - r[j][i] * mdn, t[i]);
                if (dres) store_vec<VEC>(dres + off + P.piece(j) * VEC, t);
                if (pds) {
                    if (RING)
                        load_vec<VEC>(reinterpret_cast<const T*>(st + D * (2 * sizeof(R) + sizeof(T))) +
                                          P.piece(j) * VEC, xv);
                    else if (AHEAD) unpack(xc[j], xv);
                    else load_vec<VEC>(x + off + P.piece(j) * VEC, xv);
#pragma unroll
                    for (int i = 0; i < VEC; ++i) as[j][i] = fmaf(alpha * t[i], xv[i], as[j][i]);
                }
                if (dx) {
#pragma unroll
                    for (int i = 0; i < VEC; ++i) t[i] *= sv[j][i];
                    store_vec<VEC>(dx + off + P.piece(j) * VEC, t);
                }
            }
    }
    float* cols = reinterpret_cast<float*>(smem);
    if (pdw) write_partial<VEC, NV>(aw, cols, grp, P, pdw + (size_t)blockIdx.x * D);
    if (pds) write_partial<VEC, NV>(as, cols, grp, P, pds + (size_t)blockIdx.x * D);
}

// ------------------------------------------------------------------ headnorm
// blockIdx.y = head; a row of the block = one token of that head.
template <typename T, int VEC, int NV, int KIND, int ACT, int MAXT>
__global__ void __launch_bounds__(MAXT)
    k_headnorm_fwd(const T* __restrict__ o, const T* __restrict__ z, const float* __restrict__ w, T* __restrict__ y,
                   int tokens, int H, int L, int D, int G, int w_stride, float eps) {
    __shared__ float buf[256];
    RowSum sum{buf, G, 0};
    const int grp = threadIdx.x / G, ngrp = blockDim.x / G, nvec = D / VEC;
    const Place P{(int)threadIdx.x & (G - 1), G, nvec};
    const int h = blockIdx.y;
    const float inv_d = 1.f / D;
    float wv[NV][VEC];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
#pragma unroll
        for (int i = 0; i < VEC; ++i) wv[j][i] = 1.f;
        if (w && P.has(j)) load_vec<VEC>(w + (size_t)h * w_stride + P.piece(j) * VEC, wv[j]);
    }
    Raw<T, VEC> on[NV] = {}, zn[NV] = {};
    auto fetch = [&](long long row) {
        if (row >= tokens) return;
        const int b = (int)row / L, l = (int)row - b * L;
        const size_t src = (((size_t)b * H + h) * L + l) * D, dst = ((size_t)row * H + h) * D;
#pragma unroll
        for (int j = 0; j < NV; ++j)
            if (P.has(j)) {
                on[j] = load_raw<T, VEC>(o + src + P.piece(j) * VEC);
                if (z) zn[j] = load_raw<T, VEC>(z + dst + P.piece(j) * VEC);
            }
    };
    const long long step = (long long)gridDim.x * ngrp, first = (long long)blockIdx.x * ngrp;
    constexpr bool AHEAD = kAhead<VEC, NV, false>;
    if (AHEAD) fetch(first + grp);
    for (long long row0 = first; row0 < tokens; row0 += step) {
        const long long row = row0 + grp;
        const bool live = row < tokens;
        const size_t dst = ((size_t)row * H + h) * D;
        if (!AHEAD) fetch(row);
        float r[NV][VEC];
        Raw<T, VEC> zc[NV];
#pragma unroll
        for (int j = 0; j < NV; ++j) {
#pragma unroll
            for (int i = 0; i < VEC; ++i) r[j][i] = 0.f;
            if (live && P.has(j)) unpack(on[j], r[j]);
            zc[j] = zn[j];
        }
        if (AHEAD) fetch(row + step);
        float mu, rstd;
        row_stats<KIND, VEC, NV>(sum, r, P, inv_d, eps, mu, rstd);
#pragma unroll
        for (int j = 0; j < NV; ++j)
            if (live && P.has(j)) {
                float zv[VEC];
                unpack(zc[j], zv);
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    r[j][i] = (r[j][i] - mu) * rstd * wv[j][i];
                    if (z) {
                        float f, df;
                        act_grad<T, ACT>(zv[i], f, df);
                        r[j][i] *= f;
                    }
                }
                store_vec<VEC>(y + dst + P.piece(j) * VEC, r[j]);
            }
    }
}

template <typename T, int VEC, int NV, int KIND, int ACT, int MAXT>
__global__ void __launch_bounds__(MAXT)
    k_headnorm_bwd(const T* __restrict__ o, const T* __restrict__ z, const float* __restrict__ w,
                   const T* __restrict__ dy, T* __restrict__ d_o, T* __restrict__ dz, float* __restrict__ pdw,
                   int tokens, int H, int L, int D, int G, int w_stride, float eps) {
    extern __shared__ __align__(128) uint8_t smem[];
    RowSum sum{reinterpret_cast<float*>(smem), G, 0};
    const int grp = threadIdx.x / G, ngrp = blockDim.x / G, nvec = D / VEC;
    const Place P{(int)threadIdx.x & (G - 1), G, nvec};
    const int h = blockIdx.y;
    const float inv_d = 1.f / D;
    float wv[NV][VEC], aw[NV][VEC] = {};
#pragma unroll
    for (int j = 0; j < NV; ++j) {
#pragma unroll
        for (int i = 0; i < VEC; ++i) wv[j][i] = 1.f;
        if (w && P.has(j)) load_vec<VEC>(w + (size_t)h * w_stride + P.piece(j) * VEC, wv[j]);
    }
    Raw<T, VEC> on[NV] = {}, zn[NV] = {}, dn[NV] = {};
    auto source = [&](long long row) {
        const int b = (int)row / L, l = (int)row - b * L;
        return (((size_t)b * H + h) * L + l) * D;
    };
    auto fetch = [&](long long row) {
        if (row >= tokens) return;
        const size_t src = source(row), dst = ((size_t)row * H + h) * D;
#pragma unroll
        for (int j = 0; j < NV; ++j)
            if (P.has(j)) {
                on[j] = load_raw<T, VEC>(o + src + P.piece(j) * VEC);
                dn[j] = load_raw<T, VEC>(dy + dst + P.piece(j) * VEC);
                if (z) zn[j] = load_raw<T, VEC>(z + dst + P.piece(j) * VEC);
            }
    };
    const long long step = (long long)gridDim.x * ngrp, first = (long long)blockIdx.x * ngrp;
    constexpr bool AHEAD = kAhead<VEC, NV, false>;
    if (AHEAD) fetch(first + grp);
    for (long long row0 = first; row0 < tokens; row0 += step) {
        const long long row = row0 + grp;
        const bool live = row < tokens;
        const size_t dst = ((size_t)row * H + h) * D;
        if (!AHEAD) fetch(row);
        float r[NV][VEC], d[NV][VEC];
        Raw<T, VEC> zc[NV];
#pragma unroll
        for (int j = 0; j < NV; ++j) {
#pragma unroll
            for (int i = 0; i < VEC; ++i) r[j][i] = d[j][i] = 0.f;
            if (live && P.has(j)) {
                unpack(on[j], r[j]);
                unpack(dn[j], d[j]);
            }
            zc[j] = zn[j];
        }
        if (AHEAD) fetch(row + step);
        float mu, rstd;
        row_stats<KIND, VEC, NV>(sum, r, P, inv_d, eps, mu, rstd);
        float s[2] = {0.f, 0.f};
#pragma unroll
        for (int j = 0; j < NV; ++j)
            if (live && P.has(j)) {
                float zv[VEC];
                unpack(zc[j], zv);
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    const float n = (r[j][i] - mu) * rstd;
                    if (z) {
                        float f, df;
                        act_grad<T, ACT>(zv[i], f, df);
                        zv[i] = d[j][i] * n * wv[j][i] * df;
                        d[j][i] *= f;
                    }
                    aw[j][i] = fmaf(d[j][i], n, aw[j][i]);
                    d[j][i] *= wv[j][i];
                    s[0] = fmaf(d[j][i], n, s[0]);
                    s[1] += d[j][i];
                    r[j][i] = n;
                }
                if (dz) store_vec<VEC>(dz + dst + P.piece(j) * VEC, zv);
            }
        sum(s);
        const float mdn = s[0] * inv_d, md = KIND == GLA_NORM_LAYER ? s[1] * inv_d : 0.f;
        const size_t src = live ? source(row) : 0;
#pragma unroll
        for (int j = 0; j < NV; ++j)
            if (live && P.has(j)) {
#pragma unroll
                for (int i = 0; i < VEC; ++i) d[j][i] = rstd * (d[j][i] - md - r[j][i] * mdn);
                store_vec<VEC>(d_o + src + P.piece(j) * VEC, d[j]);
            }
    }
    if (pdw)
        write_partial<VEC, NV>(aw, reinterpret_cast<float*>(smem), grp, P, pdw + ((size_t)blockIdx.x * H + h) * D);
}

// ------------------------------------------------------------------ partial rows -> dw
// out[c] = sum over i < n of part[i * stride + c]: 32 columns per block, 32 rows at a time. blockIdx.y
// picks one of two sums.
__global__ void __launch_bounds__(1024) k_colsum(const float* __restrict__ part0, float* __restrict__ out0,
                                                 const float* __restrict__ part1, float* __restrict__ out1, int n,
                                                 size_t stride, int cols) {
    __shared__ float red[32][33];
    const float* part = blockIdx.y ? part1 : part0;
    float* out = blockIdx.y ? out1 : out0;
    const int c = blockIdx.x * 32 + threadIdx.x;
    float s = 0.f;
    if (c < cols)
#pragma unroll 8
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
    int vec, nv, G, threads;
    bool big;   // more than 512 threads
};
int pow2_at_least(int n) {
    int p = 1;
    while (p < n) p *= 2;
    return p;
}
// Threads and pieces of a row: pieces of 16 bytes of the narrow type where D allows, else 4 elements, else
// one; a warp or less up to D = 512, then as many threads as one piece each needs, up to 512, then 16
// elements each.
RowPlan row_plan(int D, gla_dtype io) {
    RowPlan p;
    p.vec = io == GLA_BF16 && D % 8 == 0 ? 8 : D % 4 == 0 ? 4 : 1;
    const int nvec = D / p.vec, most = 16 / p.vec;
    if (nvec <= 32) p.nv = 1;
    else if (D <= 512 || p.vec == 1) p.nv = most;
    else p.nv = nvec <= 512 ? 1 : most;
    p.G = pow2_at_least(cdiv(nvec, p.nv));
    p.threads = p.G <= 32 ? 256 : p.G;
    p.big = p.threads > 512;
    return p;
}
// Shared memory of the column sums over a block's row groups, and of the row sums.
int plain_smem(const RowPlan& p) { return p.G <= 32 ? 4 * 256 * p.nv * p.vec : 2048; }
// Blocks that walk the rows, and so partial rows of the column sums: no more than give every SM
// kThreadsPerSm threads. The launch takes fewer where fewer fit, so that no block waits for another.
constexpr int kThreadsPerSm = 1024;
int row_blocks(const RowPlan& p, long long rows, int heads) {
    const int per = p.threads / p.G;
    const long long need = (rows + per - 1) / per;
    long long most = (long long)tc::num_sms() * (kThreadsPerSm / p.threads) / heads;
    if (most < 1) most = 1;
    return (int)(need < most ? need : most);
}
template <typename K>
int fit_blocks(K kern, const RowPlan& p, size_t smem, int blocks, int heads) {
    if ((long long)blocks * heads <= tc::num_sms()) return blocks;
    int per_sm = 0;
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kern, p.threads, smem) != cudaSuccess || per_sm < 1) {
        cudaGetLastError();
        return blocks;
    }
    const int fit = tc::num_sms() * per_sm / heads;
    return fit < 1 ? 1 : fit < blocks ? fit : blocks;
}
// Stages of the ring of rows (0: no ring): up to kRingStages in a block's share of an SM's shared memory, at
// least two if the SM holds them.
constexpr int kRingHead = 2048;        // row sums and barriers in front of the ring
constexpr int kRingSm = 220 * 1024;
int ring_stages(const RowPlan& p, int row_bytes, long long rows_per_block) {
    if (p.G <= 32 || p.vec == 1 || row_bytes % 16 || rows_per_block < 2) return 0;
    int s = (kRingSm / (kThreadsPerSm / p.threads) - kRingHead - 1024) / row_bytes;
    if (s < 2 && 2 * row_bytes + kRingHead <= kRingSm) s = 2;
    s = s < kRingStages ? s : kRingStages;
    return s < 2 ? 0 : s;
}

template <int V, int N, int M> struct Shape {
    static constexpr int vec = V, nv = N, maxt = M;
};
template <typename T, typename F>
cudaError_t by_shape(const RowPlan& p, F&& f) {
    if (p.big) {
        if constexpr (!std::is_same<T, float>::value)
            if (p.vec == 8) return f(Shape<8, 2, 1024>{});
        return p.vec == 4 ? f(Shape<4, 4, 1024>{}) : f(Shape<1, 16, 1024>{});
    }
    if constexpr (!std::is_same<T, float>::value)
        if (p.vec == 8) return p.nv == 1 ? f(Shape<8, 1, 512>{}) : f(Shape<8, 2, 512>{});
    if (p.vec == 4) return p.nv == 1 ? f(Shape<4, 1, 512>{}) : f(Shape<4, 4, 512>{});
    return p.nv == 1 ? f(Shape<1, 1, 512>{}) : f(Shape<1, 16, 512>{});
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

// One or two column sums (out1 may be null).
cudaError_t colsum(const float* part0, float* out0, const float* part1, float* out1, int n, size_t stride, int cols,
                   cudaStream_t st) {
    if (!out0) {
        part0 = part1, out0 = out1;
        out1 = nullptr;
    }
    if (!out0) return cudaSuccess;
    GLA_LAUNCH("norm_colsum", st,
               (k_colsum<<<dim3(cdiv(cols, 32), out1 ? 2 : 1), dim3(32, 32), 0, st>>>(part0, out0, part1, out1, n,
                                                                                     stride, cols)));
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
    const int P = row_blocks(row_plan(p->D, p->io), (long long)p->B * p->L, 1);
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
    const int want = row_blocks(rp, rows, 1);
    const cudaError_t e = by_dtypes(p->io, p->res, [&](auto tv, auto rv) {
        using T = decltype(tv);
        using R = decltype(rv);
        const int row_bytes = p->D * (int)(sizeof(T) + sizeof(R));
        const int stages = ring_stages(rp, row_bytes, rows / want);
        return by_shape<T>(rp, [&](auto sh) {
            return by_kind(p->kind, [&](auto kind) {
                using S = decltype(sh);
                const size_t smem = stages ? kRingHead + (size_t)stages * row_bytes : 2048;
                auto launch = [&](auto kern) {
                    static std::atomic<bool> seen[kMaxDevices];
                    const cudaError_t e = smem_attr_once(kern, kRingSm, seen);
                    if (e != cudaSuccess) return e;
                    const int blocks = fit_blocks(kern, rp, smem, want, 1);
                    GLA_LAUNCH("addnorm_fwd", st,
                               (kern<<<blocks, rp.threads, smem, st>>>(
                                   static_cast<const T*>(x), static_cast<const R*>(res), rscale, w,
                                   static_cast<R*>(r), static_cast<T*>(y), rows, p->D, rp.G, p->alpha, p->eps,
                                   stages)));
                    return cudaGetLastError();
                };
                if constexpr (S::vec > 1)
                    if (stages)
                        return launch(k_addnorm_fwd<T, R, S::vec, S::nv, decltype(kind)::value, true, S::maxt>);
                return launch(k_addnorm_fwd<T, R, S::vec, S::nv, decltype(kind)::value, false, S::maxt>);
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
    const int want = row_blocks(rp, rows, 1);
    int P = want;
    float* pdw = dw ? static_cast<float*>(ws) : nullptr;
    float* pds = drscale ? reinterpret_cast<float*>(static_cast<char*>(ws) + align_up((size_t)P * p->D * 4, 256))
                         : nullptr;
    cudaError_t e = cudaSuccess;
    if (rows > 0) {
        if (!r || !dy || (drscale && !x)) return GLA_ERR_INVALID_ARG;
        e = by_dtypes(p->io, p->res, [&](auto tv, auto rv) {
            using T = decltype(tv);
            using R = decltype(rv);
            const int row_bytes = 2 * p->D * (int)(sizeof(T) + sizeof(R));
            const int stages = ring_stages(rp, row_bytes, rows / want);
            return by_shape<T>(rp, [&](auto sh) {
                return by_kind(p->kind, [&](auto kind) {
                    using S = decltype(sh);
                    const size_t smem = stages ? kRingHead + (size_t)stages * row_bytes : plain_smem(rp);
                    auto launch = [&](auto kern) {
                        static std::atomic<bool> seen[kMaxDevices];
                        const cudaError_t e = smem_attr_once(kern, kRingSm, seen);
                        if (e != cudaSuccess) return e;
                        P = fit_blocks(kern, rp, smem, want, 1);
                        GLA_LAUNCH("addnorm_bwd", st,
                                   (kern<<<P, rp.threads, smem, st>>>(
                                       static_cast<const T*>(x), static_cast<const R*>(r), rscale, w,
                                       static_cast<const T*>(dy), static_cast<const R*>(dr), static_cast<R*>(dres),
                                       static_cast<T*>(dx), pdw, pds, rows, p->D, rp.G, p->alpha, p->eps, stages)));
                        return cudaGetLastError();
                    };
                    if constexpr (S::vec > 1)
                        if (stages)
                            return launch(k_addnorm_bwd<T, R, S::vec, S::nv, decltype(kind)::value, true, S::maxt>);
                    return launch(k_addnorm_bwd<T, R, S::vec, S::nv, decltype(kind)::value, false, S::maxt>);
                });
            });
        });
    }
    if (e == cudaSuccess) e = colsum(pdw, dw, pds, drscale, P, p->D, p->D, st);
    return record_cuda(e, "addnorm backward");
}

size_t gla_headnorm_workspace_bytes(const gla_norm_problem* p) {
    if (check(p, true) != GLA_OK) return 0;
    const int P = p->H ? row_blocks(row_plan(p->D, p->io), (long long)p->B * p->L, p->H) : 0;
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
    const int want = row_blocks(rp, tokens, p->H);
    const cudaError_t e = by_dtypes(p->io, GLA_F32, [&](auto tv, auto) {
        using T = decltype(tv);
        return by_shape<T>(rp, [&](auto sh) {
            return by_kind(p->kind, [&](auto kind) {
                return by_act(p->act, [&](auto act) {
                    using S = decltype(sh);
                    auto kern = k_headnorm_fwd<T, S::vec, S::nv, decltype(kind)::value, decltype(act)::value, S::maxt>;
                    const dim3 grid(fit_blocks(kern, rp, 0, want, p->H), p->H);
                    GLA_LAUNCH("headnorm_fwd", st,
                               (kern<<<grid, rp.threads, 0, st>>>(static_cast<const T*>(o), static_cast<const T*>(z), w,
                                                              static_cast<T*>(y), tokens, p->H, p->L, p->D, rp.G,
                                                              p->w_per_head ? p->D : 0, p->eps)));
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
    int P = p->H ? row_blocks(rp, tokens, p->H) : 0;
    float* pdw = dw ? static_cast<float*>(ws) : nullptr;
    cudaError_t e = cudaSuccess;
    if (tokens > 0 && p->H > 0) {
        if (!o || !dy || !d_o) return GLA_ERR_INVALID_ARG;
        e = by_dtypes(p->io, GLA_F32, [&](auto tv, auto) {
            using T = decltype(tv);
            return by_shape<T>(rp, [&](auto sh) {
                return by_kind(p->kind, [&](auto kind) {
                    return by_act(p->act, [&](auto act) {
                        using S = decltype(sh);
                        auto kern =
                            k_headnorm_bwd<T, S::vec, S::nv, decltype(kind)::value, decltype(act)::value, S::maxt>;
                        P = fit_blocks(kern, rp, plain_smem(rp), P, p->H);
                        GLA_LAUNCH("headnorm_bwd", st,
                                   (kern<<<dim3(P, p->H), rp.threads, plain_smem(rp), st>>>(
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
        e = p->w_per_head ? colsum(pdw, dw, nullptr, nullptr, P, (size_t)p->H * p->D, p->H * p->D, st)
                          : colsum(pdw, dw, nullptr, nullptr, P * p->H, p->D, p->D, st);
    return record_cuda(e, "headnorm backward");
}

}  // extern "C"
