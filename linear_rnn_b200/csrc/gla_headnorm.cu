// Norm and gate after a cell, per head and token over the D channels of the head:
//   y = norm(o) w act(z),   o [B,H,L,D] as the cells write it, z and y [B,L,H,D].
// Gradient, with n = norm(o), d = dy act(z) w:  d_o = d norm(o) (d),  dz = dy n w act'(z),
// dw = sum dy act(z) n. gla_norm_common.cuh describes the layout and the row sums.
#include "gla_norm_common.cuh"

namespace gla {
namespace {

using namespace norm;

// act(z) and its derivative. With bf16 data the exponential is the hardware's (its relative error grows
// with |z|, 2^-19 at |z| = 25: under a hundredth of the data's rounding); fp32 takes the exact one.
template <typename T, int ACT>
__device__ __forceinline__ void act_grad(float z, float& f, float& df) {
    const float e = std::is_same<T, float>::value ? expf(-z) : __expf(-z);
    const float p = __fdividef(1.f, 1.f + e);   // 0 where e overflows
    f = ACT == GLA_ACT_SILU ? z * p : p;
    df = ACT == GLA_ACT_SILU ? p * fmaf(z, 1.f - p, 1.f) : p * (1.f - p);
}
template <typename T, int ACT>
__device__ __forceinline__ void act_grad2(uint64_t z, uint64_t& f, uint64_t& df) {
    float z0, z1, f0, f1, d0, d1;
    f2_split(z, z0, z1);
    act_grad<T, ACT>(z0, f0, d0);
    act_grad<T, ACT>(z1, f1, d1);
    f = f2(f0, f1);
    df = f2(d0, d1);
}

// The tokens of one head that a thread's group takes, `step` apart: batch and position advance without
// divisions.
struct Token {
    long long t;
    int b, l;
    __device__ __forceinline__ void go(long long step, int sb, int sl, int L) {
        t += step;
        b += sb;
        l += sl;
        if (l >= L) l -= L, ++b;
    }
};

// blockIdx.y = head; a row of the block = one token of that head.
template <typename T, int VEC, int NV, int S, int KIND, int ACT, int MAXT>
__global__ void __launch_bounds__(MAXT)
    k_headnorm_fwd(const T* __restrict__ o, const T* __restrict__ z, const float* __restrict__ w, T* __restrict__ y,
                   int tokens, int H, int L, int D, int G, int w_stride, float eps) {
    extern __shared__ __align__(128) uint8_t smem[];
    constexpr int NP = kPairs<VEC>;
    using F = Feed<S>;
    constexpr int ZOFF = F::template bytes<T, VEC, NV>(), ROW = 2 * ZOFF;
    RowSum sum{reinterpret_cast<float*>(smem), G, 0};
    F feed{smem + kHead + 16 * threadIdx.x, ROW * (int)blockDim.x, 0, 0};
    const int grp = threadIdx.x / G, ngrp = blockDim.x / G, h = blockIdx.y;
    const Place P{(int)threadIdx.x - grp * G, G, D / VEC};
    const float inv_d = 1.f / D;
    uint64_t wv[NV][NP];
    load_columns<VEC, NV>(wv, w ? w + (size_t)h * w_stride : nullptr, P, 1.f);
    const long long step = (long long)gridDim.x * ngrp;
    const int sb = (int)(step / L), sl = (int)(step % L);
    Token in;   // the next token to copy
    in.t = (long long)blockIdx.x * ngrp + grp;
    in.b = (int)(in.t / L);
    in.l = (int)(in.t % L);
    auto source = [&](const Token& k) { return o + (((size_t)k.b * H + h) * L + k.l) * D; };
    auto copy = [&](int stage) {
        if (S > 0) {
            if (in.t < tokens) {
                const T *os = source(in), *zs = z ? z + ((size_t)in.t * H + h) * D : nullptr;
#pragma unroll
                for (int j = 0; j < NV; ++j)
                    if (P.has(j)) {
                        feed.template copy<T, VEC>(stage, 0, j, os + P.col<VEC>(j));
                        if (z) feed.template copy<T, VEC>(stage, ZOFF, j, zs + P.col<VEC>(j));
                    }
            }
            feed.commit();
            in.go(step, sb, sl, L);
        }
    };
#pragma unroll
    for (int k = 0; k + 1 < S; ++k) copy(k);
    long long t = (long long)blockIdx.x * ngrp + grp;
    for (long long first = (long long)blockIdx.x * ngrp; first < tokens; first += step, t += step) {
        const bool live = t < tokens;
        const size_t dst = ((size_t)t * H + h) * D;
        if (S > 0) {
            feed.wait();
            copy(feed.ahead());
        }
        uint64_t r[NV][NP];
#pragma unroll
        for (int j = 0; j < NV; ++j) {
#pragma unroll
            for (int i = 0; i < NP; ++i) r[j][i] = 0;
            if (live && P.has(j)) {
                if constexpr (S > 0) feed.template read<T, VEC>(0, j, r[j]);
                else load_piece<VEC>(source(in) + P.col<VEC>(j), r[j]);
            }
        }
        center<KIND, VEC, NV>(sum, r, P, inv_d);
        float s[1] = {square_sum<VEC, NV>(r)};
        sum(s);
        const uint64_t rstd = f2_all(rsqrtf(fmaf(s[0], inv_d, eps)));
#pragma unroll
        for (int j = 0; j < NV; ++j)
            if (live && P.has(j)) {
#pragma unroll
                for (int i = 0; i < NP; ++i) r[j][i] = f2_mul(f2_mul(r[j][i], rstd), wv[j][i]);
                if (z) {
                    uint64_t zv[NP];
                    if constexpr (S > 0) feed.template read<T, VEC>(ZOFF, j, zv);
                    else load_piece<VEC>(z + dst + P.col<VEC>(j), zv);
#pragma unroll
                    for (int i = 0; i < NP; ++i) {
                        uint64_t f, df;
                        act_grad2<T, ACT>(zv[i], f, df);
                        r[j][i] = f2_mul(r[j][i], f);
                    }
                }
                store_piece<VEC>(y + dst + P.col<VEC>(j), r[j]);
            }
        feed.next();
        if (S == 0) in.go(step, sb, sl, L);
    }
}

template <typename T, int VEC, int NV, int S, int KIND, int ACT, int MAXT>
__global__ void __launch_bounds__(MAXT)
    k_headnorm_bwd(const T* __restrict__ o, const T* __restrict__ z, const float* __restrict__ w,
                   const T* __restrict__ dy, T* __restrict__ d_o, T* __restrict__ dz, float* __restrict__ pdw,
                   int tokens, int H, int L, int D, int G, int w_stride, float eps) {
    extern __shared__ __align__(128) uint8_t smem[];
    constexpr int NP = kPairs<VEC>;
    using F = Feed<S>;
    constexpr int ZOFF = F::template bytes<T, VEC, NV>(), YOFF = 2 * ZOFF, ROW = 3 * ZOFF;
    RowSum sum{reinterpret_cast<float*>(smem), G, 0};
    F feed{smem + kHead + 16 * threadIdx.x, ROW * (int)blockDim.x, 0, 0};
    const int grp = threadIdx.x / G, ngrp = blockDim.x / G, h = blockIdx.y;
    const Place P{(int)threadIdx.x - grp * G, G, D / VEC};
    const float inv_d = 1.f / D;
    uint64_t wv[NV][NP], aw[NV][NP] = {};
    load_columns<VEC, NV>(wv, w ? w + (size_t)h * w_stride : nullptr, P, 1.f);
    const long long step = (long long)gridDim.x * ngrp;
    const int sb = (int)(step / L), sl = (int)(step % L);
    Token in, out;   // the next token to copy, the current one
    in.t = (long long)blockIdx.x * ngrp + grp;
    in.b = (int)(in.t / L);
    in.l = (int)(in.t % L);
    out = in;
    auto place = [&](const Token& k) { return (((size_t)k.b * H + h) * L + k.l) * D; };
    auto copy = [&](int stage) {
        if (S > 0) {
            if (in.t < tokens) {
                const size_t src = place(in), dst = ((size_t)in.t * H + h) * D;
#pragma unroll
                for (int j = 0; j < NV; ++j)
                    if (P.has(j)) {
                        feed.template copy<T, VEC>(stage, 0, j, o + src + P.col<VEC>(j));
                        feed.template copy<T, VEC>(stage, YOFF, j, dy + dst + P.col<VEC>(j));
                        if (z) feed.template copy<T, VEC>(stage, ZOFF, j, z + dst + P.col<VEC>(j));
                    }
            }
            feed.commit();
            in.go(step, sb, sl, L);
        }
    };
#pragma unroll
    for (int k = 0; k + 1 < S; ++k) copy(k);
    for (long long first = (long long)blockIdx.x * ngrp; first < tokens; first += step) {
        const bool live = out.t < tokens;
        const size_t dst = ((size_t)out.t * H + h) * D, src = place(out);
        if (S > 0) {
            feed.wait();
            copy(feed.ahead());
        }
        uint64_t r[NV][NP], d[NV][NP], q[NV][NP];   // o - mu; dy act(z) w; dy act(z), dw's factor
#pragma unroll
        for (int j = 0; j < NV; ++j) {
#pragma unroll
            for (int i = 0; i < NP; ++i) r[j][i] = 0;
            if (live && P.has(j)) {
                if constexpr (S > 0) feed.template read<T, VEC>(0, j, r[j]);
                else load_piece<VEC>(o + src + P.col<VEC>(j), r[j]);
            }
        }
        center<KIND, VEC, NV>(sum, r, P, inv_d);
        uint64_t t0 = 0, t1 = 0, t2 = 0;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
#pragma unroll
            for (int i = 0; i < NP; ++i) q[j][i] = d[j][i] = 0;
            if (live && P.has(j)) {
                uint64_t zv[NP];
                if constexpr (S > 0) feed.template read<T, VEC>(YOFF, j, q[j]);
                else load_piece<VEC>(dy + dst + P.col<VEC>(j), q[j]);
                if (z) {
                    if constexpr (S > 0) feed.template read<T, VEC>(ZOFF, j, zv);
                    else load_piece<VEC>(z + dst + P.col<VEC>(j), zv);
#pragma unroll
                    for (int i = 0; i < NP; ++i) {
                        uint64_t f, df;
                        act_grad2<T, ACT>(zv[i], f, df);
                        d[j][i] = f2_mul(f2_mul(q[j][i], wv[j][i]), df);   // dz / n, kept until n is known
                        q[j][i] = f2_mul(q[j][i], f);
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < NP; ++i) {
                const uint64_t dn = f2_mul(q[j][i], wv[j][i]);
                t0 = f2_fma(r[j][i], r[j][i], t0);
                t1 = f2_fma(dn, r[j][i], t1);
                if (KIND == GLA_NORM_LAYER) t2 = f2_add(t2, dn);
            }
        }
        float s[KIND == GLA_NORM_LAYER ? 3 : 2];
        s[0] = f2_sum(t0);
        s[1] = f2_sum(t1);
        if (KIND == GLA_NORM_LAYER) s[KIND == GLA_NORM_LAYER ? 2 : 0] = f2_sum(t2);
        sum(s);
        const float rstd = rsqrtf(fmaf(s[0], inv_d, eps));
        const uint64_t rstd2 = f2_all(rstd);
        const uint64_t mdn = f2_all(-rstd * rstd * s[1] * inv_d);
        const uint64_t md = f2_all(KIND == GLA_NORM_LAYER ? -rstd * s[KIND == GLA_NORM_LAYER ? 2 : 0] * inv_d : 0.f);
#pragma unroll
        for (int j = 0; j < NV; ++j)
            if (live && P.has(j)) {
#pragma unroll
                for (int i = 0; i < NP; ++i) {
                    const uint64_t n = f2_mul(r[j][i], rstd2);
                    d[j][i] = f2_mul(d[j][i], n);
                    aw[j][i] = f2_fma(q[j][i], n, aw[j][i]);
                    r[j][i] = f2_fma(f2_mul(q[j][i], wv[j][i]), rstd2, f2_mul(n, mdn));
                    if (KIND == GLA_NORM_LAYER) r[j][i] = f2_add(r[j][i], md);
                }
                if (dz) store_piece<VEC>(dz + dst + P.col<VEC>(j), d[j]);
                store_piece<VEC>(d_o + src + P.col<VEC>(j), r[j]);
            }
        feed.next();
        out.go(step, sb, sl, L);
    }
    grid_dep_launch();
    if (pdw)
        write_partial<VEC, NV>(aw, reinterpret_cast<float*>(smem), grp, P, pdw + ((size_t)blockIdx.x * H + h) * D);
}

template <typename F>
cudaError_t by_io(gla_dtype io, F&& f) {
    return io == GLA_F32 ? f(float{}) : f(__nv_bfloat16{});
}
template <typename F>
cudaError_t by_act(int act, F&& f) {
    return act == GLA_ACT_SILU ? f(std::integral_constant<int, GLA_ACT_SILU>{})
                               : f(std::integral_constant<int, GLA_ACT_SIGMOID>{});
}

gla_status check(const gla_norm_problem* p) {
    const gla_status s = check_common(p);
    if (s != GLA_OK) return s;
    if (p->act != GLA_ACT_SILU && p->act != GLA_ACT_SIGMOID) return GLA_ERR_INVALID_ARG;
    if (p->w_per_head != 0 && p->w_per_head != 1) return GLA_ERR_INVALID_ARG;
    return p->H > 65535 ? GLA_ERR_UNSUPPORTED : GLA_OK;
}

}  // namespace
}  // namespace gla

using namespace gla;

extern "C" {

size_t gla_headnorm_workspace_bytes(const gla_norm_problem* p) {
    if (check(p) != GLA_OK) return 0;
    const int P = p->H ? row_blocks(row_plan(p->D, p->io == GLA_BF16), (long long)p->B * p->L, p->H) : 0;
    return 256 + (size_t)P * p->H * p->D * 4;
}

gla_status gla_headnorm_fwd(const gla_norm_problem* p, const void* o, const void* z, const float* w, void* y,
                            void* stream) {
    const gla_status s = check(p);
    if (s != GLA_OK) return s;
    const void* const ptrs[] = {o, z, w, y};
    if (!all_aligned(ptrs)) return GLA_ERR_INVALID_ARG;
    const int tokens = p->B * p->L;
    if (tokens == 0 || p->H == 0) return GLA_OK;
    if (!o || !y) return GLA_ERR_INVALID_ARG;
    cudaStream_t st = (cudaStream_t)stream;
    const RowPlan rp = row_plan(p->D, p->io == GLA_BF16);
    const cudaError_t e = by_io(p->io, [&](auto tv) {
        using T = decltype(tv);
        const int thread_bytes = 2 * rp.nv * rp.vec * (int)sizeof(T);
        return by_shape<std::is_same<T, __nv_bfloat16>::value>(rp, ring_stages(rp, thread_bytes), [&](auto sh) {
            return by_kind(p->kind, [&](auto kind) {
                return by_act(p->act, [&](auto act) {
                    using Sh = decltype(sh);
                    auto kern = k_headnorm_fwd<T, Sh::vec, Sh::nv, Sh::stages, decltype(kind)::value,
                                               decltype(act)::value, Sh::maxt>;
                    const size_t smem = block_smem(rp, Sh::stages, thread_bytes);
                    static std::atomic<bool> seen[kMaxDevices];
                    const cudaError_t e = smem_attr_once(kern, kSmSmem, seen);
                    if (e != cudaSuccess) return e;
                    const dim3 grid(fit_blocks(kern, rp, smem, row_blocks(rp, tokens, p->H), p->H), p->H);
                    GLA_LAUNCH("headnorm_fwd", st,
                               (kern<<<grid, rp.threads, smem, st>>>(
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
    const gla_status s = check(p);
    if (s != GLA_OK) return s;
    const void* const ptrs[] = {o, z, w, dy, d_o, dz, dw, ws};
    if (!all_aligned(ptrs) || !ws || (dz && !z)) return GLA_ERR_INVALID_ARG;
    if (ws_bytes < gla_headnorm_workspace_bytes(p)) return GLA_ERR_WORKSPACE;
    cudaStream_t st = (cudaStream_t)stream;
    const int tokens = p->B * p->L;
    if (p->H == 0 && (!dw || p->w_per_head)) return GLA_OK;
    const RowPlan rp = row_plan(p->D, p->io == GLA_BF16);
    int P = p->H ? row_blocks(rp, tokens, p->H) : 0;
    float* pdw = dw ? static_cast<float*>(ws) : nullptr;
    cudaError_t e = cudaSuccess;
    if (tokens > 0 && p->H > 0) {
        if (!o || !dy || !d_o) return GLA_ERR_INVALID_ARG;
        e = by_io(p->io, [&](auto tv) {
            using T = decltype(tv);
            const int thread_bytes = 3 * rp.nv * rp.vec * (int)sizeof(T);
            return by_shape<std::is_same<T, __nv_bfloat16>::value>(rp, ring_stages(rp, thread_bytes), [&](auto sh) {
                return by_kind(p->kind, [&](auto kind) {
                    return by_act(p->act, [&](auto act) {
                        using Sh = decltype(sh);
                        auto kern = k_headnorm_bwd<T, Sh::vec, Sh::nv, Sh::stages, decltype(kind)::value,
                                                   decltype(act)::value, Sh::maxt>;
                        const size_t smem = block_smem(rp, Sh::stages, thread_bytes);
                        static std::atomic<bool> seen[kMaxDevices];
                        const cudaError_t e = smem_attr_once(kern, kSmSmem, seen);
                        if (e != cudaSuccess) return e;
                        P = fit_blocks(kern, rp, smem, P, p->H);
                        GLA_LAUNCH("headnorm_bwd", st,
                                   (kern<<<dim3(P, p->H), rp.threads, smem, st>>>(
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
