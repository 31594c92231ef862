// Norm and gate after a cell, per head and token over the D channels of the head:
//   y = norm(o) w act(z),   o [B,H,L,D] as the cells write it, z and y [B,L,H,D].
// Gradient, with n = norm(o), d = dy act(z) w:  d_o = d norm(o) (d),  dz = dy n w act'(z),
// dw = sum dy act(z) n. gla_norm_common.cuh describes the layout and the row sums.
#include "gla_norm_common.cuh"

namespace gla {
namespace {

using namespace norm;
using tc::ex2;

// act(z) and its derivative for two channels, from p = 1 / (1 + 2^(-z log2 e)). The product is rounded
// before the exponential: an error of up to |z| 2^-24 in p, which bf16 data leave at that (2^-19 at
// |z| = 25, below a hundredth of their rounding) and fp32 data correct by the product's remainder.
template <typename T, int ACT>
__device__ __forceinline__ void act_grad2(uint64_t z, uint64_t& f, uint64_t& df) {
    constexpr float kL = 1.44269502162933349609375f, kLo = 1.92596299e-8f;   // log2 e as a sum
    const uint64_t y = f2_mul(z, f2_all(-kL));
    float y0, y1;
    f2_split(y, y0, y1);
    uint64_t e = f2(ex2(y0), ex2(y1));
    if constexpr (std::is_same<T, float>::value) {
        // beyond |y| = 126 e is 0 or infinite to fp32's purposes, and the remainder may be anything
        uint64_t rest = f2_fma(z, f2_all(-kLo), f2_fma(z, f2_all(-kL), f2_mul(y, f2_all(-1.f))));
        float r0, r1;
        f2_split(rest, r0, r1);
        rest = f2(fabsf(y0) < 126.f ? r0 : 0.f, fabsf(y1) < 126.f ? r1 : 0.f);
        e = f2_mul(e, f2_fma(rest, f2_all(0.693147182464599609375f), f2_all(1.f)));
    }
    float u0, u1;
    f2_split(f2_add(e, f2_all(1.f)), u0, u1);
    const uint64_t p = f2(tc::rcp_approx(u0), tc::rcp_approx(u1));   // 0 where e is infinite
    if (ACT == GLA_ACT_SILU) {
        const uint64_t q = f2_fma(p, f2_all(-1.f), f2_all(1.f));   // next to z q of 1 + z q its rounding is small
        f = f2_mul(z, p);
        df = f2_mul(p, f2_fma(z, q, f2_all(1.f)));
    } else {
        // 1 - p as e p keeps its digits where p is near 1 (at z = 15 the difference is off by a fifth); where e is
        // infinite the product is NaN and the minimum 1
        float q0, q1;
        f2_split(f2_mul(e, p), q0, q1);
        f = p;
        df = f2_mul(p, f2(fminf(q0, 1.f), fminf(q1, 1.f)));
    }
}

// The tokens of one head that a thread's group takes, one every `step`: element offsets of the token in
// [B,H,L,D] and in [B,L,H,D], advanced without products or divisions.
struct Token {
    size_t src, dst;
    int l;
};
struct Walk {
    size_t dsrc, ddst, wrap;
    int sl, L;
    __device__ __forceinline__ Walk(long long step, int H, int L_, int D) : L(L_) {
        const long long sb = step / L;
        sl = (int)(step - sb * L);
        dsrc = ((size_t)sb * H * L + sl) * D;
        ddst = (size_t)step * H * D;
        wrap = (size_t)(H - 1) * L * D;   // from the next batch's head 0 to ours, less this batch's tokens
    }
    __device__ __forceinline__ Token first(long long t, int h, int H, int D) const {
        const long long b = t / L;
        Token k;
        k.l = (int)(t - b * L);
        k.src = (((size_t)b * H + h) * L + k.l) * D;
        k.dst = ((size_t)t * H + h) * D;
        return k;
    }
    __device__ __forceinline__ void go(Token& k) const {
        k.src += dsrc;
        k.dst += ddst;
        k.l += sl;
        if (k.l >= L) k.l -= L, k.src += wrap;
    }
};

// blockIdx.y = head; a row of the block = one token of that head.
template <typename T, int VEC, int NV, int S, int KIND, int ACT, int MAXT, bool ODD>
__global__ void __launch_bounds__(MAXT, MAXT == 256 ? 2 : 1)   // 68 us at 128 registers, 77 at 64
    k_headnorm_fwd(const T* __restrict__ o, const T* __restrict__ z, const float* __restrict__ w, T* __restrict__ y,
                   int tokens, int H, int L, int D, int G, int w_stride, float eps) {
    extern __shared__ __align__(128) uint8_t smem[];
    constexpr int NP = kPairs<VEC>;
    using F = std::conditional_t<ODD, RowFeed<S>, Feed<S>>;
    constexpr int ZOFF = F::template bytes<T, VEC, NV>(), ROW = 2 * ZOFF;
    RowSum sum{reinterpret_cast<float*>(smem), G, 0};
    F feed = make_feed<S, ODD>(smem + kHead, ROW, G);
    const int grp = threadIdx.x / G, ngrp = blockDim.x / G, h = blockIdx.y;
    const Place P{(int)threadIdx.x - grp * G, G, ODD ? (D + 1) / 2 : D / VEC, D};
    const float inv_d = 1.f / D;
    uint64_t wv[NV][NP];
    load_columns<VEC, NV, ODD>(wv, w ? w + (size_t)h * w_stride : nullptr, P, 1.f);
    const long long step = (long long)gridDim.x * ngrp;
    long long t = (long long)blockIdx.x * ngrp + grp, ahead = t;
    const Walk walk(step, H, L, D);
    Token in = walk.first(t, h, H, D), out = in;   // the next token to copy, the current one
    auto copy = [&](int stage) {
        if constexpr (S > 0) {
            if constexpr (ODD) {
                if (ahead < tokens) {
                    const size_t n = (size_t)tokens * H * D;
                    feed.copy_row(stage, 0, o, in.src, n, P);
                    if (z) feed.copy_row(stage, ZOFF, z, in.dst, n, P);
                }
            } else if (ahead < tokens) {
#pragma unroll
                for (int j = 0; j < NV; ++j)
                    if (P.has(j)) {
                        feed.template copy<T, VEC>(stage, 0, j, o + in.src + P.col<VEC>(j));
                        if (z) feed.template copy<T, VEC>(stage, ZOFF, j, z + in.dst + P.col<VEC>(j));
                    }
            }
            feed.commit();
            walk.go(in);
            ahead += step;
        }
    };
#pragma unroll
    for (int k = 0; k + 1 < S; ++k) copy(k);
    for (long long first = (long long)blockIdx.x * ngrp; first < tokens; first += step, t += step) {
        const bool live = t < tokens;
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
                if constexpr (S > 0) feed.template read<T, VEC>(0, j, r[j], out.src, P);
                else load_piece<VEC>(o + out.src + P.col<VEC>(j), r[j]);
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
                if (z) {
                    uint64_t zv[NP];
                    if constexpr (S > 0) feed.template read<T, VEC>(ZOFF, j, zv, out.dst, P);
                    else load_piece<VEC>(z + out.dst + P.col<VEC>(j), zv);
#pragma unroll
                    for (int i = 0; i < NP; ++i) {
                        uint64_t f, df;
                        act_grad2<T, ACT>(zv[i], f, df);
                        r[j][i] = f2_mul(r[j][i], f);
                    }
                }
                put_piece<VEC, ODD>(y + out.dst, P, j, r[j]);
            }
        feed.next();
        walk.go(out);
    }
}

template <typename T, int VEC, int NV, int S, int KIND, int ACT, int MAXT, bool ODD>
__global__ void __launch_bounds__(MAXT, MAXT == 256 ? 2 : 1)
    k_headnorm_bwd(const T* __restrict__ o, const T* __restrict__ z, const float* __restrict__ w,
                   const T* __restrict__ dy, T* __restrict__ d_o, T* __restrict__ dz, float* __restrict__ pdw,
                   int tokens, int H, int L, int D, int G, int w_stride, float eps) {
    extern __shared__ __align__(128) uint8_t smem[];
    constexpr int NP = kPairs<VEC>;
    using F = std::conditional_t<ODD, RowFeed<S>, Feed<S>>;
    constexpr int ZOFF = F::template bytes<T, VEC, NV>(), YOFF = 2 * ZOFF, ROW = 3 * ZOFF;
    RowSum sum{reinterpret_cast<float*>(smem), G, 0};
    F feed = make_feed<S, ODD>(smem + kHead, ROW, G);
    const int grp = threadIdx.x / G, ngrp = blockDim.x / G, h = blockIdx.y;
    const Place P{(int)threadIdx.x - grp * G, G, ODD ? (D + 1) / 2 : D / VEC, D};
    const float inv_d = 1.f / D;
    uint64_t wv[NV][NP], aw[NV][NP] = {};
    load_columns<VEC, NV, ODD>(wv, w ? w + (size_t)h * w_stride : nullptr, P, 1.f);
    const long long step = (long long)gridDim.x * ngrp;
    long long t = (long long)blockIdx.x * ngrp + grp, ahead = t;
    const Walk walk(step, H, L, D);
    Token in = walk.first(t, h, H, D), out = in;   // the next token to copy, the current one
    auto copy = [&](int stage) {
        if constexpr (S > 0) {
            if constexpr (ODD) {
                if (ahead < tokens) {
                    const size_t n = (size_t)tokens * H * D;
                    feed.copy_row(stage, 0, o, in.src, n, P);
                    feed.copy_row(stage, YOFF, dy, in.dst, n, P);
                    if (z) feed.copy_row(stage, ZOFF, z, in.dst, n, P);
                }
            } else if (ahead < tokens) {
#pragma unroll
                for (int j = 0; j < NV; ++j)
                    if (P.has(j)) {
                        feed.template copy<T, VEC>(stage, 0, j, o + in.src + P.col<VEC>(j));
                        feed.template copy<T, VEC>(stage, YOFF, j, dy + in.dst + P.col<VEC>(j));
                        if (z) feed.template copy<T, VEC>(stage, ZOFF, j, z + in.dst + P.col<VEC>(j));
                    }
            }
            feed.commit();
            walk.go(in);
            ahead += step;
        }
    };
#pragma unroll
    for (int k = 0; k + 1 < S; ++k) copy(k);
    for (long long first = (long long)blockIdx.x * ngrp; first < tokens; first += step, t += step) {
        const bool live = t < tokens;
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
                if constexpr (S > 0) feed.template read<T, VEC>(0, j, r[j], out.src, P);
                else load_piece<VEC>(o + out.src + P.col<VEC>(j), r[j]);
            }
        }
        center<KIND, VEC, NV, ODD>(sum, r, P, inv_d);
        uint64_t t0 = 0, t1 = 0, t2 = 0;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
#pragma unroll
            for (int i = 0; i < NP; ++i) q[j][i] = d[j][i] = 0;
            if (live && P.has(j)) {
                uint64_t zv[NP];
                if constexpr (S > 0) feed.template read<T, VEC>(YOFF, j, q[j], out.dst, P);
                else load_piece<VEC>(dy + out.dst + P.col<VEC>(j), q[j]);
                if (z) {
                    if constexpr (S > 0) feed.template read<T, VEC>(ZOFF, j, zv, out.dst, P);
                    else load_piece<VEC>(z + out.dst + P.col<VEC>(j), zv);
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
                if (dz) put_piece<VEC, ODD>(dz + out.dst, P, j, d[j]);
                put_piece<VEC, ODD>(d_o + out.src, P, j, r[j]);
            }
        feed.next();
        walk.go(out);
    }
    grid_dep_launch();
    if (pdw)
        write_partial<VEC, NV, ODD>(aw, reinterpret_cast<float*>(smem), grp, P, pdw + ((size_t)blockIdx.x * H + h) * D);
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

RowPlan plan(const gla_norm_problem* p) { return row_plan(p->D, p->io == GLA_BF16, p->io == GLA_F32); }

// Whether the blocks' column sums are the result already: one block, or one per head and head's weights.
bool is_direct(const gla_norm_problem* p, int P) { return P == 1 && (p->w_per_head || p->H == 1); }

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
    const int P = p->H ? row_blocks(plan(p), (long long)p->B * p->L, p->H) : 0;
    return is_direct(p, P) ? 256 : 256 + (size_t)P * p->H * p->D * 4;
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
    const RowPlan rp = plan(p);
    const cudaError_t e = by_io(p->io, [&](auto tv) {
        using T = decltype(tv);
        const int thread_bytes = 2 * rp.nv * rp.vec * (int)sizeof(T);
        return by_shape<sizeof(T) == 2, sizeof(T) == 4, false>(rp, ring_stages(rp, thread_bytes, p->kind), [&](auto sh) {
            return by_kind(p->kind, [&](auto kind) {
                return by_act(p->act, [&](auto act) {
                    using Sh = decltype(sh);
                    auto kern = k_headnorm_fwd<T, Sh::vec, Sh::nv, Sh::stages, decltype(kind)::value,
                                               decltype(act)::value, Sh::maxt, Sh::odd>;
                    const size_t smem = block_smem(rp, Sh::stages, thread_bytes);
                    static std::atomic<bool> seen[kMaxDevices];
                    static Occupancy known;
                    const cudaError_t e = smem_attr_once(kern, kSmSmem, seen);
                    if (e != cudaSuccess) return e;
                    const dim3 grid(fit_blocks(kern, rp, smem, row_blocks(rp, tokens, p->H), p->H, known), p->H);
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
    const int tokens = p->B * p->L;
    const RowPlan rp = plan(p);
    int P = p->H ? row_blocks(rp, tokens, p->H) : 0;
    const bool direct = is_direct(p, P), partials = P > 0 && !direct;
    if (!all_aligned(ptrs) || (!ws && partials) || (dz && !z)) return GLA_ERR_INVALID_ARG;
    if (partials && ws_bytes < gla_headnorm_workspace_bytes(p)) return GLA_ERR_WORKSPACE;
    cudaStream_t st = (cudaStream_t)stream;
    if (p->H == 0 && (!dw || p->w_per_head)) return GLA_OK;
    float* pdw = !dw || direct ? dw : static_cast<float*>(ws);
    cudaError_t e = cudaSuccess;
    if (tokens > 0 && p->H > 0) {
        if (!o || !dy || !d_o) return GLA_ERR_INVALID_ARG;
        e = by_io(p->io, [&](auto tv) {
            using T = decltype(tv);
            const int thread_bytes = 3 * rp.nv * rp.vec * (int)sizeof(T);
            return by_shape<sizeof(T) == 2, sizeof(T) == 4, false>(rp, ring_stages(rp, thread_bytes, p->kind), [&](auto sh) {
                return by_kind(p->kind, [&](auto kind) {
                    return by_act(p->act, [&](auto act) {
                        using Sh = decltype(sh);
                        auto kern = k_headnorm_bwd<T, Sh::vec, Sh::nv, Sh::stages, decltype(kind)::value,
                                                   decltype(act)::value, Sh::maxt, Sh::odd>;
                        const size_t smem = block_smem(rp, Sh::stages, thread_bytes);
                        static std::atomic<bool> seen[kMaxDevices];
                        static Occupancy known;
                        const cudaError_t e = smem_attr_once(kern, kSmSmem, seen);
                        if (e != cudaSuccess) return e;
                        P = fit_blocks(kern, rp, smem, P, p->H, known);
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
    if (e == cudaSuccess && dw && !direct)
        e = p->w_per_head ? colsum(pdw, dw, nullptr, nullptr, P, (size_t)p->H * p->D, p->H * p->D, st)
                          : colsum(pdw, dw, nullptr, nullptr, P * p->H, p->D, p->D, st);
    return record_cuda(e, "headnorm backward");
}

}  // extern "C"
