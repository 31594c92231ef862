// Gated linear recurrence with a vector state (the elementwise member of the family of the GLA
// abstract's data-dependent gates; the talk summary "Hardware-Efficient Training of Linear
// Attention Models", section 7:36, names the scan over states):
//   h_t = a_t h_{t-1} + m(a_t) x_t,  o_t = h_t,  a = e^g,  m = 1 | 1 - a | sqrt(1 - a^2),
// per (b, h, channel). Backward, with D_t = a_t dh_t the gradient handed to h_{t-1}:
//   dh_t = dO_t + D_{t+1},  dx_t = m dh_t,  dg_t = dh_t (a_t h_{t-1} + m'(g_t) x_t),  dh0 = D_0.
//
// A run of tokens maps the state before it to the state after it, h -> A h + B, with A the product
// of its decays and B its end state from zero; runs compose, (A1, B1) then (A2, B2) giving
// (A1 A2, A2 B1 + B2). The kernels use that at four levels: a thread's tokens, a warp's runs
// (shuffles), a tile's warps (shared memory), and the tiles of a thread-block cluster, which walks
// the sequence one row of tiles at a time and exchanges the tiles' (A, B) through distributed
// shared memory. So every input is read once and the sequence is split over as many SMs as
// the channels alone would leave idle. The reverse recurrence of the backward composes the same
// way from the other end with the same A.
#include <type_traits>

#include "gla_common.cuh"
#include "gla_plans.h"
#include "gla_tc_common.cuh"
#include "sm100.cuh"

namespace gla {
namespace {

using namespace sm100;

constexpr int kSaveEvery = 64;   // tokens between two saved states
constexpr int NT_S = 256;        // threads of a tile
constexpr int NW = NT_S / 32;
constexpr int VEC = 4;           // channels of a thread
constexpr int RUN = 4;           // tokens of a thread
constexpr int kMaxCluster = 8;
constexpr int kMaxStages = 4;

// How a tile reaches shared memory.
enum { LOAD_TMA = 0, LOAD_VEC4 = 1, LOAD_ONE = 2 };

// 1 - e^g and e^g. Near 0 (|g| < 0.35, where a gate's memory is long and an error in a is
// multiplied by 1 / (1 - a)) 1 - e^g is its Taylor series through g^7 / 7! (first term left out:
// g^7 / 8! < 1.7e-8 of the value), and a = 1 - t is then exact to one rounding; elsewhere the
// hardware exponential serves.
__device__ __forceinline__ void gate(float g, float& a, float& t) {
    float s = fmaf(g, 1.f / 5040.f, 1.f / 720.f);
    s = fmaf(g, s, 1.f / 120.f);
    s = fmaf(g, s, 1.f / 24.f);
    s = fmaf(g, s, 1.f / 6.f);
    s = fmaf(g, s, 0.5f);
    s = fmaf(g, s, 1.f);
    const float tn = -g * s, af = __expf(g);
    const bool near = fabsf(g) < 0.35f;
    t = near ? tn : 1.f - af;
    a = near ? 1.f - tn : af;
}

// The factor on the input and its derivative with respect to g. u = 1 - a^2 = t (1 + a); u < 0
// (g > 0) gives NaN like the formula.
template <int IN>
__device__ __forceinline__ float in_factor(float t) {
    if (IN == GLA_SCAN_PLAIN) return 1.f;
    if (IN == GLA_SCAN_COMPLEMENT) return t;
    const float u = t * (2.f - t);
    return u == 0.f ? 0.f : u * rsqrtf(u);
}
template <int IN>
__device__ __forceinline__ float in_slope(float a, float m) {
    if (IN == GLA_SCAN_PLAIN) return 0.f;
    if (IN == GLA_SCAN_COMPLEMENT) return -a;
    return m == 0.f ? 0.f : __fdividef(-a * a, m);
}

// ------------------------------------------------------------------ four channels of a token
__device__ __forceinline__ void lds4(const float* p, float (&v)[VEC]) {
    const float4 f = *reinterpret_cast<const float4*>(p);
    v[0] = f.x; v[1] = f.y; v[2] = f.z; v[3] = f.w;
}
__device__ __forceinline__ void lds4(const __nv_bfloat16* p, float (&v)[VEC]) {
    const uint2 u = *reinterpret_cast<const uint2*>(p);
    v[0] = __uint_as_float(u.x << 16); v[1] = __uint_as_float(u.x & 0xffff0000u);
    v[2] = __uint_as_float(u.y << 16); v[3] = __uint_as_float(u.y & 0xffff0000u);
}
__device__ __forceinline__ void st4(float* p, const float (&v)[VEC]) {
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
}
__device__ __forceinline__ void st4(__nv_bfloat16* p, const float (&v)[VEC]) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(v[0], v[1]), b = __floats2bfloat162_rn(v[2], v[3]);
    *reinterpret_cast<uint2*>(p) =
        make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
}
// Stores the channels c .. c+3 that exist; whole vectors where D allows.
template <int LOAD, typename T>
__device__ __forceinline__ void put4(T* p, const float (&v)[VEC], int c, int D) {
    if (LOAD != LOAD_ONE) {
        if (c < D) st4(p, v);
    } else {
#pragma unroll
        for (int i = 0; i < VEC; ++i)
            if (c + i < D) p[i] = from_f<T>(v[i]);
    }
}

// (A, B) of this CTA's tile into slot `dst` of the cluster's CTA `rank`, counted on its barrier.
__device__ __forceinline__ void st_async_pair(uint32_t dst, uint32_t bar, float a, float b) {
    asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v2.f32 [%0], {%1, %2}, [%3];" ::"r"(dst),
                 "f"(a), "f"(b), "r"(bar)
                 : "memory");
}

// Geometry of a tile: CHL lanes cover CH channels, the other lanes and the warps split TT tokens.
template <int CHL>
struct Geo {
    static constexpr int CH = CHL * VEC;
    static constexpr int RW = 32 / CHL;          // runs of a warp
    static constexpr int WT = RW * RUN;          // tokens of a warp
    static constexpr int TT = NW * WT;           // tokens of a tile
    static constexpr int ELEMS = TT * CH;
};

// Shared memory behind the ring: per-warp sums, per-warp start values, exchange slots, barriers.
template <int CHL, int SUMS>
struct Tail {
    float sum[SUMS][NW][Geo<CHL>::CH];
    float start[SUMS - 1][NW][Geo<CHL>::CH];
    float2 slot[2][kMaxCluster][Geo<CHL>::CH];
    uint64_t full[kMaxStages];
    uint64_t got[2];
};

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

// A tile's elements into shared memory by ordinary loads, zeros (the identity: a = 1, b = 0) outside.
template <int CHL, int LOAD, typename T>
__device__ __forceinline__ void fill(T* dst, const T* __restrict__ src, size_t bh, int t0, int c0, int L, int D) {
    using G = Geo<CHL>;
    if (LOAD == LOAD_VEC4) {
        constexpr int N = G::ELEMS / VEC / NT_S;
        float v[N][VEC];
#pragma unroll
        for (int k = 0; k < N; ++k) {
            const int e = threadIdx.x + k * NT_S, t = e / CHL, c = (e % CHL) * VEC;
            v[k][0] = v[k][1] = v[k][2] = v[k][3] = 0.f;
            if (t0 + t < L && c0 + c < D) lds4(src + (bh * L + t0 + t) * D + c0 + c, v[k]);
        }
#pragma unroll
        for (int k = 0; k < N; ++k) {
            const int e = threadIdx.x + k * NT_S;
            st4(dst + e * VEC, v[k]);
        }
    } else {
        constexpr int N = G::ELEMS / NT_S;
        T v[N];
#pragma unroll
        for (int k = 0; k < N; ++k) {
            const int e = threadIdx.x + k * NT_S, t = e / G::CH, c = e % G::CH;
            v[k] = from_f<T>(0.f);
            if (t0 + t < L && c0 + c < D) v[k] = src[(bh * L + t0 + t) * D + c0 + c];
        }
#pragma unroll
        for (int k = 0; k < N; ++k) dst[threadIdx.x + k * NT_S] = v[k];
    }
}

struct ScanArgs {
    const void* x;
    const float* g;
    const void* dO;
    const float* first;    // h0 (forward), dhT (backward); may be null
    void* out;             // o, dx
    float* dg;
    float* last;           // hT, dh0; may be null
    float* saved;          // written (forward, may be null), read (backward)
    int L, D, nblk, steps, stages;
};

// Inclusive composition over the runs of a warp, lanes CHL apart, from the first run on.
template <int CHL>
__device__ __forceinline__ void warp_compose_up(float (&A)[VEC], float (&B)[VEC], int run) {
#pragma unroll
    for (int off = CHL; off < 32; off <<= 1)
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            const float pa = __shfl_up_sync(0xffffffffu, A[i], off), pb = __shfl_up_sync(0xffffffffu, B[i], off);
            if (run >= off / CHL) {
                B[i] = fmaf(A[i], pb, B[i]);
                A[i] *= pa;
            }
        }
}
// The same from the last run backwards.
template <int CHL>
__device__ __forceinline__ void warp_compose_down(float (&A)[VEC], float (&B)[VEC], int run) {
#pragma unroll
    for (int off = CHL; off < 32; off <<= 1)
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            const float pa = __shfl_down_sync(0xffffffffu, A[i], off), pb = __shfl_down_sync(0xffffffffu, B[i], off);
            if (run + off / CHL < 32 / CHL) {
                B[i] = fmaf(A[i], pb, B[i]);
                A[i] *= pa;
            }
        }
}

// Sends (A, B) to every CTA of the cluster, waits for theirs and composes them onto `super` in
// sequence order (reverse order for REV). Returns the value entering this CTA's tile; `super`
// becomes the value leaving the row of tiles. Slots are used in turn, two rows of tiles apart: a
// CTA writes row i + 2 only after it has seen every CTA's row i + 1, which each thread sends after
// it has read its channel of row i.
template <int CHL, bool REV, int SUMS>
__device__ __forceinline__ float exchange(Tail<CHL, SUMS>& sm, int c, float A, float B, int cs, int rank, int i,
                                          float& super, bool& ok) {
    if (cs == 1) {
        const float in = super;
        super = fmaf(A, super, B);
        return in;
    }
    const int p = i & 1;
    if (c == 0) mbar_arrive_expect_tx(&sm.got[p], cs * Geo<CHL>::CH * (uint32_t)sizeof(float2));
    for (int r = 0; r < cs; ++r)
        st_async_pair(mapa_shared(&sm.slot[p][rank][c], r), mapa_shared(&sm.got[p], r), A, B);
    if (ok) ok = mbar_wait_cluster(&sm.got[p], (i >> 1) & 1);
    float in = super;
    for (int k = 0; k < cs; ++k) {
        const int r = REV ? cs - 1 - k : k;
        if (r == rank) in = super;
        const float2 v = sm.slot[p][r][c];
        super = fmaf(v.x, super, v.y);
    }
    return in;
}

// One cluster per (b, h, block of CH channels); its CTAs take the tiles of a row of tiles in
// order and walk the rows together. Three phases a row, with a barrier after the first two:
// (1) every thread composes its tokens, warps their runs; (2) one thread per channel composes the
// warps and the cluster's tiles; (3) every thread walks its tokens again from its start value.
// The ring of tiles hides the loads; phase 2 hides behind the SM's other CTAs.
template <typename T, int IN, int CHL, int LOAD>
__global__ void __launch_bounds__(NT_S, 3)
    k_scan_fwd(const __grid_constant__ CUtensorMap mx, const __grid_constant__ CUtensorMap mg, const ScanArgs P,
               int cs) {
    using G = Geo<CHL>;
    extern __shared__ __align__(128) uint8_t smem[];
    constexpr int kStage = G::ELEMS * (4 + (int)sizeof(T));
    Tail<CHL, 2>& sm = *reinterpret_cast<Tail<CHL, 2>*>(smem + P.stages * kStage);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int run = lane / CHL, ch = (lane % CHL) * VEC;
    const int rank = cs > 1 ? (int)cluster_rank() : 0;
    const unsigned chain = blockIdx.x / cs;
    const size_t bh = chain / P.nblk;
    const int c0 = (int)(chain % P.nblk) * G::CH;
    const int tr = warp * G::WT + run * RUN;   // this thread's first token in a tile
    const int L = P.L, D = P.D;
    bool ok = true;   // false once a wait gave up: no further wait, the results are not valid

    if (tid == 0) {
        for (int s = 0; s < kMaxStages; ++s) mbar_init(&sm.full[s], 1);
        mbar_init(&sm.got[0], 1);
        mbar_init(&sm.got[1], 1);
        mbar_fence_init();
    }
    if (cs > 1) cluster_sync();
    else __syncthreads();

    auto load = [&](int i) {   // one thread
        const int s = i % P.stages;
        float* sg = reinterpret_cast<float*>(smem + s * kStage);
        mbar_arrive_expect_tx(&sm.full[s], kStage);
        tma_load_3d(sg, &mg, c0, (i * cs + rank) * G::TT, (int)bh, &sm.full[s]);
        tma_load_3d(sg + G::ELEMS, &mx, c0, (i * cs + rank) * G::TT, (int)bh, &sm.full[s]);
    };
    if (LOAD == LOAD_TMA && tid == 0)
        for (int i = 0; i < P.stages && i < P.steps; ++i) load(i);

    float super = 0.f;
    if (tid < G::CH && P.first && c0 + tid < D) super = P.first[bh * D + c0 + tid];

    for (int i = 0; i < P.steps; ++i) {
        const int s = LOAD == LOAD_TMA ? i % P.stages : 0, t0 = (i * cs + rank) * G::TT;
        float* sg = reinterpret_cast<float*>(smem + s * kStage);
        T* sx = reinterpret_cast<T*>(sg + G::ELEMS);
        if (LOAD == LOAD_TMA) {
            if (ok) ok = mbar_wait(&sm.full[s], (i / P.stages) & 1);
        } else {
            fill<CHL, LOAD>(sg, P.g, bh, t0, c0, L, D);
            fill<CHL, LOAD>(sx, static_cast<const T*>(P.x), bh, t0, c0, L, D);
            __syncthreads();
        }
        float a[RUN][VEC], b[RUN][VEC], A[VEC], B[VEC];
#pragma unroll
        for (int j = 0; j < RUN; ++j) {
            float gv[VEC], xv[VEC];
            lds4(sg + (tr + j) * G::CH + ch, gv);
            lds4(sx + (tr + j) * G::CH + ch, xv);
#pragma unroll
            for (int k = 0; k < VEC; ++k) {
                float u;
                gate(gv[k], a[j][k], u);
                b[j][k] = in_factor<IN>(u) * xv[k];
                A[k] = j ? A[k] * a[j][k] : a[j][k];
                B[k] = j ? fmaf(a[j][k], B[k], b[j][k]) : b[j][k];
            }
        }
        warp_compose_up<CHL>(A, B, run);
        if (run == G::RW - 1) {
            st4(&sm.sum[0][warp][ch], A);
            st4(&sm.sum[1][warp][ch], B);
        }
        // what the warp's earlier runs do to the warp's start value
        float eA[VEC], eB[VEC];
#pragma unroll
        for (int k = 0; k < VEC; ++k) {
            eA[k] = __shfl_up_sync(0xffffffffu, A[k], CHL);
            eB[k] = __shfl_up_sync(0xffffffffu, B[k], CHL);
            if (run == 0) eA[k] = 1.f, eB[k] = 0.f;
        }
        __syncthreads();
        if (LOAD == LOAD_TMA && tid == 0 && i + P.stages < P.steps) load(i + P.stages);
        if (tid < G::CH) {
            float pA[NW], pB[NW], tA = 1.f, tB = 0.f;
#pragma unroll
            for (int w = 0; w < NW; ++w) {
                pA[w] = tA, pB[w] = tB;
                const float wa = sm.sum[0][w][tid], wb = sm.sum[1][w][tid];
                tB = fmaf(wa, tB, wb);
                tA *= wa;
            }
            const float in = exchange<CHL, false>(sm, tid, tA, tB, cs, rank, i, super, ok);
#pragma unroll
            for (int w = 0; w < NW; ++w) {
                const float h = fmaf(pA[w], in, pB[w]);
                sm.start[0][w][tid] = h;
                const int t = t0 + w * G::WT;
                if (w * G::WT % kSaveEvery == 0 && P.saved && t < L && c0 + tid < D)
                    P.saved[(bh * cdiv(L, kSaveEvery) + t / kSaveEvery) * D + c0 + tid] = h;
            }
        }
        __syncthreads();
        if (P.out) {
            float h[VEC];
            lds4(&sm.start[0][warp][ch], h);
            T* op = static_cast<T*>(P.out) + (bh * L + t0 + tr) * D + c0 + ch;
#pragma unroll
            for (int k = 0; k < VEC; ++k) h[k] = fmaf(eA[k], h[k], eB[k]);
#pragma unroll
            for (int j = 0; j < RUN; ++j) {
#pragma unroll
                for (int k = 0; k < VEC; ++k) h[k] = fmaf(a[j][k], h[k], b[j][k]);
                if (t0 + tr + j < L) put4<LOAD>(op + (size_t)j * D, h, c0 + ch, D);
            }
        }
    }
    if (P.last && rank == 0 && tid < G::CH && c0 + tid < D) P.last[bh * D + c0 + tid] = super;
    if (cs > 1) cluster_sync();   // no CTA leaves while another may still write to its slots
}

// The same walk from the sequence's end, with the states recomputed inside each tile from the saved
// ones: phase 1 also composes the reverse recurrence, phase 2 starts the forward one from
// the saved state of every 64 tokens and carries the reverse one through the cluster, and phase 3
// walks forward for h_{t-1}, then backward for the gradients.
template <typename T, int IN, int CHL, int LOAD>
__global__ void __launch_bounds__(NT_S, 2)
    k_scan_bwd(const __grid_constant__ CUtensorMap mx, const __grid_constant__ CUtensorMap mg,
               const __grid_constant__ CUtensorMap md, const ScanArgs P, int cs) {
    using G = Geo<CHL>;
    extern __shared__ __align__(128) uint8_t smem[];
    constexpr int kStage = G::ELEMS * (4 + 2 * (int)sizeof(T));
    Tail<CHL, 3>& sm = *reinterpret_cast<Tail<CHL, 3>*>(smem + P.stages * kStage);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int run = lane / CHL, ch = (lane % CHL) * VEC;
    const int rank = cs > 1 ? (int)cluster_rank() : 0;
    const unsigned chain = blockIdx.x / cs;
    const size_t bh = chain / P.nblk;
    const int c0 = (int)(chain % P.nblk) * G::CH;
    const int tr = warp * G::WT + run * RUN;
    const int L = P.L, D = P.D;
    bool ok = true;   // false once a wait gave up: no further wait, the results are not valid

    if (tid == 0) {
        for (int s = 0; s < kMaxStages; ++s) mbar_init(&sm.full[s], 1);
        mbar_init(&sm.got[0], 1);
        mbar_init(&sm.got[1], 1);
        mbar_fence_init();
    }
    if (cs > 1) cluster_sync();
    else __syncthreads();

    // rows are counted from the end: row i holds the tiles (steps - 1 - i) cs + rank
    auto load = [&](int i) {
        const int s = i % P.stages, t0 = ((P.steps - 1 - i) * cs + rank) * G::TT;
        float* sg = reinterpret_cast<float*>(smem + s * kStage);
        T* sx = reinterpret_cast<T*>(sg + G::ELEMS);
        mbar_arrive_expect_tx(&sm.full[s], kStage);
        tma_load_3d(sg, &mg, c0, t0, (int)bh, &sm.full[s]);
        tma_load_3d(sx, &mx, c0, t0, (int)bh, &sm.full[s]);
        tma_load_3d(sx + G::ELEMS, &md, c0, t0, (int)bh, &sm.full[s]);
    };
    if (LOAD == LOAD_TMA && tid == 0)
        for (int i = 0; i < P.stages - 1 && i < P.steps; ++i) load(i);

    float super = 0.f;
    if (tid < G::CH && P.first && c0 + tid < D) super = P.first[bh * D + c0 + tid];

    for (int i = 0; i < P.steps; ++i) {
        const int s = LOAD == LOAD_TMA ? i % P.stages : 0, t0 = ((P.steps - 1 - i) * cs + rank) * G::TT;
        float* sg = reinterpret_cast<float*>(smem + s * kStage);
        T* sx = reinterpret_cast<T*>(sg + G::ELEMS);
        T* sd = sx + G::ELEMS;
        constexpr int NS = G::TT / kSaveEvery;   // saved states of a tile
        float sv[NS];
        if (tid < G::CH)
#pragma unroll
            for (int n = 0; n < NS; ++n) {
                const int t = t0 + n * kSaveEvery;
                sv[n] = t < L && c0 + tid < D
                            ? P.saved[(bh * cdiv(L, kSaveEvery) + t / kSaveEvery) * D + c0 + tid] : 0.f;
            }
        if (LOAD == LOAD_TMA) {
            if (ok) ok = mbar_wait(&sm.full[s], (i / P.stages) & 1);
        } else {
            __syncthreads();   // the previous row's readers
            fill<CHL, LOAD>(sg, P.g, bh, t0, c0, L, D);
            fill<CHL, LOAD>(sx, static_cast<const T*>(P.x), bh, t0, c0, L, D);
            fill<CHL, LOAD>(sd, static_cast<const T*>(P.dO), bh, t0, c0, L, D);
            __syncthreads();
        }
        float a[RUN][VEC], m[RUN][VEC], A[VEC], B[VEC], Q[VEC], R[VEC];
#pragma unroll
        for (int j = 0; j < RUN; ++j) {
            float gv[VEC], xv[VEC];
            lds4(sg + (tr + j) * G::CH + ch, gv);
            lds4(sx + (tr + j) * G::CH + ch, xv);
#pragma unroll
            for (int k = 0; k < VEC; ++k) {
                float u;
                gate(gv[k], a[j][k], u);
                m[j][k] = in_factor<IN>(u);
                A[k] = j ? A[k] * a[j][k] : a[j][k];
                B[k] = j ? fmaf(a[j][k], B[k], m[j][k] * xv[k]) : m[j][k] * xv[k];
            }
        }
#pragma unroll
        for (int j = RUN - 1; j >= 0; --j) {
            float dv[VEC];
            lds4(sd + (tr + j) * G::CH + ch, dv);
#pragma unroll
            for (int k = 0; k < VEC; ++k) R[k] = a[j][k] * (j == RUN - 1 ? dv[k] : dv[k] + R[k]);
        }
#pragma unroll
        for (int k = 0; k < VEC; ++k) Q[k] = A[k];
        warp_compose_up<CHL>(A, B, run);
        warp_compose_down<CHL>(Q, R, run);
        if (run == G::RW - 1) {
            st4(&sm.sum[0][warp][ch], A);
            st4(&sm.sum[1][warp][ch], B);
        }
        if (run == 0) st4(&sm.sum[2][warp][ch], R);
        float eA[VEC], eB[VEC], fA[VEC], fB[VEC];
#pragma unroll
        for (int k = 0; k < VEC; ++k) {
            eA[k] = __shfl_up_sync(0xffffffffu, A[k], CHL);
            eB[k] = __shfl_up_sync(0xffffffffu, B[k], CHL);
            if (run == 0) eA[k] = 1.f, eB[k] = 0.f;
            fA[k] = __shfl_down_sync(0xffffffffu, Q[k], CHL);
            fB[k] = __shfl_down_sync(0xffffffffu, R[k], CHL);
            if (run == G::RW - 1) fA[k] = 1.f, fB[k] = 0.f;
        }
        __syncthreads();
        // every thread is past the previous row, so its stage is free
        if (LOAD == LOAD_TMA && tid == 0 && i + P.stages - 1 < P.steps) load(i + P.stages - 1);
        if (tid < G::CH) {
            float wa[NW], qA[NW], qR[NW], tA = 1.f, tR = 0.f, h = 0.f;
#pragma unroll
            for (int w = 0; w < NW; ++w) {
                wa[w] = sm.sum[0][w][tid];
                if (w * G::WT % kSaveEvery == 0) h = sv[w * G::WT / kSaveEvery];
                sm.start[0][w][tid] = h;
                h = fmaf(wa[w], h, sm.sum[1][w][tid]);
            }
#pragma unroll
            for (int w = NW - 1; w >= 0; --w) {
                qA[w] = tA, qR[w] = tR;
                tR = fmaf(wa[w], tR, sm.sum[2][w][tid]);
                tA *= wa[w];
            }
            const float in = exchange<CHL, true>(sm, tid, tA, tR, cs, rank, i, super, ok);
#pragma unroll
            for (int w = 0; w < NW; ++w) sm.start[1][w][tid] = fmaf(qA[w], in, qR[w]);
        }
        __syncthreads();
        float h[VEC], d[VEC], hp[RUN][VEC];
        lds4(&sm.start[0][warp][ch], h);
        lds4(&sm.start[1][warp][ch], d);
#pragma unroll
        for (int k = 0; k < VEC; ++k) {
            h[k] = fmaf(eA[k], h[k], eB[k]);
            d[k] = fmaf(fA[k], d[k], fB[k]);
        }
#pragma unroll
        for (int j = 0; j < RUN; ++j) {
            float xv[VEC];
            lds4(sx + (tr + j) * G::CH + ch, xv);
#pragma unroll
            for (int k = 0; k < VEC; ++k) {
                // a h_{t-1} + m' x, dg's factor next to dh
                const float ah = a[j][k] * h[k];
                hp[j][k] = fmaf(in_slope<IN>(a[j][k], m[j][k]), xv[k], ah);
                h[k] = fmaf(m[j][k], xv[k], ah);
            }
        }
        const size_t at = (bh * L + t0 + tr) * D + c0 + ch;
        T* xp = static_cast<T*>(P.out) + at;
        float* gp = P.dg + at;
#pragma unroll
        for (int j = RUN - 1; j >= 0; --j) {
            float dv[VEC];
            lds4(sd + (tr + j) * G::CH + ch, dv);
            float ox[VEC], og[VEC];
#pragma unroll
            for (int k = 0; k < VEC; ++k) {
                const float dh = dv[k] + d[k];
                ox[k] = m[j][k] * dh;
                og[k] = hp[j][k] * dh;
                d[k] = a[j][k] * dh;
            }
            if (t0 + tr + j < L) {
                put4<LOAD>(xp + (size_t)j * D, ox, c0 + ch, D);
                put4<LOAD>(gp + (size_t)j * D, og, c0 + ch, D);
            }
        }
    }
    if (P.last && rank == 0 && tid < G::CH && c0 + tid < D) P.last[bh * D + c0 + tid] = super;
    if (cs > 1) cluster_sync();
}

// One token: the state is read and written once.
constexpr int NT_D = 128;
template <typename T, int IN>
__global__ void __launch_bounds__(NT_D) k_scan_decode(const T* __restrict__ x, const float* __restrict__ g,
                                                      float* __restrict__ state, T* __restrict__ o, size_t n) {
    const size_t i = (size_t)blockIdx.x * NT_D + threadIdx.x;
    if (i >= n) return;
    float a, u;
    gate(g[i], a, u);
    const float h = fmaf(a, state[i], in_factor<IN>(u) * to_f(x[i]));
    state[i] = h;
    o[i] = from_f<T>(h);
}

// Calls f(T{}, integral_constant<IN>) for the problem's dtype and input factor.
template <typename F>
cudaError_t dispatch(const gla_problem* p, int input, F&& f) {
    if (p->io == GLA_BF16) {
        if (input == GLA_SCAN_PLAIN) return f(__nv_bfloat16{}, std::integral_constant<int, GLA_SCAN_PLAIN>{});
        if (input == GLA_SCAN_COMPLEMENT) return f(__nv_bfloat16{}, std::integral_constant<int, GLA_SCAN_COMPLEMENT>{});
        return f(__nv_bfloat16{}, std::integral_constant<int, GLA_SCAN_NORM>{});
    }
    if (input == GLA_SCAN_PLAIN) return f(float{}, std::integral_constant<int, GLA_SCAN_PLAIN>{});
    if (input == GLA_SCAN_COMPLEMENT) return f(float{}, std::integral_constant<int, GLA_SCAN_COMPLEMENT>{});
    return f(float{}, std::integral_constant<int, GLA_SCAN_NORM>{});
}

bool aligned16(const void* x) { return x == nullptr || (reinterpret_cast<uintptr_t>(x) & 15u) == 0; }

gla_status check(const gla_problem* p) {
    if (!p || p->B < 0 || p->H < 0 || p->L < 0 || p->Dk != p->Dv || p->Dk < 1) return GLA_ERR_INVALID_ARG;
    if (p->io != GLA_F32 && p->io != GLA_BF16) return GLA_ERR_INVALID_ARG;
    if (p->gate != GLA_GATE_PER_KEY) return GLA_ERR_INVALID_ARG;
    if (p->Dk > 65536 || p->L > 1 << 30) return GLA_ERR_UNSUPPORTED;
    // at most 2^27 clusters of 8
    if ((long long)p->B * p->H * cdiv(p->Dk, 32) > 1 << 27) return GLA_ERR_UNSUPPORTED;
    return GLA_OK;
}
bool input_ok(int input) { return input >= GLA_SCAN_PLAIN && input <= GLA_SCAN_NORM; }

// 3D map over [BH][L][D] with a box of box_l x box_c.
template <typename T>
bool scan_map(CUtensorMap* m, const void* base, int D, int L, int BH, int box_c, int box_l) {
    auto fn = tc::encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)L, (cuuint64_t)BH};
    const cuuint64_t strides[2] = {(cuuint64_t)D * sizeof(T), (cuuint64_t)D * sizeof(T) * L};
    const cuuint32_t box[3] = {(cuuint32_t)box_c, (cuuint32_t)box_l, 1}, estr[3] = {1, 1, 1};
    return fn(m, std::is_same<T, float>::value ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3,
              const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Launches a walk: chooses the channels of a tile, the cluster and the ring.
template <typename T, int IN, int CHL, int LOAD, bool BWD>
cudaError_t launch_walk(const gla_problem* p, ScanArgs P, const CUtensorMap (&maps)[3], cudaStream_t st) {
    using G = Geo<CHL>;
    P.nblk = cdiv(P.D, G::CH);
    const long long chains = (long long)p->B * p->H * P.nblk;
    const int tiles = cdiv(P.L, G::TT), want = tc::num_sms() * 3;
    int cs = 1;
    while (cs < kMaxCluster && chains * cs < want && cs < tiles) cs *= 2;
    P.steps = cdiv(tiles, cs);
    constexpr int kStage = G::ELEMS * (4 + (BWD ? 2 : 1) * (int)sizeof(T));
    constexpr int most = LOAD == LOAD_TMA ? (BWD ? 3 : sizeof(T) == 2 ? 3 : 2) : 1;
    P.stages = P.steps < most ? P.steps : most;
    if (BWD && LOAD == LOAD_TMA && P.stages < 2) P.stages = 2;
    if (P.stages < 1) P.stages = 1;
    const size_t bytes = (size_t)P.stages * kStage + sizeof(Tail<CHL, BWD ? 3 : 2>);
    static std::atomic<bool> seen[kMaxDevices];
    const size_t top = (size_t)(most < 2 ? 2 : most) * kStage + sizeof(Tail<CHL, BWD ? 3 : 2>);
    cudaError_t e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(chains * cs));
    cfg.blockDim = dim3(NT_S);
    cfg.dynamicSmemBytes = bytes;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = cs;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if constexpr (BWD) {
        auto kern = k_scan_bwd<T, IN, CHL, LOAD>;
        if ((e = smem_attr_once(kern, top, seen)) != cudaSuccess) return e;
        GLA_LAUNCH("scan_bwd", st, (e = cudaLaunchKernelEx(&cfg, kern, maps[0], maps[1], maps[2], P, cs)));
    } else {
        auto kern = k_scan_fwd<T, IN, CHL, LOAD>;
        if ((e = smem_attr_once(kern, top, seen)) != cudaSuccess) return e;
        GLA_LAUNCH("scan_fwd", st, (e = cudaLaunchKernelEx(&cfg, kern, maps[0], maps[1], P, cs)));
    }
    return e;
}

template <typename T, int IN, bool BWD>
cudaError_t walk(const gla_problem* p, const ScanArgs& P, cudaStream_t st) {
    CUtensorMap maps[3] = {};
    const int BH = p->B * p->H, D = P.D, L = P.L;
    // TMA boxes need rows of whole 16-byte pieces, and are not used for rows shorter than a box
    if (D % (16 / (int)sizeof(T)) == 0 && D >= 32 && L > 0) {
        const bool wide = D >= 64 && (long long)BH * cdiv(D, 64) * kMaxCluster >= 3 * tc::num_sms();
        const int ch = wide ? Geo<16>::CH : Geo<8>::CH, tt = wide ? Geo<16>::TT : Geo<8>::TT;
        if (scan_map<T>(&maps[0], P.x, D, L, BH, ch, tt) && scan_map<float>(&maps[1], P.g, D, L, BH, ch, tt) &&
            (!BWD || scan_map<T>(&maps[2], P.dO, D, L, BH, ch, tt)))
            return wide ? launch_walk<T, IN, 16, LOAD_TMA, BWD>(p, P, maps, st)
                        : launch_walk<T, IN, 8, LOAD_TMA, BWD>(p, P, maps, st);
    }
    return D % 4 == 0 ? launch_walk<T, IN, 8, LOAD_VEC4, BWD>(p, P, maps, st)
                      : launch_walk<T, IN, 8, LOAD_ONE, BWD>(p, P, maps, st);
}

cudaError_t fwd(const gla_problem* p, int input, const void* x, const float* g, const float* h0, void* o, float* hT,
                float* saved, cudaStream_t st) {
    const ScanArgs P{x, g, nullptr, h0, o, nullptr, hT, saved, p->L, p->Dk, 0, 0, 0};
    return dispatch(p, input, [&](auto tv, auto in) {
        return walk<decltype(tv), decltype(in)::value, false>(p, P, st);
    });
}

}  // namespace
}  // namespace gla

using namespace gla;

extern "C" {

size_t gla_scan_saved_bytes(const gla_problem* p) {
    if (check(p) != GLA_OK) return 0;
    return 4 * (size_t)p->B * p->H * cdiv(p->L, kSaveEvery) * p->Dk;
}

size_t gla_scan_workspace_bytes(const gla_problem* p, int for_backward) {
    if (check(p) != GLA_OK) return 0;
    return for_backward ? align_up(gla_scan_saved_bytes(p), 256) + 256 : 256;
}

gla_status gla_scan_fwd(const gla_problem* p, int input, const void* x, const float* g, const float* h0, void* o,
                        float* hT, void* ws, size_t ws_bytes, void* stream) {
    return gla_scan_fwd_save(p, input, x, g, h0, o, hT, nullptr, ws, ws_bytes, stream);
}

gla_status gla_scan_fwd_save(const gla_problem* p, int input, const void* x, const float* g, const float* h0, void* o,
                             float* hT, float* saved, void* ws, size_t ws_bytes, void* stream) {
    const gla_status s = check(p);
    if (s != GLA_OK) return s;
    if (!input_ok(input) || !ws) return GLA_ERR_INVALID_ARG;
    const bool empty = (size_t)p->B * p->H * p->L == 0;
    if (!empty && (!x || !g || !o)) return GLA_ERR_INVALID_ARG;
    const void* ptrs[] = {x, g, h0, o, hT, saved, ws};
    for (const void* q : ptrs)
        if (!aligned16(q)) return GLA_ERR_INVALID_ARG;
    if (ws_bytes < gla_scan_workspace_bytes(p, 0)) return GLA_ERR_WORKSPACE;
    if ((size_t)p->B * p->H == 0) return GLA_OK;
    return record_cuda(fwd(p, input, x, g, h0, o, hT, saved, (cudaStream_t)stream), "scan forward");
}

gla_status gla_scan_bwd(const gla_problem* p, int input, const void* x, const float* g, const float* h0,
                        const void* dO, const float* dhT, void* dx, float* dg, float* dh0, void* ws, size_t ws_bytes,
                        void* stream) {
    return gla_scan_bwd_saved(p, input, x, g, h0, dO, dhT, nullptr, dx, dg, dh0, ws, ws_bytes, stream);
}

gla_status gla_scan_bwd_saved(const gla_problem* p, int input, const void* x, const float* g, const float* h0,
                              const void* dO, const float* dhT, const float* saved, void* dx, float* dg, float* dh0,
                              void* ws, size_t ws_bytes, void* stream) {
    const gla_status s = check(p);
    if (s != GLA_OK) return s;
    if (!input_ok(input) || !ws) return GLA_ERR_INVALID_ARG;
    const bool empty = (size_t)p->B * p->H * p->L == 0;
    if (!empty && (!x || !g || !dO || !dx || !dg)) return GLA_ERR_INVALID_ARG;
    const void* ptrs[] = {x, g, h0, dO, dhT, saved, dx, dg, dh0, ws};
    for (const void* q : ptrs)
        if (!aligned16(q)) return GLA_ERR_INVALID_ARG;
    if (ws_bytes < gla_scan_workspace_bytes(p, 1)) return GLA_ERR_WORKSPACE;
    if ((size_t)p->B * p->H == 0) return GLA_OK;
    cudaStream_t st = (cudaStream_t)stream;
    if (!saved) {
        float* own = static_cast<float*>(ws);
        const cudaError_t e = fwd(p, input, x, g, h0, nullptr, nullptr, own, st);
        if (e != cudaSuccess) return record_cuda(e, "scan states");
        saved = own;
    }
    const ScanArgs P{x, g, dO, dhT, dx, dg, dh0, const_cast<float*>(saved), p->L, p->Dk, 0, 0, 0};
    const cudaError_t e = dispatch(p, input, [&](auto tv, auto in) {
        return walk<decltype(tv), decltype(in)::value, true>(p, P, st);
    });
    return record_cuda(e, "scan backward");
}

gla_status gla_scan_decode(const gla_problem* p, int input, const void* x, const float* g, float* state, void* o,
                           void* stream) {
    const gla_status s = check(p);
    if (s != GLA_OK) return s;
    if (!input_ok(input) || p->L != 1) return GLA_ERR_INVALID_ARG;
    const size_t n = (size_t)p->B * p->H * p->Dk;
    if (n == 0) return GLA_OK;
    if (!x || !g || !state || !o) return GLA_ERR_INVALID_ARG;
    const void* ptrs[] = {x, g, state, o};
    for (const void* q : ptrs)
        if (!aligned16(q)) return GLA_ERR_INVALID_ARG;
    cudaStream_t st = (cudaStream_t)stream;
    const cudaError_t e = dispatch(p, input, [&](auto tv, auto in) {
        using T = decltype(tv);
        const size_t blocks = (n + NT_D - 1) / NT_D;
        if (blocks > 2147483647u) return cudaErrorInvalidConfiguration;
        GLA_LAUNCH("scan_decode", st,
                   (k_scan_decode<T, decltype(in)::value><<<(unsigned)blocks, NT_D, 0, st>>>(
                       static_cast<const T*>(x), g, state, static_cast<T*>(o), n)));
        return cudaGetLastError();
    });
    return record_cuda(e, "scan decode");
}

}  // extern "C"
