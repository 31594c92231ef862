// Gated linear recurrence with a vector state (the elementwise member of the family of the GLA
// abstract's data-dependent gates; the talk summary "Hardware-Efficient Training of Linear
// Attention Models", section 7:36, names the scan over states):
//   h_t = a_t h_{t-1} + m(a_t) x_t,  o_t = h_t,  a = e^g,  m = 1 | 1 - a | sqrt(1 - a^2),
// per (b, h, channel). Backward, with D_t = a_t dh_t the gradient handed to h_{t-1}:
//   dh_t = dO_t + D_{t+1},  dx_t = m dh_t,  dg_t = dh_t (a_t h_{t-1} + m'(g_t) x_t),  dh0 = D_0.
//
// A run of tokens maps the state before it to the state after it, h -> A h + B, with A the product
// of its decays and B its end state from zero; runs compose, (A1, B1) then (A2, B2) giving
// (A1 A2, A2 B1 + B2). The kernels use that at three levels: a thread's tokens, a tile's runs (through
// shared memory), and the tiles of a thread-block cluster, which walks the sequence one row of tiles
// at a time and exchanges the tiles' (A, B) through distributed shared memory. So every input is read
// once and the sequence is split over SMs that the channels alone would leave idle. The reverse
// recurrence of the backward composes the same way from the other end with the same A.
//
// Bound by HBM (8 bytes an element forward, 14 backward in bf16) while enough CTAs are resident.
// Measured, device time and share of the copy rate: forward 8 x 16 heads x 2048 x 64 27.5 us (0.75),
// 8 heads x 65536 x 128 102 us (0.80); training pair 4 x 16 x 4096 x 256 289 us (0.78 of both calls' bytes).
#include <type_traits>

#include "gla_common.cuh"
#include "gla_plans.h"
#include "gla_tc_common.cuh"
#include "sm100.cuh"

namespace gla {
namespace {

using namespace sm100;

constexpr int kSaveEvery = 64;   // tokens between two saved states
constexpr int NW = 8;            // warps that hold a tile's tokens
constexpr int VEC = 4;           // channels of a thread, two packed pairs
constexpr int CHL = 8;           // lanes along the channels
constexpr int CH = CHL * VEC;    // channels of a tile: 128-byte rows of g
constexpr int RUN = 4;           // tokens of a thread
constexpr int RW = 32 / CHL;     // runs of a warp
constexpr int WT = RW * RUN;     // tokens of a warp
constexpr int TT = NW * WT;      // tokens of a tile
constexpr int ELEMS = TT * CH;
constexpr int kMaxCluster = 16;  // above 8 only with the attribute for it
constexpr int kFwdStages = 3;    // tiles of the forward's ring

// How a tile reaches shared memory: whole boxes by TMA, or each thread's own four channels by cp.async, in pieces of
// four, two or one channel(s) as D allows. bf16 pieces of one channel (odd D) are narrower than cp.async's
// 4 bytes: plain loads and shared stores.
enum { LOAD_TMA = 0, LOAD_4 = 4, LOAD_2 = 2, LOAD_1 = 1 };

// ------------------------------------------------------------------ packed pairs of fp32
using tc::ex2;
using tc::f2;
using tc::f2_add;
using tc::f2_all;
using tc::f2_fma;
using tc::f2_mul;
using tc::f2_split;
using tc::f2_to_bf2;
__device__ __forceinline__ float rsqrt_approx(float x) {
    float y;
    asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// a = e^g and t = 1 - e^g for two channels. For -0.30 <= g <= 0.05, where a gate's memory is long
// and an error in a is multiplied by 1 / (1 - a), t = -g P(g) with P the degree-4 polynomial closest
// to (e^g - 1) / g there with P(0) = 1 (least largest relative error, 2.2e-8), so t is within 2 and
// a = 1 - t within 1.3 units of 2^-24; elsewhere the hardware exponential serves (2^-22, and |g| 2^-24 from
// the rounding of its argument).
__device__ __forceinline__ void gate2(uint64_t g, uint64_t& a, uint64_t& t) {
    uint64_t s = f2_fma(g, f2_all(-0.007552224211394787f), f2_all(-0.041534192860126495f));
    s = f2_fma(g, s, f2_all(-0.1666625589132309f));
    s = f2_fma(g, s, f2_all(-0.5000003576278687f));
    s = f2_fma(g, s, f2_all(-1.f));
    const uint64_t tn = f2_mul(g, s), an = f2_fma(tn, f2_all(-1.f), f2_all(1.f));
    const uint64_t y = f2_mul(g, f2_all(1.4426950408889634f)), w = f2_add(g, f2_all(0.125f));
    float y0, y1, w0, w1, a0, a1, t0, t1;
    f2_split(y, y0, y1);
    f2_split(w, w0, w1);
    f2_split(an, a0, a1);
    f2_split(tn, t0, t1);
    const float e0 = ex2(y0), e1 = ex2(y1);
    float q0, q1;
    f2_split(f2_fma(f2(e0, e1), f2_all(-1.f), f2_all(1.f)), q0, q1);
    const bool n0 = fabsf(w0) <= 0.175f, n1 = fabsf(w1) <= 0.175f;
    a = f2(n0 ? a0 : e0, n1 ? a1 : e1);
    t = f2(n0 ? t0 : q0, n1 ? t1 : q1);
}

// The factor on the input, from t, and for GLA_SCAN_NORM its inverse (0 where the factor is 0).
// u = 1 - a^2 = t (2 - t), m = u / sqrt(u); u < 0 (g > 0) gives NaN like the formula, u below the normal
// numbers 0.
template <int IN>
__device__ __forceinline__ uint64_t in_factor2(uint64_t t, uint64_t& inv) {
    if (IN == GLA_SCAN_PLAIN) return f2_all(1.f);
    if (IN == GLA_SCAN_COMPLEMENT) return t;
    const uint64_t u = f2_mul(t, f2_fma(t, f2_all(-1.f), f2_all(2.f)));
    float u0, u1;
    f2_split(u, u0, u1);
    inv = f2(fabsf(u0) < 1.1754944e-38f ? 0.f : rsqrt_approx(u0),
             fabsf(u1) < 1.1754944e-38f ? 0.f : rsqrt_approx(u1));
    return f2_mul(u, inv);
}
template <int IN>
__device__ __forceinline__ uint64_t times_factor2(uint64_t m, uint64_t x) {
    return IN == GLA_SCAN_PLAIN ? x : f2_mul(m, x);
}
// The factor's derivative with respect to g (0, -a, -a^2 / m) times x, plus c.
template <int IN>
__device__ __forceinline__ uint64_t slope_fma2(uint64_t a, uint64_t inv, uint64_t x, uint64_t c) {
    if (IN == GLA_SCAN_PLAIN) return c;
    const uint64_t ax = f2_mul(f2_mul(a, f2_all(-1.f)), x);
    return IN == GLA_SCAN_COMPLEMENT ? f2_add(ax, c) : f2_fma(f2_mul(a, inv), ax, c);
}

// ------------------------------------------------------------------ four channels of a token
__device__ __forceinline__ void ld4(const float* p, uint64_t (&v)[2]) {
    const ulonglong2 f = *reinterpret_cast<const ulonglong2*>(p);
    v[0] = f.x;
    v[1] = f.y;
}
__device__ __forceinline__ void ld4(const __nv_bfloat16* p, uint64_t (&v)[2]) {
    const uint2 u = *reinterpret_cast<const uint2*>(p);
    v[0] = f2(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u));
    v[1] = f2(__uint_as_float(u.y << 16), __uint_as_float(u.y & 0xffff0000u));
}
__device__ __forceinline__ void st4(float* p, const uint64_t (&v)[2]) {
    *reinterpret_cast<ulonglong2*>(p) = make_ulonglong2(v[0], v[1]);
}
__device__ __forceinline__ void st4(__nv_bfloat16* p, const uint64_t (&v)[2]) {
    *reinterpret_cast<uint2*>(p) = make_uint2(f2_to_bf2(v[0]), f2_to_bf2(v[1]));
}
// Stores the channels c .. c+3 that exist, in pieces of PIECE (D is a multiple of it; p too is aligned to it).
template <int PIECE>
__device__ __forceinline__ void put4(float* p, const uint64_t (&v)[2], int c, int D) {
    if (PIECE == 4) {
        if (c < D) st4(p, v);
    } else {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            float lo, hi;
            f2_split(v[k], lo, hi);
            if (PIECE == 2) {
                if (c + 2 * k < D) *reinterpret_cast<float2*>(p + 2 * k) = make_float2(lo, hi);
            } else {
                if (c + 2 * k < D) p[2 * k] = lo;
                if (c + 2 * k + 1 < D) p[2 * k + 1] = hi;
            }
        }
    }
}
template <int PIECE>
__device__ __forceinline__ void put4(__nv_bfloat16* p, const uint64_t (&v)[2], int c, int D) {
    if (PIECE == 4) {
        if (c < D) st4(p, v);
    } else {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            if (PIECE == 2) {
                if (c + 2 * k < D) *reinterpret_cast<uint32_t*>(p + 2 * k) = f2_to_bf2(v[k]);
            } else {
                float lo, hi;
                f2_split(v[k], lo, hi);
                if (c + 2 * k < D) p[2 * k] = __float2bfloat16_rn(lo);
                if (c + 2 * k + 1 < D) p[2 * k + 1] = __float2bfloat16_rn(hi);
            }
        }
    }
}
// Loads them the same way, zeros (the identity: a = 1, b = 0) where there are none.
template <int PIECE, typename T>
__device__ __forceinline__ void get4(const T* p, uint64_t (&v)[2], bool row, int c, int D) {
    v[0] = v[1] = 0;
    if (!row) return;
    if (PIECE == 4) {
        if (c < D) ld4(p, v);
    } else {
        float f[VEC];
#pragma unroll
        for (int i = 0; i < VEC; ++i) f[i] = c + i < D ? to_f(p[i]) : 0.f;
        v[0] = f2(f[0], f[1]);
        v[1] = f2(f[2], f[3]);
    }
}
// Copies them to shared memory, asynchronously where a piece has 4 bytes or more; zeros where there are none.
template <int PIECE, typename T>
__device__ __forceinline__ void fetch4(T* dst, const T* src, bool row, int c, int D) {
    constexpr int B = PIECE * (int)sizeof(T);
    if constexpr (B >= 4) {
#pragma unroll
        for (int i = 0; i < VEC; i += PIECE) {
            const int n = row && c + i < D ? B : 0;   // bytes read; the rest is filled with zeros
            if constexpr (B == 16)
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst + i)),
                             "l"(src + (n ? i : 0)), "r"(n)
                             : "memory");
            else
                asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(smem_u32(dst + i)),
                             "l"(src + (n ? i : 0)), "n"(B), "r"(n)
                             : "memory");
        }
    } else {
#pragma unroll
        for (int i = 0; i < VEC; ++i) dst[i] = row && c + i < D ? src[i] : from_f<T>(0.f);
    }
}
__device__ __forceinline__ void fetch_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void fetch_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// A pair into shared memory of a CTA of the cluster, counted on that CTA's barrier.
__device__ __forceinline__ void st_async_pair(uint32_t dst, uint32_t bar, float a, float b) {
    asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v2.f32 [%0], {%1, %2}, [%3];" ::"r"(dst),
                 "f"(a), "f"(b), "r"(bar)
                 : "memory");
}
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

// ------------------------------------------------------------------ waits that may give up
__device__ int scan_status;   // kDevStatus bits of the device's calls since gla_scan_check_device_status last read them

// A thread whose wait gave up waits no more: it runs the walk out, sends nothing to other CTAs, and says so here at the
// end. The threads do not tell each other on the way: looking for that at every wait cost the training pair 4 %.
__device__ __forceinline__ void report(bool ok) {
    if (!ok) atomicOr(&scan_status, kDevStatusTimeout);
}

// Waits for the last copies of a ring that n loads have gone through, one barrier a stage: none may be on its way when
// the CTA's shared memory is given up, whatever the walk came to.
template <int S>
__device__ __forceinline__ void land(uint64_t (&full)[S], int n) {
    for (int i = n < S ? 0 : n - S; i < n; ++i) mbar_wait(&full[i % S], (i / S) & 1);
}

struct ScanArgs {
    const void* x;
    const float* g;
    const void* dO;
    const float* first;    // h0 (forward), dhT (backward); may be null
    void* out;             // o (may be null), dx
    float* dg;
    float* last;           // hT, dh0; may be null
    float* saved;          // written (forward, may be null), read (backward)
    int L, D, nblk, steps;
};

// ------------------------------------------------------------------ products that leave fp32's range
// A composed run multiplies its decays before the state meets them, and their product may be no fp32 number where
// every state is one: e^(g n) over growing gates is infinite, and 0 times it NaN, while the state stays 0; over
// strong gates it is 0, and an infinite state would become NaN. Both show: a state that is not finite stays so to the
// end of a walk. So a walk composes, its end is looked at, and only where that is not finite the tile goes
// again, with the steps that composition cannot take made token by token from the inputs in global memory (the
// ring's stage may be free already). The look costs 1 to 3 %: forward 8 heads x 65536 x 128 102.6 -> 104.6 us, pair
// 4 x 16 x 4096 x 256 292 -> 296. Rows that go again take up to 4 times as long, by tokens (an infinite state under
// strong gates) 60 times.
__device__ __forceinline__ bool is_finite(float v) { return fabsf(v) <= 3.402823466e38f; }
// In any lane: the warp goes again as one, which spares the branch its bookkeeping.
__device__ __forceinline__ bool any_not_finite(float v) { return __any_sync(0xffffffffu, !is_finite(v)); }

// The tokens of one channel of a head: v is x (forward: h <- a h + m x) or dO (REV: d <- a (dO + d)), L rows D apart.
template <bool REV, int IN, typename T>
struct Tokens {
    const float* g;
    const T* v;
    int D, L;
    // What the n tokens from t0 on, (A, B) when composed, make of state h. A NaN stays; growth leaves the state 0.
    __device__ __forceinline__ float step(float A, float B, float h, int t0, int n) const {
        if (h != h) return h;
        if (is_finite(B)) {
            if ((A > 0.f && is_finite(A)) || (A == 0.f && is_finite(h))) return fmaf(A, h, B);
            if (A > 0.f && h == 0.f) return B;
        }
#pragma unroll 1
        for (int j0 = 0; j0 < n && h == h; j0 += RUN) {   // a run's loads together; the identity past L
            float gv[RUN], w[RUN];
#pragma unroll
            for (int j = 0; j < RUN; ++j) {
                const int t = t0 + (REV ? n - 1 - j0 - j : j0 + j);
                gv[j] = t < L ? g[(size_t)t * D] : 0.f;
                w[j] = t < L ? to_f(v[(size_t)t * D]) : 0.f;
            }
#pragma unroll
            for (int j = 0; j < RUN; ++j) {
                uint64_t a, u, inv;
                gate2(f2(gv[j], 0.f), a, u);
                float a0, b0, none;
                f2_split(a, a0, none);
                if (REV) {
                    h = a0 * (w[j] + h);
                } else {
                    f2_split(times_factor2<IN>(in_factor2<IN>(u, inv), f2(w[j], 0.f)), b0, none);
                    h = fmaf(a0, h, b0);
                }
            }
        }
        return h;
    }
};

// Walks N runs of a channel in a tile (A and B of run r lie at r * CH) from run r0, REV: back from r0 + N - 1, with
// state h: put(r, h) gets the state entering run r and may write it over the run's B. Returns the state after the
// runs; kept: the B's, for another walk.
template <bool REV, int N, typename Put>
__device__ __forceinline__ float walk_runs(const float* A, const float* B, int r0, float h, float (&kept)[N], Put put) {
#pragma unroll
    for (int j = 0; j < N; ++j) {
        const int r = REV ? r0 + N - 1 - j : r0 + j;
        kept[j] = B[r * CH];
        put(r, h);
        h = fmaf(A[r * CH], h, kept[j]);
    }
    return h;
}
// Sends (A, B) to every CTA of the cluster, waits for theirs and composes them onto `super` in
// sequence order (reverse order for REV). Returns the value entering this CTA's tile; `super`
// becomes the value leaving the row of tiles. Slots are used in turn, two rows of tiles apart: a
// CTA writes row i + 2 only after it has seen every CTA's row i + 1, which each thread sends after
// it has read its channel of row i.
template <bool REV, typename Tail>
__device__ __forceinline__ float exchange(Tail& sm, int c, float A, float B, int cs, int rank, int i,
                                          float& super, bool& ok) {
    float in = super;
    const int p = i & 1;
    if (c == 0 && ok) mbar_arrive_expect_tx(&sm.got[p], cs * CH * (uint32_t)sizeof(float2));
    for (int r = 0; r < cs && ok; ++r)   // nothing more is sent after a wait that gave up
        st_async_pair(mapa_shared(&sm.slot[(p * cs + rank) * CH + c], r), mapa_shared(&sm.got[p], r), A, B);
    if (ok) ok = mbar_wait_cluster(&sm.got[p], (i >> 1) & 1);
    for (int k = 0; k < cs; ++k) {
        const int r = REV ? cs - 1 - k : k;
        if (r == rank) in = super;
        const float2 v = sm.slot[(p * cs + r) * CH + c];
        super = fmaf(v.x, super, v.y);
    }
    return in;
}
// Puts back what a walk over N runs from r0 replaced.
template <int N>
__device__ __forceinline__ void restore(float* B, int r0, const float (&kept)[N], bool rev) {
#pragma unroll
    for (int j = 0; j < N; ++j) B[(rev ? r0 + N - 1 - j : r0 + j) * CH] = kept[j];
}
// The same once more by Tokens::step: the tiles of the row from its first token on (cs > 1; `super` becomes the value
// leaving the row; else the value leaving the runs), then the N runs from r0 of this CTA's tile. row: the row's first
// token. One loop for both, as code beside the fast path costs it time: with a copy of the step for each the long
// forward takes 108 us instead of 104.5.
template <bool REV, int N, typename Tok, typename Put>
__device__ __forceinline__ void go_again(const float* A, const float* B, const float2* slot, int cs, int rank, int row,
                                         int r0, float& super, const Tok& tok, Put put) {
    float e = super, in = e;
    int k = cs > 1 ? -cs : 0;
#pragma unroll 1
    for (; k < N; ++k) {
        const bool tile = k < 0;
        if (k == 0 && cs > 1) {
            super = e;
            e = in;
        }
        const int r = tile ? (REV ? -1 - k : cs + k) : (REV ? r0 + N - 1 - k : r0 + k);
        if (tile && r == rank) in = e;
        const float a = tile ? slot[r * CH].x : A[r * CH], b = tile ? slot[r * CH].y : B[r * CH];
        if (!tile) put(r, e);
        e = tok.step(a, b, e, tile ? row + r * TT : row + rank * TT + r * RUN, tile ? TT : RUN);
    }
    if (cs == 1) super = e;
}

// Shared memory of the forward behind its ring: the runs' (A, B) of a tile, their start values, the
// barriers, and (clusters only) the exchange slots [2][cs][CH].
constexpr int RUNS = TT / RUN;
constexpr int NT_F = 32 * NW + 64;   // + the warp that composes the runs, + the warp that loads
struct FwdTail {
    float A[RUNS][CH], B[RUNS][CH];
    float start[RUNS][CH];
    uint64_t full[kFwdStages], empty[kFwdStages];
    uint64_t sums, starts;
    uint64_t got[2];
    float2 slot[1];   // as many as the launch asks for
};

// One cluster per (b, h, block of CH channels); its CTAs take the tiles of a row of tiles in
// order and walk the rows together. Three kinds of warps, which meet only at shared-memory barriers:
//   warps 0-7  compose their runs of tile i (keeping a, b in registers), hand (A, B) on, and then
//              walk tile i - 1 from its start values to the outputs;
//   warp 8     lane = channel: composes the runs and, across the cluster, the tiles, and hands the
//              runs' start values back - behind the others' work on the next tile;
//   warp 9     keeps the ring of tiles full.
template <typename T, int IN, int LOAD>
__global__ void __launch_bounds__(NT_F, 2)
    k_scan_fwd(const __grid_constant__ CUtensorMap mx, const __grid_constant__ CUtensorMap mg, const ScanArgs P,
               int cs) {
    extern __shared__ __align__(128) uint8_t smem[];
    constexpr int kStage = ELEMS * (4 + (int)sizeof(T));
    constexpr int PIECE = LOAD == LOAD_TMA ? 4 : LOAD;
    FwdTail& sm = *reinterpret_cast<FwdTail*>(smem + kFwdStages * kStage);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rank = cs > 1 ? (int)cluster_rank() : 0;
    const unsigned chain = blockIdx.x / cs;
    const size_t bh = chain / P.nblk;
    const int c0 = (int)(chain % P.nblk) * CH;
    const int L = P.L, D = P.D;
    bool ok = true;   // false once a wait gave up: no further wait, the results are not valid

    if (tid == 0) {
        for (int s = 0; s < kFwdStages; ++s) {
            mbar_init(&sm.full[s], 1);
            mbar_init(&sm.empty[s], NW);
        }
        mbar_init(&sm.sums, NW);
        mbar_init(&sm.starts, 1);
        mbar_init(&sm.got[0], 1);
        mbar_init(&sm.got[1], 1);
        mbar_fence_init();
    }
    if (cs > 1) cluster_sync();
    else __syncthreads();

    if (warp < NW) {
        const int run = warp * RW + lane / CHL, ch = (lane % CHL) * VEC;
        const int tr = run * RUN;   // this thread's first token in a tile
        const T* xg = static_cast<const T*>(P.x) + bh * L * D + c0 + ch;
        const float* gg = P.g + bh * L * D + c0 + ch;
        T* og = static_cast<T*>(P.out) + bh * L * D + c0 + ch;

        auto fetch = [&](int i) {   // this thread's part of tile i, without TMA
            if (i < P.steps) {
                const int s = i % kFwdStages, t = (i * cs + rank) * TT + tr;
                float* sg = reinterpret_cast<float*>(smem + s * kStage) + tr * CH + ch;
                T* sx = reinterpret_cast<T*>(smem + s * kStage + ELEMS * 4) + tr * CH + ch;
#pragma unroll
                for (int j = 0; j < RUN; ++j) {
                    const size_t at = (size_t)(t + j) * D;
                    const bool row = t + j < L && c0 + ch < D;
                    fetch4<PIECE>(sg + j * CH, row ? gg + at : P.g, row, c0 + ch, D);
                    fetch4<PIECE>(sx + j * CH, row ? xg + at : static_cast<const T*>(P.x), row, c0 + ch, D);
                }
            }
            fetch_commit();
        };
        if (LOAD != LOAD_TMA)
            for (int i = 0; i + 1 < kFwdStages; ++i) fetch(i);
        auto compose = [&](int i, uint64_t (&a)[RUN][2], uint64_t (&b)[RUN][2], uint64_t (&A)[2], uint64_t (&B)[2]) {
            const int s = i % kFwdStages;
            const float* sg = reinterpret_cast<const float*>(smem + s * kStage) + tr * CH + ch;
            const T* sx = reinterpret_cast<const T*>(smem + s * kStage + ELEMS * 4) + tr * CH + ch;
            if (LOAD == LOAD_TMA) {
                if (ok) ok = mbar_wait(&sm.full[s], (i / kFwdStages) & 1);
            } else {
                fetch_wait<kFwdStages - 2>();
            }
            uint64_t gv[RUN][2], xv[RUN][2];
#pragma unroll
            for (int j = 0; j < RUN; ++j) {
                ld4(sg + j * CH, gv[j]);
                ld4(sx + j * CH, xv[j]);
            }
            if (LOAD == LOAD_TMA) {
                __syncwarp();
                if (lane == 0) mbar_arrive(&sm.empty[s]);
            } else {
                fetch(i + kFwdStages - 1);   // into the stage of tile i - 1, which this thread has read
            }
#pragma unroll
            for (int j = 0; j < RUN; ++j)
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    uint64_t u, inv;
                    gate2(gv[j][k], a[j][k], u);
                    b[j][k] = times_factor2<IN>(in_factor2<IN>(u, inv), xv[j][k]);
                    A[k] = j ? f2_mul(A[k], a[j][k]) : a[j][k];
                    B[k] = j ? f2_fma(a[j][k], B[k], b[j][k]) : b[j][k];
                }
        };
        auto hand_on = [&](const uint64_t (&A)[2], const uint64_t (&B)[2]) {
            st4(&sm.A[run][ch], A);
            st4(&sm.B[run][ch], B);
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm.sums);
        };
        auto take_start = [&](int i, uint64_t (&h)[2]) {
            if (ok) ok = mbar_wait(&sm.starts, i & 1);
            ld4(&sm.start[run][ch], h);
        };
        auto finish = [&](int i, uint64_t (&h)[2], const uint64_t (&a)[RUN][2], const uint64_t (&b)[RUN][2]) {
            if (!P.out) return;
            const int t = (i * cs + rank) * TT + tr;
#pragma unroll
            for (int j = 0; j < RUN; ++j) {
#pragma unroll
                for (int k = 0; k < 2; ++k) h[k] = f2_fma(a[j][k], h[k], b[j][k]);
                if (t + j < L) put4<PIECE>(og + (size_t)(t + j) * D, h, c0 + ch, D);
            }
        };
        // The runs' sums and start values have one buffer each: (A, B) of tile i are written after the
        // start values of tile i - 1 are there (so its sums have been read) and have been read.
        uint64_t a0[RUN][2], b0[RUN][2], a1[RUN][2], b1[RUN][2], A[2], B[2], h[2];
        if (P.steps > 0) {
            compose(0, a0, b0, A, B);
            hand_on(A, B);
        }
        for (int i = 1; i <= P.steps; i += 2) {
            if (i < P.steps) compose(i, a1, b1, A, B);
            take_start(i - 1, h);
            if (i < P.steps) hand_on(A, B);
            finish(i - 1, h, a0, b0);
            if (i == P.steps) break;
            if (i + 1 < P.steps) compose(i + 1, a0, b0, A, B);
            take_start(i, h);
            if (i + 1 < P.steps) hand_on(A, B);
            finish(i, h, a1, b1);
        }
    } else if (warp == NW) {
        const bool live = c0 + lane < D;
        // read for live channels only: the others' states are 0
        const size_t at = bh * L * D + c0 + lane;
        const Tokens<false, IN, T> tok{P.g + at, static_cast<const T*>(P.x) + at, D, L};
        float super = P.first && live ? P.first[bh * D + c0 + lane] : 0.f;
        for (int i = 0; i < P.steps; ++i) {
            const int t0 = (i * cs + rank) * TT;
            if (ok) ok = mbar_wait(&sm.sums, i & 1);
            const float before = super;
            float in = super;
            if (cs > 1) {
                float tA = 1.f, tB = 0.f;
#pragma unroll
                for (int r = 0; r < RUNS; ++r) {
                    const float ra = sm.A[r][lane];
                    tB = fmaf(ra, tB, sm.B[r][lane]);
                    tA *= ra;
                }
                in = exchange<false>(sm, lane, tA, tB, cs, rank, i, super, ok);
            }
            auto put = [&](int r, float v) {
                sm.start[r][lane] = v;
                const int t = t0 + r * RUN;
                if (r * RUN % kSaveEvery == 0 && P.saved && t < L && live)
                    P.saved[(bh * cdiv(L, kSaveEvery) + t / kSaveEvery) * D + c0 + lane] = v;
            };
            float kept[RUNS];
            float h = walk_runs<false>(&sm.A[0][lane], &sm.B[0][lane], 0, in, kept, put);
            if (cs == 1) super = h;
            if (any_not_finite(super)) {
                super = before;
                go_again<false, RUNS>(&sm.A[0][lane], &sm.B[0][lane], &sm.slot[(i & 1) * cs * CH + lane], cs, rank,
                                      i * cs * TT, 0, super, tok, put);
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm.starts);
        }
        if (P.last && rank == 0 && live) P.last[bh * D + c0 + lane] = super;
    } else if (LOAD == LOAD_TMA && lane == 0) {
        int i = 0;
        for (; i < P.steps; ++i) {
            const int s = i % kFwdStages, t0 = (i * cs + rank) * TT;
            float* sg = reinterpret_cast<float*>(smem + s * kStage);
            if (i >= kFwdStages && !(ok = mbar_wait(&sm.empty[s], (i / kFwdStages - 1) & 1))) break;
            mbar_arrive_expect_tx(&sm.full[s], kStage);
            tma_load_3d(sg, &mg, c0, t0, (int)bh, &sm.full[s]);
            tma_load_3d(sg + ELEMS, &mx, c0, t0, (int)bh, &sm.full[s]);
        }
        land(sm.full, i);
    }
    report(ok);
    __syncwarp();
    if (cs > 1) cluster_sync();   // no CTA leaves while another may still write to its slots
}

// Shared memory of the backward behind its ring. The composing warp replaces a run's B and R by the
// state and the gradient that enter the run (from its first and last token).
template <int STAGES>
struct BwdTail {
    float A[RUNS][CH], B[RUNS][CH], R[RUNS][CH];
    uint64_t full[STAGES], empty[STAGES];
    uint64_t sums, starts;
    uint64_t got[2];
    float2 slot[1];
};
// Tiles of the ring: two CTAs share an SM's 227 KB. Without TMA a thread refills its part of a stage itself,
// after the walk of the tile before last: three tiles, so that one is always on its way.
template <typename T, int LOAD>
constexpr int bwd_stages() { return sizeof(T) == 2 || LOAD != LOAD_TMA ? 3 : 2; }

// The same walk from the sequence's end, by the same three kinds of warps. The states are
// recomputed inside each tile from the saved ones of every 64 tokens. A tile stays in the ring until
// its gradients are out: the walk to the gradients reads it again and forms the gates anew, which
// costs less than the registers that would keep them (the ring is then free for the tile after next).
template <typename T, int IN, int LOAD>
__global__ void __launch_bounds__(NT_F, 2)
    k_scan_bwd(const __grid_constant__ CUtensorMap mx, const __grid_constant__ CUtensorMap mg,
               const __grid_constant__ CUtensorMap md, const ScanArgs P, int cs) {
    extern __shared__ __align__(128) uint8_t smem[];
    constexpr int kStage = ELEMS * (4 + 2 * (int)sizeof(T)), S = bwd_stages<T, LOAD>();
    constexpr int PIECE = LOAD == LOAD_TMA ? 4 : LOAD;
    BwdTail<S>& sm = *reinterpret_cast<BwdTail<S>*>(smem + S * kStage);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rank = cs > 1 ? (int)cluster_rank() : 0;
    const unsigned chain = blockIdx.x / cs;
    const size_t bh = chain / P.nblk;
    const int c0 = (int)(chain % P.nblk) * CH;
    const int L = P.L, D = P.D;
    bool ok = true;
    // rows are counted from the end: row i holds the tiles (steps - 1 - i) cs + rank
    auto first_token = [&](int i) { return ((P.steps - 1 - i) * cs + rank) * TT; };

    if (tid == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(&sm.full[s], 1);
            mbar_init(&sm.empty[s], NW);
        }
        mbar_init(&sm.sums, NW);
        mbar_init(&sm.starts, 1);
        mbar_init(&sm.got[0], 1);
        mbar_init(&sm.got[1], 1);
        mbar_fence_init();
    }
    if (cs > 1) cluster_sync();
    else __syncthreads();

    if (warp < NW) {
        const int run = warp * RW + lane / CHL, ch = (lane % CHL) * VEC;
        const int tr = run * RUN;
        const size_t base = bh * L * D + c0 + ch;
        const T *xg = static_cast<const T*>(P.x) + base, *dg = static_cast<const T*>(P.dO) + base;
        const float* gg = P.g + base;
        T* xo = static_cast<T*>(P.out) + base;
        float* go = P.dg + base;

        // token j of this thread's run in stage s
        auto sg = [&](int s, int j) { return reinterpret_cast<float*>(smem + s * kStage) + (tr + j) * CH + ch; };
        auto sx = [&](int s, int j) {
            return reinterpret_cast<T*>(smem + s * kStage + ELEMS * 4) + (tr + j) * CH + ch;
        };
        auto sd = [&](int s, int j) { return sx(s, j) + ELEMS; };
        auto fetch = [&](int i) {   // this thread's part of row i's tile, without TMA
            if (i < P.steps) {
                const int s = i % S, t = first_token(i) + tr;
#pragma unroll
                for (int j = 0; j < RUN; ++j) {
                    const size_t at = (size_t)(t + j) * D;
                    const bool row = t + j < L && c0 + ch < D;
                    fetch4<PIECE>(sg(s, j), row ? gg + at : P.g, row, c0 + ch, D);
                    fetch4<PIECE>(sx(s, j), row ? xg + at : static_cast<const T*>(P.x), row, c0 + ch, D);
                    fetch4<PIECE>(sd(s, j), row ? dg + at : static_cast<const T*>(P.dO), row, c0 + ch, D);
                }
            }
            fetch_commit();
        };
        if (LOAD != LOAD_TMA) fetch(0);
        auto compose = [&](int i, uint64_t (&A)[2], uint64_t (&B)[2], uint64_t (&R)[2]) {
            const int s = i % S;
            if (LOAD == LOAD_TMA) {
                if (ok) ok = mbar_wait(&sm.full[s], (i / S) & 1);
            } else {
                fetch(i + 1);   // into the stage of row i - 2
                fetch_wait<1>();
            }
            uint64_t a[RUN][2];
#pragma unroll
            for (int j = 0; j < RUN; ++j) {
                uint64_t gv[2], xv[2], u, inv;
                ld4(sg(s, j), gv);
                ld4(sx(s, j), xv);
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    gate2(gv[k], a[j][k], u);
                    const uint64_t b = times_factor2<IN>(in_factor2<IN>(u, inv), xv[k]);
                    A[k] = j ? f2_mul(A[k], a[j][k]) : a[j][k];
                    B[k] = j ? f2_fma(a[j][k], B[k], b) : b;
                }
            }
#pragma unroll
            for (int j = RUN - 1; j >= 0; --j) {
                uint64_t dv[2];
                ld4(sd(s, j), dv);
#pragma unroll
                for (int k = 0; k < 2; ++k) R[k] = f2_mul(a[j][k], j == RUN - 1 ? dv[k] : f2_add(dv[k], R[k]));
            }
        };
        auto hand_on = [&](const uint64_t (&A)[2], const uint64_t (&B)[2], const uint64_t (&R)[2]) {
            st4(&sm.A[run][ch], A);
            st4(&sm.B[run][ch], B);
            st4(&sm.R[run][ch], R);
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm.sums);
        };
        auto finish = [&](int i, uint64_t (&h)[2], uint64_t (&d)[2]) {
            const int s = i % S, t = first_token(i) + tr;
            uint64_t a[RUN][2], m[RUN][2], hp[RUN][2];
#pragma unroll
            for (int j = 0; j < RUN; ++j) {
                uint64_t gv[2], xv[2], u, inv;
                ld4(sg(s, j), gv);
                ld4(sx(s, j), xv);
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    gate2(gv[k], a[j][k], u);
                    m[j][k] = in_factor2<IN>(u, inv);
                    // a h_{t-1} + m' x, dg's factor next to dh
                    const uint64_t ah = f2_mul(a[j][k], h[k]);
                    hp[j][k] = slope_fma2<IN>(a[j][k], inv, xv[k], ah);
                    h[k] = f2_add(times_factor2<IN>(m[j][k], xv[k]), ah);
                }
            }
#pragma unroll
            for (int j = RUN - 1; j >= 0; --j) {
                uint64_t dv[2], ox[2], og[2];
                ld4(sd(s, j), dv);
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const uint64_t dh = f2_add(dv[k], d[k]);
                    ox[k] = times_factor2<IN>(m[j][k], dh);
                    og[k] = f2_mul(hp[j][k], dh);
                    d[k] = f2_mul(a[j][k], dh);
                }
                if (t + j < L) {
                    put4<PIECE>(xo + (size_t)(t + j) * D, ox, c0 + ch, D);
                    put4<PIECE>(go + (size_t)(t + j) * D, og, c0 + ch, D);
                }
            }
            if (LOAD == LOAD_TMA) {
                __syncwarp();
                if (lane == 0) mbar_arrive(&sm.empty[s]);
            }
        };
        uint64_t A[2], B[2], R[2], h[2], d[2];
        for (int i = 0; i <= P.steps; ++i) {
            if (i < P.steps) compose(i, A, B, R);
            if (i > 0) {
                if (ok) ok = mbar_wait(&sm.starts, (i - 1) & 1);
                ld4(&sm.B[run][ch], h);
                ld4(&sm.R[run][ch], d);
            }
            if (i < P.steps) hand_on(A, B, R);
            if (i > 0) finish(i - 1, h, d);
        }
    } else if (warp == NW) {
        const bool live = c0 + lane < D;
        const size_t ns = cdiv(L, kSaveEvery);
        constexpr int NS = TT / kSaveEvery;   // saved states of a tile
        static_assert(NS == 2, "");
        const size_t at = bh * L * D + c0 + lane;
        const Tokens<true, IN, T> back{P.g + at, static_cast<const T*>(P.dO) + at, D, L};
        const Tokens<false, IN, T> tok{P.g + at, static_cast<const T*>(P.x) + at, D, L};
        float super = P.first && live ? P.first[bh * D + c0 + lane] : 0.f;
        for (int i = 0; i < P.steps; ++i) {
            const int t0 = first_token(i);
            float sv[NS];
#pragma unroll
            for (int n = 0; n < NS; ++n) {
                const int t = t0 + n * kSaveEvery;
                sv[n] = t < L && live ? P.saved[(bh * ns + t / kSaveEvery) * D + c0 + lane] : 0.f;
            }
            if (ok) ok = mbar_wait(&sm.sums, i & 1);
            const float before = super;
            float in = super;
            if (cs > 1) {
                float tA = 1.f, tR = 0.f;
#pragma unroll
                for (int r = RUNS - 1; r >= 0; --r) {
                    const float ra = sm.A[r][lane];
                    tR = fmaf(ra, tR, sm.R[r][lane]);
                    tA *= ra;
                }
                in = exchange<true>(sm, lane, tA, tR, cs, rank, i, super, ok);
            }
            {
                auto put = [&](int r, float v) { sm.R[r][lane] = v; };
                float kept[RUNS];
                float d = walk_runs<true>(&sm.A[0][lane], &sm.R[0][lane], 0, in, kept, put);
                if (cs == 1) super = d;
                if (any_not_finite(super)) {
                    super = before;
                    restore(&sm.R[0][lane], 0, kept, true);
                    go_again<true, RUNS>(&sm.A[0][lane], &sm.R[0][lane], &sm.slot[(i & 1) * cs * CH + lane], cs, rank,
                                         t0 - rank * TT, 0, super, back, put);
                }
            }
            constexpr int N = RUNS / NS;
            auto put = [&](int r, float v) { sm.B[r][lane] = v; };
            float kept[NS][N];
            bool finite = true;
#pragma unroll
            for (int n = 0; n < NS; ++n) {
                float h = walk_runs<false>(&sm.A[0][lane], &sm.B[0][lane], n * N, sv[n], kept[n], put);
                finite = finite && is_finite(h);
            }
            if (__any_sync(0xffffffffu, !finite)) {
#pragma unroll
                for (int n = 0; n < NS; ++n) restore(&sm.B[0][lane], n * N, kept[n], false);
#pragma unroll 1
                for (int n = 0; n < NS; ++n) {
                    float h = n ? sv[NS - 1] : sv[0];   // NS is 2
                    go_again<false, N>(&sm.A[0][lane], &sm.B[0][lane], nullptr, 1, 0, t0, n * N, h, tok, put);
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm.starts);
        }
        if (P.last && rank == 0 && live) P.last[bh * D + c0 + lane] = super;
    } else if (LOAD == LOAD_TMA && lane == 0) {
        int i = 0;
        for (; i < P.steps; ++i) {
            const int s = i % S, t0 = first_token(i);
            float* sg = reinterpret_cast<float*>(smem + s * kStage);
            T* sx = reinterpret_cast<T*>(sg + ELEMS);
            if (i >= S && !(ok = mbar_wait(&sm.empty[s], (i / S - 1) & 1))) break;
            mbar_arrive_expect_tx(&sm.full[s], kStage);
            tma_load_3d(sg, &mg, c0, t0, (int)bh, &sm.full[s]);
            tma_load_3d(sx, &mx, c0, t0, (int)bh, &sm.full[s]);
            tma_load_3d(sx + ELEMS, &md, c0, t0, (int)bh, &sm.full[s]);
        }
        land(sm.full, i);
    }
    report(ok);
    __syncwarp();
    if (cs > 1) cluster_sync();
}

// Short sequences: a tile would be mostly empty, and its warps' hand-overs cost more than the walk itself. One
// thread walks four channels, kBatch tokens' loads at a time.
constexpr int NT_W = 64;
constexpr int kBatch = 8;
template <typename T, int IN, int PIECE>
__global__ void __launch_bounds__(NT_W) k_scan_fwd_short(const ScanArgs P) {
    const int c = (blockIdx.y * NT_W + threadIdx.x) * VEC;
    const int L = P.L, D = P.D;
    if (c >= D) return;
    const size_t bh = blockIdx.x, end = bh * D + c;
    const T* x = static_cast<const T*>(P.x) + bh * L * D + c;
    const float* g = P.g + bh * L * D + c;
    T* o = static_cast<T*>(P.out) + bh * L * D + c;
    uint64_t h[2] = {0, 0};
    if (P.first) get4<PIECE>(P.first + end, h, true, c, D);
    for (int t0 = 0; t0 < L; t0 += kBatch) {
        if (P.saved && t0 % kSaveEvery == 0)
            put4<PIECE>(P.saved + (bh * cdiv(L, kSaveEvery) + t0 / kSaveEvery) * D + c, h, c, D);
        uint64_t gv[kBatch][2], xv[kBatch][2];
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            get4<PIECE>(g + (size_t)(t0 + j) * D, gv[j], t0 + j < L, c, D);
            get4<PIECE>(x + (size_t)(t0 + j) * D, xv[j], t0 + j < L, c, D);
        }
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                uint64_t a, u, inv;
                gate2(gv[j][k], a, u);
                h[k] = f2_fma(a, h[k], times_factor2<IN>(in_factor2<IN>(u, inv), xv[j][k]));   // the identity past L
            }
            if (P.out && t0 + j < L) put4<PIECE>(o + (size_t)(t0 + j) * D, h, c, D);
        }
    }
    if (P.last) put4<PIECE>(P.last + end, h, c, D);
}
// The states h_{t-1} of the forward walk wait in dg, where the same thread's reverse walk replaces them.
template <typename T, int IN, int PIECE>
__global__ void __launch_bounds__(NT_W) k_scan_bwd_short(const ScanArgs P) {
    const int c = (blockIdx.y * NT_W + threadIdx.x) * VEC;
    const int L = P.L, D = P.D;
    if (c >= D) return;
    const size_t bh = blockIdx.x, end = bh * D + c, base = bh * L * D + c;
    const T *x = static_cast<const T*>(P.x) + base, *dO = static_cast<const T*>(P.dO) + base;
    const float* g = P.g + base;
    T* dx = static_cast<T*>(P.out) + base;
    float* dg = P.dg + base;
    uint64_t h[2] = {0, 0}, d[2] = {0, 0};
    if (L > 0) get4<PIECE>(P.saved + bh * cdiv(L, kSaveEvery) * D + c, h, true, c, D);
    for (int t0 = 0; t0 < L; t0 += kBatch) {
        uint64_t gv[kBatch][2], xv[kBatch][2];
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            get4<PIECE>(g + (size_t)(t0 + j) * D, gv[j], t0 + j < L, c, D);
            get4<PIECE>(x + (size_t)(t0 + j) * D, xv[j], t0 + j < L, c, D);
        }
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            if (t0 + j < L) put4<PIECE>(dg + (size_t)(t0 + j) * D, h, c, D);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                uint64_t a, u, inv;
                gate2(gv[j][k], a, u);
                h[k] = f2_fma(a, h[k], times_factor2<IN>(in_factor2<IN>(u, inv), xv[j][k]));
            }
        }
    }
    if (P.first) get4<PIECE>(P.first + end, d, true, c, D);
    for (int t0 = (L - 1) / kBatch * kBatch; L > 0 && t0 >= 0; t0 -= kBatch) {
        uint64_t gv[kBatch][2], xv[kBatch][2], dv[kBatch][2], hv[kBatch][2];
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            const size_t at = (size_t)(t0 + j) * D;
            get4<PIECE>(g + at, gv[j], t0 + j < L, c, D);
            get4<PIECE>(x + at, xv[j], t0 + j < L, c, D);
            get4<PIECE>(dO + at, dv[j], t0 + j < L, c, D);
            get4<PIECE>(dg + at, hv[j], t0 + j < L, c, D);
        }
#pragma unroll
        for (int j = kBatch - 1; j >= 0; --j) {
            uint64_t ox[2], og[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                uint64_t a, u, inv;
                gate2(gv[j][k], a, u);
                const uint64_t m = in_factor2<IN>(u, inv), dh = f2_add(dv[j][k], d[k]);
                ox[k] = times_factor2<IN>(m, dh);
                og[k] = f2_mul(slope_fma2<IN>(a, inv, xv[j][k], f2_mul(a, hv[j][k])), dh);
                d[k] = f2_mul(a, dh);   // unchanged past L: a = 1, dO = 0
            }
            if (t0 + j < L) {
                put4<PIECE>(dx + (size_t)(t0 + j) * D, ox, c, D);
                put4<PIECE>(dg + (size_t)(t0 + j) * D, og, c, D);
            }
        }
    }
    if (P.last) put4<PIECE>(P.last + end, d, c, D);
}

// One token: the state is read and written once. Four channels a thread; the last threads take single
// ones.
constexpr int NT_D = 128;
template <typename T, int IN>
__global__ void __launch_bounds__(NT_D) k_scan_decode(const T* __restrict__ x, const float* __restrict__ g,
                                                      float* __restrict__ state, T* __restrict__ o, size_t n) {
    const size_t i = ((size_t)blockIdx.x * NT_D + threadIdx.x) * VEC;
    if (i >= n) return;
    uint64_t xv[2], gv[2], h[2];
    const bool whole = i + VEC <= n;
    if (whole) {
        ld4(x + i, xv);
        ld4(g + i, gv);
        ld4(state + i, h);
    } else {
        get4<1>(x + i, xv, true, 0, (int)(n - i));
        get4<1>(g + i, gv, true, 0, (int)(n - i));
        get4<1>(state + i, h, true, 0, (int)(n - i));
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        uint64_t a, t, inv;
        gate2(gv[k], a, t);
        h[k] = f2_fma(a, h[k], times_factor2<IN>(in_factor2<IN>(t, inv), xv[k]));
    }
    if (whole) {
        st4(state + i, h);
        st4(o + i, h);
    } else {
        put4<1>(state + i, h, 0, (int)(n - i));
        put4<1>(o + i, h, 0, (int)(n - i));
    }
}

// Waits that nothing completes, one of each kind, which give up after `polls` polls.
__global__ void __launch_bounds__(64) k_scan_wait_timeout(uint32_t polls) {
    __shared__ __align__(8) uint64_t bar;
    if (threadIdx.x == 0) {
        mbar_init(&bar, 1);
        mbar_fence_init();
    }
    __syncthreads();
    bool ok = true;
    if (threadIdx.x == 0) ok = mbar_wait(&bar, 0, polls);
    if (threadIdx.x == 32) ok = mbar_wait_cluster(&bar, 0, polls);
    report(ok);
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
    // at most 2^27 chains; B * H first, as the product of all three may pass 64 bits
    const long long bh = (long long)p->B * p->H;
    if (bh > 1 << 27 || bh * cdiv(p->Dk, CH) > 1 << 27) return GLA_ERR_UNSUPPORTED;
    return GLA_OK;
}
bool input_ok(int input) { return input >= GLA_SCAN_PLAIN && input <= GLA_SCAN_NORM; }

// 3D map over [BH][L][D] with a box of TT tokens x CH channels.
template <typename T>
bool scan_map(CUtensorMap* m, const void* base, int D, int L, int BH) {
    auto fn = tc::encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)L, (cuuint64_t)BH};
    const cuuint64_t strides[2] = {(cuuint64_t)D * sizeof(T), (cuuint64_t)D * sizeof(T) * L};
    const cuuint32_t box[3] = {CH, TT, 1}, estr[3] = {1, 1, 1};
    return fn(m, std::is_same<T, float>::value ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3,
              const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// CTAs that the current device holds at once in clusters of `cs`, asked of the runtime once per kernel and
// device (a cluster stays within a GPC, so not every SM is filled by every size).
template <typename K>
int resident_ctas(K kern, cudaLaunchConfig_t cfg, int cs, size_t smem, std::atomic<int> (&known)[kMaxCluster + 1]) {
    int n = known[cs].load(std::memory_order_relaxed);
    if (n) return n;
    cfg.attrs[0].val.clusterDim.x = cs;
    cfg.gridDim = dim3(cs);
    cfg.dynamicSmemBytes = smem;
    int clusters = 0;
    if (cudaOccupancyMaxActiveClusters(&clusters, kern, &cfg) != cudaSuccess) {
        cudaGetLastError();
        clusters = 0;
    }
    n = clusters > 0 ? clusters * cs : -1;
    known[cs].store(n, std::memory_order_relaxed);
    return n;
}

// Launches a walk. CTAs per cluster: the split with the least time in a model of equal waves, each as many rows of
// tiles as a CTA walks plus kFill for filling and draining its pipeline. Measured (forward, us): 256
// chains of 16 tiles 26 / 36 / 43 / 56 in clusters of 1 / 2 / 4 / 8; 32 chains of 512 tiles 387 / 291 /
// 149 / 99.
template <typename T, int IN, int LOAD, bool BWD>
cudaError_t launch_walk(const gla_problem* p, ScanArgs P, const CUtensorMap (&maps)[3], cudaStream_t st) {
    constexpr int kFill = 4;
    P.nblk = cdiv(P.D, CH);
    const long long chains = (long long)p->B * p->H * P.nblk;
    const int tiles = cdiv(P.L, TT);
    constexpr int kStage = ELEMS * (4 + (BWD ? 2 : 1) * (int)sizeof(T));
    constexpr size_t ring = (size_t)kStage * (BWD ? bwd_stages<T, LOAD>() : kFwdStages);
    constexpr size_t tail = BWD ? sizeof(BwdTail<bwd_stages<T, LOAD>()>) : sizeof(FwdTail);
    auto smem = [&](int c) { return ring + tail + (c > 1 ? 2 * CH * sizeof(float2) * c : 0); };
    auto kern = [] {
        if constexpr (BWD) return k_scan_bwd<T, IN, LOAD>;
        else return k_scan_fwd<T, IN, LOAD>;
    }();
    static std::atomic<bool> seen[kMaxDevices];
    static std::atomic<int> known[kMaxDevices][kMaxCluster + 1];
    cudaError_t e = smem_attr_once(kern, smem(kMaxCluster), seen);
    if (e != cudaSuccess) return e;
    int dev = 0;
    if ((e = cudaGetDevice(&dev)) != cudaSuccess) return e;
    if (known[dev][1].load(std::memory_order_relaxed) == 0 &&
        (e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1)) != cudaSuccess)
        return e;
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(NT_F);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int cs = 1;
    long long best = -1;
    for (int c = 1; c <= kMaxCluster && (c == 1 || c <= tiles); ++c) {
        const int slots = resident_ctas(kern, cfg, c, smem(c), known[dev]);
        if (slots <= 0) continue;
        const long long cost = (chains * c + slots - 1) / slots * (cdiv(tiles, c) + kFill);
        if (best < 0 || cost < best) best = cost, cs = c;
    }
    P.steps = cdiv(tiles, cs);
    attr[0].val.clusterDim.x = cs;
    cfg.gridDim = dim3((unsigned)(chains * cs));
    cfg.dynamicSmemBytes = smem(cs);
    if constexpr (BWD)
        GLA_LAUNCH("scan_bwd", st, (e = cudaLaunchKernelEx(&cfg, kern, maps[0], maps[1], maps[2], P, cs)));
    else
        GLA_LAUNCH("scan_fwd", st, (e = cudaLaunchKernelEx(&cfg, kern, maps[0], maps[1], P, cs)));
    return e;
}

template <typename T, int IN, int PIECE, bool BWD>
cudaError_t launch_short(const gla_problem* p, const ScanArgs& P, cudaStream_t st) {
    const dim3 grid((unsigned)(p->B * p->H), cdiv(P.D, NT_W * VEC));
    if constexpr (BWD)
        GLA_LAUNCH("scan_bwd_short", st, (k_scan_bwd_short<T, IN, PIECE><<<grid, NT_W, 0, st>>>(P)));
    else
        GLA_LAUNCH("scan_fwd_short", st, (k_scan_fwd_short<T, IN, PIECE><<<grid, NT_W, 0, st>>>(P)));
    return cudaGetLastError();
}

// Whether threads walk sequences alone: up to 64 tokens, when their batches of loads (about 1.6 us each, forward) cost
// less than the waves of CTAs of mostly empty tiles (about 3 us each, two CTAs an SM). Measured, us forward /
// training pair, alone and by tiles: 1 x 4 heads x 64, 8 tokens 1.9 / 6.1 and 2.7 / 6.8, 32 tokens 4.8 / 15 and
// 3.0 / 6.7; 64 x 4096 channels, 32 tokens 20 / 68 and 77 / 182, 128 tokens 79 / 330 and 88 / 225.
bool is_short(const gla_problem* p) {
    const long long chains = (long long)p->B * p->H * cdiv(p->Dk, CH), at_once = 2 * tc::num_sms();
    return p->L <= 64 && cdiv(p->L, kBatch) < 2 * ((chains + at_once - 1) / at_once);
}

template <typename T, int IN, bool BWD>
cudaError_t walk(const gla_problem* p, const ScanArgs& P, cudaStream_t st) {
    CUtensorMap maps[3] = {};
    const int BH = p->B * p->H, D = P.D, L = P.L;
    if (is_short(p))
        return D % 4 == 0   ? launch_short<T, IN, 4, BWD>(p, P, st)
               : D % 2 == 0 ? launch_short<T, IN, 2, BWD>(p, P, st)
                            : launch_short<T, IN, 1, BWD>(p, P, st);
    // TMA boxes need rows of whole 16-byte pieces, and are not used for rows shorter than a box
    if (D % (16 / (int)sizeof(T)) == 0 && D >= CH && scan_map<T>(&maps[0], P.x, D, L, BH) &&
        scan_map<float>(&maps[1], P.g, D, L, BH) && (!BWD || scan_map<T>(&maps[2], P.dO, D, L, BH)))
        return launch_walk<T, IN, LOAD_TMA, BWD>(p, P, maps, st);
    return D % 4 == 0   ? launch_walk<T, IN, LOAD_4, BWD>(p, P, maps, st)
           : D % 2 == 0 ? launch_walk<T, IN, LOAD_2, BWD>(p, P, maps, st)
                        : launch_walk<T, IN, LOAD_1, BWD>(p, P, maps, st);
}

cudaError_t fwd(const gla_problem* p, int input, const void* x, const float* g, const float* h0, void* o, float* hT,
                float* saved, cudaStream_t st) {
    const ScanArgs P{x, g, nullptr, h0, o, nullptr, hT, saved, p->L, p->Dk, 0, 0};
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

size_t gla_scan_bwd_workspace_bytes(const gla_problem* p) {
    if (check(p) != GLA_OK) return 0;
    return align_up(gla_scan_saved_bytes(p), 256) + 256;
}

gla_status gla_scan_fwd(const gla_problem* p, int input, const void* x, const float* g, const float* h0, void* o,
                        float* hT, void* stream) {
    return gla_scan_fwd_save(p, input, x, g, h0, o, hT, nullptr, stream);
}

gla_status gla_scan_fwd_save(const gla_problem* p, int input, const void* x, const float* g, const float* h0, void* o,
                             float* hT, float* saved, void* stream) {
    const gla_status s = check(p);
    if (s != GLA_OK) return s;
    if (!input_ok(input)) return GLA_ERR_INVALID_ARG;
    const bool empty = (size_t)p->B * p->H * p->L == 0;
    if (!empty && (!x || !g || !o)) return GLA_ERR_INVALID_ARG;
    const void* ptrs[] = {x, g, h0, o, hT, saved};
    for (const void* q : ptrs)
        if (!aligned16(q)) return GLA_ERR_INVALID_ARG;
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
    // no states are needed, saved or recomputed, where there are no tokens: an empty buffer's address may be null
    const bool recompute = !saved && gla_scan_saved_bytes(p) > 0;
    if (!input_ok(input) || (recompute && !ws)) return GLA_ERR_INVALID_ARG;
    const bool empty = (size_t)p->B * p->H * p->L == 0;
    if (!empty && (!x || !g || !dO || !dx || !dg)) return GLA_ERR_INVALID_ARG;
    const void* ptrs[] = {x, g, h0, dO, dhT, saved, dx, dg, dh0, ws};
    for (const void* q : ptrs)
        if (!aligned16(q)) return GLA_ERR_INVALID_ARG;
    if (recompute && ws_bytes < gla_scan_bwd_workspace_bytes(p)) return GLA_ERR_WORKSPACE;
    if ((size_t)p->B * p->H == 0) return GLA_OK;
    cudaStream_t st = (cudaStream_t)stream;
    if (recompute) {
        float* own = static_cast<float*>(ws);
        const cudaError_t e = fwd(p, input, x, g, h0, nullptr, nullptr, own, st);
        if (e != cudaSuccess) return record_cuda(e, "scan states");
        saved = own;
    }
    const ScanArgs P{x, g, dO, dhT, dx, dg, dh0, const_cast<float*>(saved), p->L, p->Dk, 0, 0};
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
        const size_t blocks = (n + NT_D * VEC - 1) / (NT_D * VEC);
        if (blocks > 2147483647u) return cudaErrorInvalidConfiguration;
        GLA_LAUNCH("scan_decode", st,
                   (k_scan_decode<T, decltype(in)::value><<<(unsigned)blocks, NT_D, 0, st>>>(
                       static_cast<const T*>(x), g, state, static_cast<T*>(o), n)));
        return cudaGetLastError();
    });
    return record_cuda(e, "scan decode");
}

gla_status gla_scan_check_device_status(void* stream) {
    cudaStream_t st = (cudaStream_t)stream;
    int word = 0;
    cudaError_t e = cudaMemcpyFromSymbolAsync(&word, scan_status, sizeof(int), 0, cudaMemcpyDeviceToHost, st);
    if (e == cudaSuccess) e = cudaStreamSynchronize(st);
    if (e == cudaSuccess && word != kDevStatusOk) {
        const int none = kDevStatusOk;
        e = cudaMemcpyToSymbolAsync(scan_status, &none, sizeof(int), 0, cudaMemcpyHostToDevice, st);
        if (e == cudaSuccess) e = cudaStreamSynchronize(st);
    }
    if (e != cudaSuccess) return record_cuda(e, "scan status");
    return word == kDevStatusOk ? GLA_OK : GLA_ERR_TIMEOUT;
}

gla_status gla_debug_scan_wait_timeout(unsigned polls, void* stream) {
    if (polls == 0 || polls > kWaitPolls) return GLA_ERR_INVALID_ARG;
    cudaStream_t st = (cudaStream_t)stream;
    GLA_LAUNCH("debug_scan_wait_timeout", st, (k_scan_wait_timeout<<<1, 64, 0, st>>>(polls)));
    return record_cuda(cudaGetLastError(), "scan wait-timeout kernel launch");
}

}  // extern "C"
