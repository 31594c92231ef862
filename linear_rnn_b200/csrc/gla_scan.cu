// Gated linear recurrence with a vector state (the elementwise member of the family of the GLA
// abstract's data-dependent gates; the talk summary "Hardware-Efficient Training of Linear
// Attention Models", section 7:36, names the scan over states):
//   h_t = a_t h_{t-1} + m(a_t) x_t,  o_t = h_t,  a = e^g,  m = 1 | 1 - a | sqrt(1 - a^2),
// per (b, h, channel). Backward, with D_t = a_t dh_t the gradient handed to h_{t-1}:
//   dh_t = dO_t + D_{t+1},  dx_t = m dh_t,  dg_t = dh_t (a_t h_{t-1} + m'(g_t) x_t),  dh0 = D_0.
#include <type_traits>

#include "gla_common.cuh"

namespace gla {
namespace {

constexpr int kSaveEvery = 64;   // tokens between two saved states
constexpr int NT_S = 128;

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

// The factor on the input and its derivative with respect to g.
template <int IN>
__device__ __forceinline__ float in_factor(float t) {
    if (IN == GLA_SCAN_PLAIN) return 1.f;
    if (IN == GLA_SCAN_COMPLEMENT) return t;
    return sqrtf(t * (2.f - t));   // 1 - a^2 = (1 - a)(1 + a)
}
template <int IN>
__device__ __forceinline__ float in_slope(float a, float m) {
    if (IN == GLA_SCAN_PLAIN) return 0.f;
    if (IN == GLA_SCAN_COMPLEMENT) return -a;
    return m == 0.f ? 0.f : -a * a / m;
}

// One thread per channel walks the tokens.
template <typename T, int IN>
__global__ void __launch_bounds__(NT_S) k_scan_fwd(const T* __restrict__ x, const float* __restrict__ g,
                                                   const float* __restrict__ h0, T* __restrict__ o,
                                                   float* __restrict__ hT, float* __restrict__ saved, int L, int D) {
    const int d = blockIdx.y * NT_S + threadIdx.x;
    if (d >= D) return;
    const size_t bh = blockIdx.x, row = bh * D + d;
    const size_t base = bh * L * D + d;
    const int ns = cdiv(L, kSaveEvery);
    float h = h0 ? h0[row] : 0.f;
    for (int t = 0; t < L; ++t) {
        if (saved && t % kSaveEvery == 0) saved[(bh * ns + t / kSaveEvery) * D + d] = h;
        float a, u;
        gate(g[base + (size_t)t * D], a, u);
        h = fmaf(a, h, in_factor<IN>(u) * to_f(x[base + (size_t)t * D]));
        if (o) o[base + (size_t)t * D] = from_f<T>(h);
    }
    if (hT) hT[row] = h;
}

template <typename T, int IN>
__global__ void __launch_bounds__(NT_S) k_scan_bwd(const T* __restrict__ x, const float* __restrict__ g,
                                                   const T* __restrict__ dO, const float* __restrict__ dhT,
                                                   const float* __restrict__ saved, T* __restrict__ dx,
                                                   float* __restrict__ dg, float* __restrict__ dh0, int L, int D) {
    __shared__ float hs[kSaveEvery][NT_S];
    const int d = blockIdx.y * NT_S + threadIdx.x;
    if (d >= D) return;
    const size_t bh = blockIdx.x, row = bh * D + d;
    const size_t base = bh * L * D + d;
    const int ns = cdiv(L, kSaveEvery);
    float carry = dhT ? dhT[row] : 0.f;
    for (int s = ns - 1; s >= 0; --s) {
        const int t0 = s * kSaveEvery, n = min(kSaveEvery, L - t0);
        float h = saved[(bh * ns + s) * D + d];
        for (int i = 0; i < n; ++i) {
            hs[i][threadIdx.x] = h;
            float a, u;
            gate(g[base + (size_t)(t0 + i) * D], a, u);
            h = fmaf(a, h, in_factor<IN>(u) * to_f(x[base + (size_t)(t0 + i) * D]));
        }
        for (int i = n - 1; i >= 0; --i) {
            const size_t at = base + (size_t)(t0 + i) * D;
            float a, u;
            gate(g[at], a, u);
            const float m = in_factor<IN>(u), xv = to_f(x[at]);
            const float dh = carry + to_f(dO[at]);
            dx[at] = from_f<T>(m * dh);
            dg[at] = dh * fmaf(a, hs[i][threadIdx.x], in_slope<IN>(a, m) * xv);
            carry = a * dh;
        }
    }
    if (dh0) dh0[row] = carry;
}

template <typename T, int IN>
__global__ void __launch_bounds__(NT_S) k_scan_decode(const T* __restrict__ x, const float* __restrict__ g,
                                                      float* __restrict__ state, T* __restrict__ o, size_t n) {
    const size_t i = (size_t)blockIdx.x * NT_S + threadIdx.x;
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
    if (p->Dk > 65536 || (long long)p->B * p->H > 1 << 24) return GLA_ERR_UNSUPPORTED;
    return GLA_OK;
}
bool input_ok(int input) { return input >= GLA_SCAN_PLAIN && input <= GLA_SCAN_NORM; }

cudaError_t fwd(const gla_problem* p, int input, const void* x, const float* g, const float* h0, void* o, float* hT,
                float* saved, cudaStream_t st) {
    return dispatch(p, input, [&](auto tv, auto in) {
        using T = decltype(tv);
        dim3 grid(p->B * p->H, cdiv(p->Dk, NT_S));
        GLA_LAUNCH("scan_fwd", st,
                   (k_scan_fwd<T, decltype(in)::value><<<grid, NT_S, 0, st>>>(
                       static_cast<const T*>(x), g, h0, static_cast<T*>(o), hT, saved, p->L, p->Dk)));
        return cudaGetLastError();
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
    const cudaError_t e = dispatch(p, input, [&](auto tv, auto in) {
        using T = decltype(tv);
        dim3 grid(p->B * p->H, cdiv(p->Dk, NT_S));
        GLA_LAUNCH("scan_bwd", st,
                   (k_scan_bwd<T, decltype(in)::value><<<grid, NT_S, 0, st>>>(
                       static_cast<const T*>(x), g, static_cast<const T*>(dO), dhT, saved, static_cast<T*>(dx), dg,
                       dh0, p->L, p->Dk)));
        return cudaGetLastError();
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
        const size_t blocks = (n + NT_S - 1) / NT_S;
        if (blocks > 2147483647u) return cudaErrorInvalidConfiguration;
        GLA_LAUNCH("scan_decode", st,
                   (k_scan_decode<T, decltype(in)::value><<<(unsigned)blocks, NT_S, 0, st>>>(
                       static_cast<const T*>(x), g, state, static_cast<T*>(o), n)));
        return cudaGetLastError();
    });
    return record_cuda(e, "scan decode");
}

}  // extern "C"
