// What the norms around a block share (gla_addnorm.cu, gla_headnorm.cu):
//   norm(r) = n = (r - mu) rstd,  rstd = 1 / sqrt(mean((r - mu)^2) + eps);  mu = 0 for the RMS norm.
// Gradient of a norm, d the gradient of n:  dr = rstd (d - n mean(d n) - [layer] mean(d)); with
// mean(d n) = rstd mean(d (r - mu)) it needs one set of row sums for the RMS norm and two for the layer
// norm (mu, then the sums about it).
//
// The kernels are bound by HBM, and next by instruction issue (a bf16 element has 6 to 14 bytes of
// traffic to hide 25 to 50 instructions behind). So a row is read once and held by the G threads that
// share it, 16 elements a thread, so that the row sums' exchange is spread over many elements;
// arithmetic is on packed pairs of fp32; several sums share their shuffles; and every thread copies its
// own pieces of the next rows into shared memory asynchronously (a ring that only its own thread
// reads, so no barrier guards it; odd rows share theirs). Rows of up to 512 elements belong to a warp or less, longer ones to a
// block. Blocks walk many rows and keep the column sums (dw) in registers.
// Measured, device time and share of the copy rate: addnorm forward 16384 x 4096 (fp32 residual) 134 us
// (0.92), backward 16384 x 2048 in bf16 layer norm 80 us (0.77), RMS 73 us (0.84); headnorm forward
// 4 x 16 x 4096 x 256 69 us (0.89), backward 2 x 8 x 8192 x 256 68 us (0.75).
#pragma once
#include <type_traits>

#include "gla_common.cuh"
#include "gla_plans.h"
#include "gla_tc_common.cuh"
#include "sm100.cuh"

namespace gla {
namespace norm {

using namespace sm100;
using tc::f2;
using tc::f2_add;
using tc::f2_all;
using tc::f2_fma;
using tc::f2_mul;
using tc::f2_split;
using tc::f2_to_bf2;

__device__ __forceinline__ float f2_sum(uint64_t v) {
    float a, b;
    f2_split(v, a, b);
    return a + b;
}

// ------------------------------------------------------------------ pieces of a row
// A piece: VEC elements, held as NP pairs (VEC = 1: one pair whose second half is 0).
template <int VEC>
constexpr int kPairs = VEC == 1 ? 1 : VEC / 2;

template <int VEC>
__device__ __forceinline__ void load_piece(const float* p, uint64_t (&v)[kPairs<VEC>]) {
    if constexpr (VEC == 1) {
        v[0] = f2(*p, 0.f);
    } else if constexpr (VEC == 2) {
        v[0] = *reinterpret_cast<const uint64_t*>(p);
    } else {
#pragma unroll
        for (int i = 0; i < VEC / 4; ++i) {
            const ulonglong2 u = *reinterpret_cast<const ulonglong2*>(p + 4 * i);
            v[2 * i] = u.x;
            v[2 * i + 1] = u.y;
        }
    }
}
template <int VEC>
__device__ __forceinline__ void load_piece(const __nv_bfloat16* p, uint64_t (&v)[kPairs<VEC>]) {
    if constexpr (VEC == 1) {
        v[0] = f2(__bfloat162float(*p), 0.f);
    } else {
        uint32_t w[VEC / 2];
        if constexpr (VEC == 2) {
            w[0] = *reinterpret_cast<const uint32_t*>(p);
        } else if constexpr (VEC == 8) {
            const uint4 u = *reinterpret_cast<const uint4*>(p);
            w[0] = u.x; w[1] = u.y; w[2] = u.z; w[3] = u.w;
        } else {
            const uint2 u = *reinterpret_cast<const uint2*>(p);
            w[0] = u.x; w[1] = u.y;
        }
#pragma unroll
        for (int i = 0; i < VEC / 2; ++i) v[i] = f2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
    }
}
template <int VEC>
__device__ __forceinline__ void store_piece(float* p, const uint64_t (&v)[kPairs<VEC>]) {
    if constexpr (VEC == 1) {
        float a, b;
        f2_split(v[0], a, b);
        *p = a;
    } else if constexpr (VEC == 2) {
        *reinterpret_cast<uint64_t*>(p) = v[0];
    } else {
#pragma unroll
        for (int i = 0; i < VEC / 4; ++i)
            *reinterpret_cast<ulonglong2*>(p + 4 * i) = make_ulonglong2(v[2 * i], v[2 * i + 1]);
    }
}
template <int VEC>
__device__ __forceinline__ void store_piece(__nv_bfloat16* p, const uint64_t (&v)[kPairs<VEC>]) {
    if constexpr (VEC == 1) {
        float a, b;
        f2_split(v[0], a, b);
        *p = __float2bfloat16_rn(a);
    } else if constexpr (VEC == 2) {
        *reinterpret_cast<uint32_t*>(p) = f2_to_bf2(v[0]);
    } else if constexpr (VEC == 8) {
        *reinterpret_cast<uint4*>(p) =
            make_uint4(f2_to_bf2(v[0]), f2_to_bf2(v[1]), f2_to_bf2(v[2]), f2_to_bf2(v[3]));
    } else {
        *reinterpret_cast<uint2*>(p) = make_uint2(f2_to_bf2(v[0]), f2_to_bf2(v[1]));
    }
}

// Where a thread's pieces of a row are. The last piece of an odd row has one column of its pair.
struct Place {
    int at, G, nvec, D;
    __device__ __forceinline__ bool has(int j) const { return at + j * G < nvec; }
    template <int VEC>
    __device__ __forceinline__ int col(int j) const { return (at + j * G) * VEC; }
    __device__ __forceinline__ bool half(int j) const { return 2 * (at + j * G) + 1 == D; }
};

// Pairs of an odd row: no alignment beyond the element's, and the second column may be missing.
__device__ __forceinline__ void store_pair(float* p, uint64_t v, bool half) {
    float a, b;
    f2_split(v, a, b);
    p[0] = a;
    if (!half) p[1] = b;
}
__device__ __forceinline__ void store_pair(__nv_bfloat16* p, uint64_t v, bool half) {
    const uint32_t w = f2_to_bf2(v);
    if (!half && (reinterpret_cast<uintptr_t>(p) & 2) == 0) {
        *reinterpret_cast<uint32_t*>(p) = w;
        return;
    }
    const __nv_bfloat162 h = *reinterpret_cast<const __nv_bfloat162*>(&w);
    p[0] = h.x;
    if (!half) p[1] = h.y;
}
// Piece j of the row at `row` (element 0 of it).
template <int VEC, bool ODD, typename T>
__device__ __forceinline__ void put_piece(T* row, const Place& P, int j, const uint64_t (&v)[kPairs<VEC>]) {
    if constexpr (ODD) store_pair(row + P.col<VEC>(j), v[0], P.half(j));
    else store_piece<VEC>(row + P.col<VEC>(j), v);
}

// ------------------------------------------------------------------ the ring
// Elements of a row that a thread of an odd row's group holds, and the room of such a row in shared memory, in
// elements: it starts up to 14 bytes into its first 16-byte unit, and its last pair's word may be read beyond it.
constexpr int kRowElems = 16;
__host__ __device__ constexpr int odd_room(int G) { return kRowElems * G + 16; }

// S stages of shared memory that belong to the thread alone. Piece j of an input is a unit of 4, 8 or 16 bytes, blockDim
// units of that size apart from the next piece, so that a warp's accesses are contiguous.
// Stages are written by cp.async, one commit group per row; wait() leaves the groups of the S - 1 rows that
// follow in flight.
template <int S>
struct Feed {
    uint8_t* mine;      // first stage, 16 bytes per thread on
    int stage_bytes;
    int s;              // stage of the current row

    // Room of one input's NV pieces, in bytes per thread.
    template <typename T, int VEC, int NV>
    static constexpr int bytes() { return VEC * (int)sizeof(T) * NV; }

    template <typename T, int VEC>
    __device__ __forceinline__ uint8_t* at(int stage, int thread_off, int j) const {
        constexpr int B = VEC * (int)sizeof(T);
        uint8_t* d = mine + stage * stage_bytes + (thread_off + j * B) * (int)blockDim.x;
        return d - (16 - B) * (int)threadIdx.x;   // `mine` is 16 bytes a thread on
    }
    template <typename T, int VEC>
    __device__ __forceinline__ void copy(int stage, int thread_off, int j, const T* src) const {
        constexpr int B = VEC * (int)sizeof(T);
        uint8_t* d = at<T, VEC>(stage, thread_off, j);
        if constexpr (B == 16) {
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(d)), "l"(src) : "memory");
        } else {
            static_assert(B == 4 || B == 8, "");
            asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(smem_u32(d)), "l"(src), "n"(B) : "memory");
        }
    }
    template <typename T, int VEC>
    __device__ __forceinline__ void read(int thread_off, int j, uint64_t (&v)[kPairs<VEC>], size_t,
                                         const Place&) const {   // the row's place matters to a RowFeed only
        load_piece<VEC>(reinterpret_cast<const T*>(at<T, VEC>(s, thread_off, j)), v);
    }
    __device__ __forceinline__ void commit() const { asm volatile("cp.async.commit_group;" ::: "memory"); }
    __device__ __forceinline__ void wait() const {
        asm volatile("cp.async.wait_group %0;" ::"n"(S > 2 ? S - 2 : 0) : "memory");
    }
    __device__ __forceinline__ int ahead() const { return s == 0 ? S - 1 : s - 1; }   // stage of the row S - 1 ahead
    __device__ __forceinline__ void next() { s = s + 1 == S ? 0 : s + 1; }
};

// The ring for odd rows with bf16 in them, where no copy of 4 bytes or more fits a thread's own columns: the group
// copies the 16-byte units that the row touches, wherever in them it starts, and reads each other's, so a
// row costs a barrier of the group's threads (wait()). Pieces are pairs; a pair that straddles two words is
// joined from both. 16384 x 1001 in bf16, backward: 100 us; with loads of single elements 233.
template <int S>
struct RowFeed {
    uint8_t* mine;      // the group's first stage
    int stage_bytes, pad, G, s;   // pad: room of a row, in elements

    __device__ __forceinline__ RowFeed(uint8_t* ring, int thread_bytes, int G_)
        : pad(odd_room(G_)), G(G_), s(0) {
        const int row = thread_bytes / kRowElems * pad;
        stage_bytes = row * ((int)blockDim.x / G);
        mine = ring + (int)threadIdx.x / G * row;
    }
    template <typename T, int VEC, int NV>
    static constexpr int bytes() { return VEC * (int)sizeof(T) * NV; }

    // This thread's share of the row that starts at element e0 of an input of n elements in all.
    template <typename T>
    __device__ __forceinline__ void copy_row(int stage, int thread_off, const T* src, size_t e0, size_t n,
                                             const Place& P) const {
        constexpr size_t B = sizeof(T);
        const size_t from = e0 * B & ~(size_t)15, to = (e0 + P.D) * B, all = n * B;
        const uint32_t d = smem_u32(mine + stage * stage_bytes + thread_off / kRowElems * pad);
        for (int c = 16 * P.at; from + c < to; c += 16 * G) {
            const int m = all - (from + c) < 16 ? (int)(all - (from + c)) : 16;   // the rest is filled with zeros
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(d + c),
                         "l"(reinterpret_cast<const uint8_t*>(src) + from + c), "r"(m)
                         : "memory");
        }
    }
    template <typename T, int VEC>
    __device__ __forceinline__ void read(int thread_off, int j, uint64_t (&v)[kPairs<VEC>], size_t e0,
                                         const Place& P) const {
        const int at = ((int)(e0 * sizeof(T)) & 15) + P.col<VEC>(j) * (int)sizeof(T);
        const uint8_t* d = mine + s * stage_bytes + thread_off / kRowElems * pad;
        if constexpr (sizeof(T) == 4) {
            const float* f = reinterpret_cast<const float*>(d + at);
            const float b = f[1];
            v[0] = f2(f[0], P.half(j) ? 0.f : b);
        } else {
            const uint32_t* w = reinterpret_cast<const uint32_t*>(d + (at & ~3));
            uint32_t u = w[0];
            if (at & 2) u = __funnelshift_r(u, w[1], 16);
            v[0] = f2(__uint_as_float(u << 16), P.half(j) ? 0.f : __uint_as_float(u & 0xffff0000u));
        }
    }
    __device__ __forceinline__ void commit() const { asm volatile("cp.async.commit_group;" ::: "memory"); }
    // Waits for the row of stage s, and until the group has read the stage before it.
    __device__ __forceinline__ void wait() const {
        asm volatile("cp.async.wait_group %0;" ::"n"(S > 2 ? S - 2 : 0) : "memory");
        if (G > 32) __syncthreads();
        else __syncwarp();
    }
    __device__ __forceinline__ int ahead() const { return s == 0 ? S - 1 : s - 1; }
    __device__ __forceinline__ void next() { s = s + 1 == S ? 0 : s + 1; }
};
template <int S, bool ODD>
__device__ __forceinline__ auto make_feed(uint8_t* ring, int thread_bytes, int G) {
    if constexpr (ODD) return RowFeed<S>(ring, thread_bytes, G);
    else return Feed<S>{ring + 16 * threadIdx.x, thread_bytes * (int)blockDim.x, 0};
}

// ------------------------------------------------------------------ sums over a row
// Sums of K <= 4 values over the G threads of a row; every thread of the block calls. G < 32: plain
// shuffles (G a power of two). From a warp up, K values share their shuffles: each exchange halves either the
// lanes or the values a lane still carries. G > 32: the block is one row; a warp's sums go through
// `buf`, which alternates between two halves so that one barrier per call is enough.
struct RowSum {
    float* buf;   // [2][32 warps][4]
    int G, half;

    template <int K>
    __device__ __forceinline__ void operator()(float (&v)[K]) {
        static_assert(K >= 1 && K <= 4, "");
        const int lane = threadIdx.x & 31;
        if (G < 32) {
            for (int off = G >> 1; off; off >>= 1)
#pragma unroll
                for (int k = 0; k < K; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], off);
            return;
        }
        // after this, lanes of index 32 / KP * k .. hold the warp's sum k in x
        constexpr int KP = K == 1 ? 1 : K == 2 ? 2 : 4;
        float x;
        if constexpr (KP == 1) {
            x = v[0] + __shfl_xor_sync(0xffffffffu, v[0], 16);
            x += __shfl_xor_sync(0xffffffffu, x, 8);
        } else if constexpr (KP == 2) {
            const bool hi = lane & 16;
            x = (hi ? v[1] : v[0]) + __shfl_xor_sync(0xffffffffu, hi ? v[0] : v[1], 16);
            x += __shfl_xor_sync(0xffffffffu, x, 8);
        } else {
            const float v3 = K == 4 ? v[K - 1] : 0.f;
            const bool hi = lane & 16, mid = lane & 8;
            const float a = (hi ? v[2] : v[0]) + __shfl_xor_sync(0xffffffffu, hi ? v[0] : v[2], 16);
            const float b = (hi ? v3 : v[1]) + __shfl_xor_sync(0xffffffffu, hi ? v[1] : v3, 16);
            x = (mid ? b : a) + __shfl_xor_sync(0xffffffffu, mid ? a : b, 8);
        }
        x += __shfl_xor_sync(0xffffffffu, x, 4);
        x += __shfl_xor_sync(0xffffffffu, x, 2);
        x += __shfl_xor_sync(0xffffffffu, x, 1);
        constexpr int W = 32 / KP;
        if (G == 32) {
#pragma unroll
            for (int k = 0; k < K; ++k) v[k] = __shfl_sync(0xffffffffu, x, W * k);
            return;
        }
        float* b = buf + half * 128;
        half ^= 1;
        const int warp = threadIdx.x >> 5, nw = G >> 5;
        if ((lane & (W - 1)) == 0) b[warp * 4 + lane / W] = x;
        __syncthreads();
        // lane = 4 warp + k: adds the warps 8 apart, then over the lanes of one k
        x = 0.f;
        for (int w = lane >> 2; w < nw; w += 8)
            if ((lane & 3) < K) x += b[w * 4 + (lane & 3)];
        x += __shfl_xor_sync(0xffffffffu, x, 4);
        x += __shfl_xor_sync(0xffffffffu, x, 8);
        x += __shfl_xor_sync(0xffffffffu, x, 16);
#pragma unroll
        for (int k = 0; k < K; ++k) v[k] = __shfl_sync(0xffffffffu, x, k);
    }
};

// r -= mean(r) for the layer norm (elements beyond the row stay 0).
template <int KIND, int VEC, int NV, bool ODD>
__device__ __forceinline__ void center(RowSum& sum, uint64_t (&r)[NV][kPairs<VEC>], const Place& P, float inv_d) {
    if (KIND != GLA_NORM_LAYER) return;
    uint64_t t = 0;
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < kPairs<VEC>; ++i) t = f2_add(t, r[j][i]);
    float s[1] = {f2_sum(t)};
    sum(s);
    const float mu = -s[0] * inv_d;
    const uint64_t m2 = VEC == 1 ? f2(mu, 0.f) : f2_all(mu);
#pragma unroll
    for (int j = 0; j < NV; ++j)
        if (P.has(j))
#pragma unroll
            for (int i = 0; i < kPairs<VEC>; ++i) r[j][i] = f2_add(r[j][i], ODD && P.half(j) ? f2(mu, 0.f) : m2);
}

template <int VEC, int NV>
__device__ __forceinline__ float square_sum(const uint64_t (&r)[NV][kPairs<VEC>]) {
    uint64_t t = 0;
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < kPairs<VEC>; ++i) t = f2_fma(r[j][i], r[j][i], t);
    return f2_sum(t);
}

// This thread's columns of a weight vector times c (null: c).
template <int VEC, int NV, bool ODD>
__device__ __forceinline__ void load_columns(uint64_t (&v)[NV][kPairs<VEC>], const float* p, const Place& P, float c) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
#pragma unroll
        for (int i = 0; i < kPairs<VEC>; ++i) v[j][i] = f2_all(1.f);
        if (p && P.has(j)) {
            const float* c0 = p + P.col<VEC>(j);
            if constexpr (ODD) v[j][0] = f2(c0[0], P.half(j) ? 1.f : c0[1]);
            else load_piece<VEC>(c0, v[j]);
        }
#pragma unroll
        for (int i = 0; i < kPairs<VEC>; ++i) v[j][i] = f2_mul(v[j][i], f2_all(c));
    }
}

// Sums a column accumulator over the row groups of a block and writes the block's partial row.
// smem: blockDim * NV * VEC floats where the block has several rows.
template <int VEC, int NV, bool ODD>
__device__ __forceinline__ void write_partial(const uint64_t (&acc)[NV][kPairs<VEC>], float* smem, int grp,
                                              const Place& P, float* out) {
    const int D = P.D, ngrp = P.G >= 32 && P.G == (int)blockDim.x ? 1 : blockDim.x / P.G;
    if (ngrp == 1) {
#pragma unroll
        for (int j = 0; j < NV; ++j)
            if (P.has(j)) put_piece<VEC, ODD>(out, P, j, acc[j]);
        return;
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < NV; ++j)
        if (P.has(j))
#pragma unroll
            for (int i = 0; i < kPairs<VEC>; ++i) {
                float a, b;
                f2_split(acc[j][i], a, b);
                smem[grp * D + P.col<VEC>(j) + 2 * i] = a;
                if (VEC > 1 && !(ODD && P.half(j))) smem[grp * D + P.col<VEC>(j) + 2 * i + 1] = b;
            }
    __syncthreads();
    for (int c = threadIdx.x; c < D; c += blockDim.x) {
        float s = 0.f;
        for (int k = 0; k < ngrp; ++k) s += smem[k * D + c];
        out[c] = s;
    }
}

// ------------------------------------------------------------------ partial rows -> dw
// out[c] = sum over i < n of part[i * stride + c]: 32 columns per block, 32 rows at a time. blockIdx.y
// picks one of two sums.
static __global__ void __launch_bounds__(1024) k_colsum(const float* __restrict__ part0, float* __restrict__ out0,
                                                        const float* __restrict__ part1, float* __restrict__ out1,
                                                        int n, size_t stride, int cols) {
    __shared__ float red[32][33];
    const float* part = blockIdx.y ? part1 : part0;
    float* out = blockIdx.y ? out1 : out0;
    grid_dep_wait();   // launched while the kernel that writes the partial rows drains
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
// One or two column sums (out1 may be null).
inline cudaError_t colsum(const float* part0, float* out0, const float* part1, float* out1, int n, size_t stride,
                          int cols, cudaStream_t st) {
    if (!out0) {
        part0 = part1, out0 = out1;
        out1 = nullptr;
    }
    if (!out0) return cudaSuccess;
    cudaError_t e;
    GLA_LAUNCH("norm_colsum", st,
               (e = tc::launch_ex(k_colsum, dim3(cdiv(cols, 32), out1 ? 2 : 1), dim3(32, 32), 0, st, n > 0, 1, part0,
                                      out0, part1, out1, n, stride, cols)));
    return e;
}

// ------------------------------------------------------------------ host side
// Threads and pieces of a row. A piece is 16 bytes of the widest type in the row (8 bf16, or 4 where
// fp32 stands beside them: with 8 the fp32 accesses of a warp would leave every other 16 bytes out,
// 305 instead of 212 us for the backward of 16384 x 4096 with an fp32 residual), 4 elements where D is no
// multiple of 8, then 2, then 1; pairs in an odd row (RowFeed) with bf16, up to 512 threads, and in
// one of fp32 beyond 2048 elements while two stages fit (16384 x 3001, backward: 310 us, 1706 with single
// elements). A thread holds 16 elements, so that the row sums' exchange and the addresses of a row are spread
// over many; with narrower pieces 4 of them while 512 threads do. A row has a power of two of lanes up to a warp,
// whole warps beyond.
struct RowPlan {
    int vec, nv, G, threads;
    bool ring;   // pieces of 4 bytes or more in every operand, or rows of a RowFeed; at most 512 threads (kWide)
    bool odd;    // of a RowFeed
    bool all_f32;
};
// wide_rows: 8 elements a thread for 4096 < D <= 6144, where 16 would leave an SM one block of 9 to 12 warps, their
// registers too many for two. addnorm backward, 16384 x 5120 in bf16: 240 us, 287 with 16 elements (layer norm); the
// forward, of fewer registers, loses (16384 x 6144 with an fp32 residual: 219, and 196 with 16).
constexpr int kWide = 768;
inline RowPlan row_plan(int D, bool all_bf16, bool all_f32, bool wide_rows = false) {
    RowPlan p;
    p.vec = all_bf16 && D % 8 == 0 ? 8 : D % 4 == 0 ? 4 : D % 2 == 0 ? 2 : 1;
    p.all_f32 = all_f32;
    p.odd = D % 2 == 1 && (all_f32 ? D > 2048 && D <= 416 * kRowElems : D <= 512 * kRowElems);
    if (p.odd) p.vec = 2;
    const int nvec = cdiv(D, p.vec);
    const bool wide = wide_rows && p.vec >= 4 && D > 4096 && D <= 8 * kWide;
    p.nv = p.odd ? kRowElems / 2 : wide ? 8 / p.vec : p.vec < 4 && nvec <= 2048 ? 4 : 16 / p.vec;
    const int need = cdiv(nvec, p.nv);
    if (need > 32) {
        p.G = cdiv(need, 32) * 32;
        p.threads = p.G;
    } else {
        for (p.G = 1; p.G < need;) p.G *= 2;
        p.threads = 256;
    }
    p.ring = p.odd || p.threads <= (wide ? kWide : 512) && !(p.vec == 1 && p.nv > 4);
    return p;
}
// Shared memory in front of the ring: the row sums' buffer; it and the ring are free again when the column
// sums of a block's row groups need their blockDim * 16 floats at most.
constexpr int kHead = 1024;
constexpr int kSmSmem = 220 * 1024;    // of an SM, for its blocks
inline int stage_bytes(const RowPlan& p, int thread_bytes) {
    return p.odd ? thread_bytes / kRowElems * odd_room(p.G) * (p.threads / p.G) : thread_bytes * p.threads;
}
// Stages of the ring: 3 or 2, or none where 2 do not fit. fp32 alone: 3 where two blocks of them fit an SM. With bf16 in
// the row the arithmetic wants 14 warps: 3 where they have them, or 2 would not bring more blocks (512 threads fill
// the registers at 128 each), or a single block is all that fits with 2. 16384 rows backward with an fp32 residual,
// layer norm, us with 3 and with 2 stages: x 2048 122 / 108, x 2560 174 / 140, x 3000 187 / 200; 8192 in bf16 303 / 328.
// The RMS norm, of less arithmetic, keeps 3 in blocks of up to 128 threads too: x 1280 72 / 78, x 2048 101 / 106, but
// x 2560 137 / 132, and odd rows x 1001 113 / 92.
inline int ring_stages(const RowPlan& p, int thread_bytes, int kind) {
    const int row = stage_bytes(p, thread_bytes);
    if (!p.ring) return 0;
    const int n3 = kSmSmem / (3 * row + kHead + 1024), n2 = kSmSmem / (2 * row + kHead + 1024);
    if (n3 >= 2 && (p.all_f32 || n3 * p.threads >= 448 || n3 >= (n2 < 512 / p.threads ? n2 : 512 / p.threads) ||
                    (kind == GLA_NORM_RMS && p.threads <= 128 && !p.odd)))
        return 3;
    if (!p.all_f32 && n2 < 2 && n3 * p.threads >= 448) return 3;
    return n2 ? 2 : 0;
}
inline size_t block_smem(const RowPlan& p, int stages, int thread_bytes) {
    const size_t ring = kHead + (size_t)stages * stage_bytes(p, thread_bytes);
    const size_t cols = p.threads == p.G ? 0 : (size_t)4 * p.threads * p.nv * p.vec;
    return ring > cols ? ring : cols;
}

// Blocks that walk the rows, and so partial rows of the column sums: no more than give every SM
// 1024 threads, 2048 where a warp holds a row. The launch takes fewer where fewer fit, so that no block
// waits for another.
inline int row_blocks(const RowPlan& p, long long rows, int heads) {
    const int per = p.threads / p.G;
    const long long need = (rows + per - 1) / per;
    long long most = (long long)tc::num_sms() * ((p.G <= 32 ? 2048 : 1024) / p.threads) / heads;
    if (most < 1) most = 1;
    return (int)(need < most ? need : most);
}
// Blocks of `kern` that an SM holds, asked of the runtime once per kernel, device and group (`known`; a kernel's threads
// and shared memory follow from these: groups up to a warp stand in blocks of 256, longer ones are the block).
using Occupancy = std::atomic<int>[kMaxDevices][33 + 33];
template <typename K>
int fit_blocks(K kern, const RowPlan& p, size_t smem, int blocks, int heads, Occupancy& known) {
    if ((long long)blocks * heads <= tc::num_sms()) return blocks;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return blocks;
    std::atomic<int>& slot = known[dev][p.G <= 32 ? 33 + p.G : p.G / 32];
    int per_sm = slot.load(std::memory_order_relaxed);
    if (per_sm == 0) {
        if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kern, p.threads, smem) != cudaSuccess ||
            per_sm < 1) {
            cudaGetLastError();
            return blocks;
        }
        slot.store(per_sm, std::memory_order_relaxed);
    }
    const int fit = tc::num_sms() * per_sm / heads;
    return fit < 1 ? 1 : fit < blocks ? fit : blocks;
}

// Picks the kernel's shape: VEC, NV, ring stages, largest block.
template <int V, int N, int S, int M, bool O = false> struct Shape {
    static constexpr int vec = V, nv = N, stages = S, maxt = M;
    static constexpr bool odd = O;
};
// BF16, F32: every operand of the row has that type, so pieces of 8, and a ring of single elements, exist too.
// Blocks of up to 256 threads (D <= 4096 with pieces of 4 or 8) have kernels of their own, which need not fit their
// registers into a larger block's share. Without a ring only rows beyond 8192 elements (up to 1024 threads, which
// with 16 elements each spill 500 bytes and more), odd fp32 rows beyond 6656, and fp32 rows too long for two stages. The
// backwards with two stages and 512 threads spill 32 to 96 bytes.
template <int V, int N, int S, bool O = false, typename F>
cudaError_t by_block(const RowPlan& p, F&& f) {
    return p.threads <= 256 ? f(Shape<V, N, S, 256, O>{}) : f(Shape<V, N, S, 512, O>{});
}
template <int V, int N, bool F32, typename F>
cudaError_t no_ring(const RowPlan& p, F&& f) {
    if constexpr (F32)
        if (p.threads <= 512) return f(Shape<V, N, 0, 512>{});
    return f(Shape<V, N, 0, 1024>{});   // with bf16 in the row always more threads
}
template <bool BF16, bool F32, bool WIDE, typename F>
cudaError_t by_shape(const RowPlan& p, int stages, F&& f) {
    if (p.odd) {
        if (stages == 2) return f(Shape<2, 8, 2, 512, true>{});
        if constexpr (F32) return f(Shape<2, 8, 3, 512, true>{});
        else return by_block<2, 8, 3, true>(p, f);
    }
    if (p.vec == 1) {
        if constexpr (F32)
            if (p.nv == 4) return by_block<1, 4, 3>(p, f);   // three stages of 512 threads fit twice
        return no_ring<1, 16, F32>(p, f);
    }
    if (p.vec == 2) {
        if (p.nv == 4) return stages == 3 ? by_block<2, 4, 3>(p, f) : f(Shape<2, 4, 2, 512>{});
        return stages == 3 ? f(Shape<2, 8, 3, 512>{}) : stages == 2 ? f(Shape<2, 8, 2, 512>{}) : no_ring<2, 8, F32>(p, f);
    }
    if constexpr (WIDE)
        if (p.vec * p.nv == 8) {
            if constexpr (BF16)
                if (p.vec == 8) return stages == 3 ? f(Shape<8, 1, 3, kWide>{}) : f(Shape<8, 1, 2, kWide>{});
            return stages == 3 ? f(Shape<4, 2, 3, kWide>{}) : f(Shape<4, 2, 2, kWide>{});
        }
    if constexpr (BF16)
        if (p.vec == 8)
            return stages == 3   ? by_block<8, 2, 3>(p, f)
                   : stages == 2 ? f(Shape<8, 2, 2, 512>{})
                                 : f(Shape<8, 2, 0, 1024>{});
    return stages == 3   ? by_block<4, 4, 3>(p, f)
           : stages == 2 ? f(Shape<4, 4, 2, 512>{})
                         : no_ring<4, 4, F32>(p, f);
}
template <typename F>
cudaError_t by_kind(int kind, F&& f) {
    return kind == GLA_NORM_RMS ? f(std::integral_constant<int, GLA_NORM_RMS>{})
                                : f(std::integral_constant<int, GLA_NORM_LAYER>{});
}

inline bool aligned16(const void* x) { return x == nullptr || (reinterpret_cast<uintptr_t>(x) & 15u) == 0; }
template <int N>
bool all_aligned(const void* const (&ptrs)[N]) {
    for (const void* q : ptrs)
        if (!aligned16(q)) return false;
    return true;
}
// What both operators ask of a problem.
inline gla_status check_common(const gla_norm_problem* p) {
    if (!p || p->B < 0 || p->H < 0 || p->L < 0 || p->D < 1) return GLA_ERR_INVALID_ARG;
    if (p->io != GLA_F32 && p->io != GLA_BF16) return GLA_ERR_INVALID_ARG;
    if (p->kind != GLA_NORM_RMS && p->kind != GLA_NORM_LAYER) return GLA_ERR_INVALID_ARG;
    if (!(p->eps > 0.f) || p->eps > 3.4e38f) return GLA_ERR_INVALID_ARG;
    if (p->D > 16384 || (long long)p->B * p->L > 2147483647LL) return GLA_ERR_UNSUPPORTED;
    return GLA_OK;
}

}  // namespace norm
}  // namespace gla
