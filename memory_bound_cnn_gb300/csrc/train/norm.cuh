// Root-mean-square norm with the residual's addition, and its gradient (wtconv_norm.h).  Bound by memory: a row
// stays in the registers of its threads between the sum over it and what uses the sum, so that each tensor is
// read or written once; w comes from the first-level cache after a CTA's first row.
#pragma once

#include <cuda_fp8.h>

#include <algorithm>
#include <type_traits>

#include "column_sums.cuh"
#include "norm.h"
#include "train_device.cuh"

namespace wtconv {

__device__ __forceinline__ float max_nan(float a, float b) {  // a NaN comes through
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// What LANES threads of a row (one warp, or a whole CTA) make of their values, in the same order every time.
// meet: a float for each of the row's warps; a CTA takes turns between two of them, so that one barrier does.
template <int LANES, bool MAX> __device__ __forceinline__ float across_row(float v, float *meet) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
        const float o = __shfl_xor_sync(0xffffffffu, v, d);
        v = MAX ? max_nan(v, o) : v + o;
    }
    if (LANES == 32) return v;
    if (threadIdx.x % 32 == 0) meet[threadIdx.x / 32] = v;
    __syncthreads();
    v = meet[0];
#pragma unroll
    for (int i = 1; i < LANES / 32; ++i) v = MAX ? max_nan(v, meet[i]) : v + meet[i];
    return v;
}

// A row's values: element (j * LANES + lane) * V + i of it is v[j * V + i].
template <typename S, int LANES, int EACH, int V>
__device__ __forceinline__ void load_row(const S *row, int lane, int C, float (&v)[EACH]) {
#pragma unroll
    for (int j = 0; j < EACH / V; ++j) {
        const int at = (j * LANES + lane) * V;
        float q[V] = {};
        if (at < C) load_vec<S, V>(row + at, q);
#pragma unroll
        for (int i = 0; i < V; ++i) v[j * V + i] = q[i];
    }
}
template <typename S, int LANES, int EACH, int V>
__device__ __forceinline__ void store_row(S *row, int lane, int C, const float (&v)[EACH]) {
#pragma unroll
    for (int j = 0; j < EACH / V; ++j) {
        const int at = (j * LANES + lane) * V;
        float q[V];
#pragma unroll
        for (int i = 0; i < V; ++i) q[i] = v[j * V + i];
        if (at < C) store_vec<S, V>(row + at, q);
    }
}

constexpr int kNormThreads = 128;  // of a CTA whose warps have a row each

// CTAs to an SM that registers have to suffice for, 40 a thread (16,384 rows of 2048 in e4m3 with an fp32 residual:
// 62.7 us; with 44 and a CTA less 67.7).
constexpr int norm_ctas(int threads, int each, int v) { return each == 8 && v > 1 ? 1536 / threads : 1; }

// LANES threads to a row, EACH values to a thread; V neighbours (C is a multiple of V).
template <typename T, typename R, int LANES, int EACH, int V, bool E4M3>
__global__ void __launch_bounds__(LANES == 32 ? kNormThreads : LANES, norm_ctas(LANES == 32 ? kNormThreads : LANES, EACH, V)) norm_forward_kernel(const __grid_constant__ NormArgs a) {
    constexpr int ROWS = LANES == 32 ? kNormThreads / 32 : 1, WARPS = LANES / 32;
    __shared__ float meet[2][2][WARPS];
    __shared__ float tops[E4M3 && V == 1 ? ROWS : 1][E4M3 && V == 1 ? EACH * WARPS : 1];  // max |y| of 32 neighbours
    begin_kernel();
    const int lane = threadIdx.x % LANES, slot = threadIdx.x / LANES, C = a.s.C;
    int turn = 0;
    for (int row = blockIdx.x * ROWS + slot; row < a.s.rows; row += gridDim.x * ROWS, turn ^= 1) {  // (at most 2^30)
        float v[EACH];
        load_row<T, LANES, EACH, V>(static_cast<const T *>(a.x.p) + row * a.x.row, lane, C, v);
        if (a.residual.p != nullptr) {
            float r[EACH];
            load_row<R, LANES, EACH, V>(static_cast<const R *>(a.residual.p) + row * a.residual.row, lane, C, r);
#pragma unroll
            for (int i = 0; i < EACH; ++i) v[i] = to_f32(from_f32<R>(v[i] + r[i]));  // as it is stored
            store_row<R, LANES, EACH, V>(static_cast<R *>(a.total.p) + row * a.total.row, lane, C, v);
        }
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < EACH; ++i) s = fmaf(v[i], v[i], s);
        s = across_row<LANES, false>(s, meet[turn][0]);
        float rstd = rsqrtf(s / C + a.s.eps);
        if (a.rstd != nullptr && lane == 0) a.rstd[row] = rstd;
        // Of rstd = power x rest the power of two alone is in what the codes are made of: they do not depend on the root's
        // rounding, and largest values keep clear of the type's ends.
        const uint32_t bits = __float_as_uint(rstd), regular = rstd > 0.f && rstd < INFINITY;
        const float power = __uint_as_float(regular ? bits & 0x7f800000u : 0x3f800000u);
        if (E4M3) rstd = __uint_as_float(regular ? (bits & 0x007fffffu) | 0x3f800000u : bits);
        float w[EACH];
        load_row<float, LANES, EACH, V>(a.w, lane, C, w);
#pragma unroll
        for (int i = 0; i < EACH; ++i) v[i] = E4M3 ? v[i] * power * w[i] : v[i] * (rstd * w[i]);
        if constexpr (!E4M3) {
            store_row<T, LANES, EACH, V>(static_cast<T *>(a.y.p) + row * a.y.row, lane, C, v);
        } else {
            float top[EACH / V];  // of the block that each vector lies in
#pragma unroll
            for (int j = 0; j < EACH / V; ++j) {
                top[j] = 0.f;
#pragma unroll
                for (int i = 0; i < V; ++i) top[j] = max_nan(top[j], fabsf(v[j * V + i]));
            }
            if (a.block == 0) {
#pragma unroll
                for (int j = 1; j < EACH / V; ++j) top[0] = max_nan(top[0], top[j]);
                top[0] = across_row<LANES, true>(top[0], meet[turn][1]);
#pragma unroll
                for (int j = 1; j < EACH / V; ++j) top[j] = top[0];
            } else if constexpr (V > 1) {  // 128 elements: 128 / V neighbouring lanes
#pragma unroll
                for (int j = 0; j < EACH / V; ++j)
#pragma unroll
                    for (int d = 64 / V; d > 0; d >>= 1) top[j] = max_nan(top[j], __shfl_xor_sync(0xffffffffu, top[j], d));
            } else {  // four times 32 lanes
                const int warp = lane / 32;
#pragma unroll
                for (int j = 0; j < EACH; ++j) {
                    float m = top[j];
#pragma unroll
                    for (int d = 16; d > 0; d >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, d));
                    if (lane % 32 == 0) tops[slot][j * WARPS + warp] = m;
                }
                if (LANES == 32) __syncwarp();
                else __syncthreads();
#pragma unroll
                for (int j = 0; j < EACH; ++j) {
                    const float *m = tops[slot] + (j * WARPS + warp) / 4 * 4;
                    top[j] = max_nan(max_nan(m[0], m[1]), max_nan(m[2], m[3]));
                }
                if (LANES == 32) __syncwarp();  // (a CTA: the next row's sum has a barrier before these are written)
            }
#pragma unroll
            for (int j = 0; j < EACH / V; ++j) {
                const int at = (j * LANES + lane) * V;
                if (at >= C) continue;
                const float most = top[j] * rstd;
                const bool nothing = most < 7.7037197775489434e-34f;  // 2^-110
                const float inverse = nothing ? 0.f : 448.f / top[j];
                Vec<unsigned char, V> q;
#pragma unroll
                for (int i = 0; i < V; ++i) q.v[i] = __nv_cvt_float_to_fp8(v[j * V + i] * inverse, __NV_SATFINITE, __NV_E4M3);
                *reinterpret_cast<Vec<unsigned char, V> *>(a.q + (long long)row * C + at) = q;
                if (a.block == 0 ? at == 0 : at % 128 == 0)
                    a.scales[(long long)row * a.blocks + (a.block == 0 ? 0 : at / 128)] = nothing ? 0.f : most / 448.f;
            }
        }
    }
}

// A CTA goes through its rows with dw of its threads' columns in registers.
template <typename T, typename R, int LANES, int EACH, int V>
__global__ void __launch_bounds__(LANES == 32 ? kNormThreads : LANES) norm_backward_kernel(const __grid_constant__ NormArgs a) {
    constexpr int ROWS = LANES == 32 ? kNormThreads / 32 : 1, WARPS = LANES / 32;
    __shared__ float meet[2][WARPS];
    __shared__ float columns[LANES == 32 ? ROWS * 32 * EACH : 1];
    begin_kernel();
    const int lane = threadIdx.x % LANES, slot = threadIdx.x / LANES, C = a.s.C;
    float dw[EACH] = {};
    int turn = 0;
    for (long long row = (long long)blockIdx.x * ROWS + slot; row < a.s.rows; row += (long long)gridDim.x * ROWS, turn ^= 1) {
        float n[EACH], g[EACH];
        load_row<R, LANES, EACH, V>(static_cast<const R *>(a.total.p) + row * a.total.row, lane, C, n);
        load_row<T, LANES, EACH, V>(static_cast<const T *>(a.dy.p) + row * a.dy.row, lane, C, g);
        float d[EACH] = {};
        if (a.d_total.p != nullptr) load_row<R, LANES, EACH, V>(static_cast<const R *>(a.d_total.p) + row * a.d_total.row, lane, C, d);
        const float rstd = a.rstd_in[row];
        float w[EACH], s = 0.f;
        load_row<float, LANES, EACH, V>(a.w, lane, C, w);
#pragma unroll
        for (int i = 0; i < EACH; ++i) {
            n[i] *= rstd;
            dw[i] = fmaf(g[i], n[i], dw[i]);
            g[i] *= w[i];
            s = fmaf(g[i], n[i], s);
        }
        const float mean = across_row<LANES, false>(s, meet[turn]) / C;
#pragma unroll
        for (int i = 0; i < EACH; ++i) g[i] = fmaf(rstd, fmaf(-n[i], mean, g[i]), d[i]);
        if (a.dx.p != nullptr) store_row<T, LANES, EACH, V>(static_cast<T *>(a.dx.p) + row * a.dx.row, lane, C, g);
        if (a.d_residual.p != nullptr)
            store_row<R, LANES, EACH, V>(static_cast<R *>(a.d_residual.p) + row * a.d_residual.row, lane, C, g);
    }
    if (a.dw == nullptr) return;
    float *const to = a.part + (long long)blockIdx.x * C;
    if constexpr (LANES == 32) {  // the CTA's warps have the same columns
#pragma unroll
        for (int i = 0; i < EACH; ++i) columns[(slot * EACH + i) * 32 + lane] = dw[i];
        __syncthreads();
        for (int e = threadIdx.x; e < 32 * EACH; e += kNormThreads) {
            const int i = e / 32, at = (i / V * 32 + e % 32) * V + i % V;
            float v = 0.f;
            for (int r = 0; r < ROWS; ++r) v += columns[r * 32 * EACH + e];
            if (at < C) to[at] = v;
        }
    } else {
#pragma unroll
        for (int i = 0; i < EACH; ++i) {
            const int at = (i / V * LANES + lane) * V + i % V;
            if (at < C) to[at] = dw[i];
        }
    }
}

// The fewest threads and values that hold a row of C.
template <typename F> cudaError_t with_row_shape(int C, F f) {
    using std::integral_constant;
    if (C <= 256) return f(integral_constant<int, 32>(), integral_constant<int, 8>());
    if (C <= 512) return f(integral_constant<int, 32>(), integral_constant<int, 16>());
    if (C <= 1024) return f(integral_constant<int, 128>(), integral_constant<int, 8>());
    if (C <= 2048) return f(integral_constant<int, 256>(), integral_constant<int, 8>());
    if (C <= 4096) return f(integral_constant<int, 256>(), integral_constant<int, 16>());
    if (C <= 8192) return f(integral_constant<int, 512>(), integral_constant<int, 16>());
    return f(integral_constant<int, 512>(), integral_constant<int, 32>());
}

template <typename T, typename R> cudaError_t launch_norm_forward(const NormArgs &a, cudaStream_t st) {
    return with_row_shape(a.s.C, [&](auto lanes, auto each) {
        constexpr int LANES = lanes.value, EACH = each.value, V = 16 / sizeof(T);
        constexpr unsigned THREADS = LANES == 32 ? kNormThreads : LANES;
        // as many CTAs as run at once, or fewer where there are fewer rows (with 8 to an SM where 6 ran at once, 16,384 rows of
        // 2048 took 78 us)
        const auto launch = [&](auto kernel) {
            const int most = sm_count() * resident_ctas(kernel, THREADS);
            return launch_kernel(kernel, (unsigned)std::min(ceil_div(a.s.rows, LANES == 32 ? kNormThreads / 32 : 1), most), THREADS, 0, st, 1, a);
        };
        if (a.q != nullptr)
            return a.wide ? launch(norm_forward_kernel<T, R, LANES, EACH, V, true>) : launch(norm_forward_kernel<T, R, LANES, EACH, 1, true>);
        return a.wide ? launch(norm_forward_kernel<T, R, LANES, EACH, V, false>) : launch(norm_forward_kernel<T, R, LANES, EACH, 1, false>);
    });
}
template <typename T, typename R> cudaError_t launch_norm_backward(const NormArgs &a, cudaStream_t st) {
    const int grid = norm_backward_grid(a.s.rows, a.s.C);
    const cudaError_t e = with_row_shape(a.s.C, [&](auto lanes, auto each) {
        constexpr int LANES = lanes.value, EACH = each.value, V = 16 / sizeof(T);
        constexpr unsigned THREADS = LANES == 32 ? kNormThreads : LANES;
        return a.wide ? launch_kernel(norm_backward_kernel<T, R, LANES, EACH, V>, (unsigned)grid, THREADS, 0, st, 1, a)
                      : launch_kernel(norm_backward_kernel<T, R, LANES, EACH, 1>, (unsigned)grid, THREADS, 0, st, 1, a);
    });
    if (e != cudaSuccess || a.dw == nullptr) return e;
    ColumnSums s = {};
    s.parts = grid, s.part[0] = a.part, s.out[0] = a.dw, s.width[0] = a.s.C;
    return launch_column_sums(s, st);
}

}  // namespace wtconv
