// Short causal convolution of every channel along its sequence (wtconv_ssm.h).  Bound by memory: each activation
// is read once (a strip's first K-1 inputs twice) and each result written once, in vectors of 16 bytes where
// addresses allow it.
#pragma once

#include "causal.h"
#include "column_sums.cuh"
#include "train_device.cuh"

namespace wtconv {

constexpr float kCausalLog2E = 1.4426950408889634f;

__device__ __forceinline__ float causal_sigmoid(float v) {
    float e;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(-kCausalLog2E * v));
    return reciprocal(1.f + e);
}
__device__ __forceinline__ float causal_f(float pre, int silu) { return silu ? pre * causal_sigmoid(pre) : pre; }
__device__ __forceinline__ float causal_slope(float pre, int silu) {
    if (!silu) return 1.f;
    const float p = causal_sigmoid(pre);
    return p * fmaf(pre, 1.f - p, 1.f);
}
__device__ __forceinline__ int length_of(const CausalArgs &a, int b) {
    return a.lengths == nullptr ? a.s.T : min(max(a.lengths[b], 0), a.s.T);
}

// One channel's input at a position of [-(K-1), length): the state holds the negative ones.
template <typename T, int K> __device__ __forceinline__ float input_at(const CausalArgs &a, int b, int c, int t) {
    if (t < 0) {
        if (a.state == nullptr) return 0.f;
        return to_f32(static_cast<const T *>(a.state)[((long long)b * a.s.C + c) * (K - 1) + t + K - 1]);
    }
    const bool planes = a.s.layout == WTCONV_SCAN_PLANES;
    return to_f32(static_cast<const T *>(a.x.p)[b * a.x.batch + (planes ? c : t) * a.x.row + (planes ? t : c)]);
}

// The states' ends, a thread for each (sequence, channel): after the forward's CTAs and the backward's.
template <typename T, int K> __device__ __forceinline__ void write_state_last(const CausalArgs &a, long long i) {
    if (i >= (long long)a.s.B * a.s.C) return;
    const int b = i / a.s.C, c = i % a.s.C, length = length_of(a, b);
#pragma unroll
    for (int j = 0; j < K - 1; ++j)
        static_cast<T *>(a.state_last)[i * (K - 1) + j] = from_f32<T>(input_at<T, K>(a, b, c, length - K + 1 + j));
}
template <typename T, int K> __device__ __forceinline__ void write_d_state(const CausalArgs &a, long long i) {
    if (i >= (long long)a.s.B * a.s.C) return;
    const int b = i / a.s.C, c = i % a.s.C, length = length_of(a, b);
    const bool planes = a.s.layout == WTCONV_SCAN_PLANES;
    float w[K], slope[K - 1];
#pragma unroll
    for (int k = 0; k < K; ++k) w[k] = a.w[(long long)c * K + k];
#pragma unroll
    for (int t = 0; t < K - 1; ++t) {
        slope[t] = 0.f;
        if (t >= length) continue;
        float pre = a.bias == nullptr ? 0.f : a.bias[c];
#pragma unroll
        for (int k = 0; k < K; ++k) pre = fmaf(w[k], input_at<T, K>(a, b, c, t - K + 1 + k), pre);
        const T *dy = static_cast<const T *>(a.dy.p) + b * a.dy.batch + (planes ? c : t) * a.dy.row + (planes ? t : c);
        slope[t] = to_f32(*dy) * causal_slope(pre, a.s.silu);
    }
#pragma unroll
    for (int j = 0; j < K - 1; ++j) {  // position j - (K-1), which reaches positions 0 to j
        float v = 0.f;
#pragma unroll
        for (int t = 0; t <= j; ++t) v = fmaf(w[j - t], slope[t], v);
        if (a.d_last != nullptr && j >= length)  // place j - length of the last state
            v += to_f32(static_cast<const T *>(a.d_last)[i * (K - 1) + j - length]);
        static_cast<T *>(a.d_state)[i * (K - 1) + j] = from_f32<T>(v);
    }
}

// --------------------------------------------------------------------------------------- tokens

// A warp's lanes take neighbouring vectors of channels, a thread goes along its strip of positions with the last K
// inputs in registers.
template <typename T, int K, int V> __global__ void __launch_bounds__(256) causal_tokens_forward_kernel(const __grid_constant__ CausalArgs a) {
    constexpr int AHEAD = 4;  // positions loaded before the first is used
    begin_kernel();
    const int columns = (a.s.C + 32 * V - 1) / (32 * V), groups = (a.strips + 7) / 8;
    const unsigned main = (unsigned)a.s.B * groups * columns;
    if (blockIdx.x >= main) return write_state_last<T, K>(a, (long long)(blockIdx.x - main) * 256 + threadIdx.x);
    const int column = blockIdx.x % columns, rest = blockIdx.x / columns, b = rest / groups;
    const int strip = rest % groups * 8 + threadIdx.x / 32, c = (column * 32 + threadIdx.x % 32) * V;
    if (strip >= a.strips || c >= a.s.C) return;
    const int first = strip * a.strip, end = min(first + a.strip, a.s.T), length = length_of(a, b), stop = min(end, length);
    const T *x = static_cast<const T *>(a.x.p) + b * a.x.batch + c;
    T *y = static_cast<T *>(a.y.p) + b * a.y.batch + c;
    if (first < stop) {
        float w[K][V], bias[V], in[K - 1 + AHEAD][V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            bias[i] = a.bias == nullptr ? 0.f : a.bias[c + i];
#pragma unroll
            for (int k = 0; k < K; ++k) w[k][i] = a.w[(long long)(c + i) * K + k];
        }
#pragma unroll
        for (int k = 0; k < K - 1; ++k) {
            const int t = first - K + 1 + k;
            if (t >= 0) load_vec<T, V>(x + t * a.x.row, in[k]);
            else
#pragma unroll
                for (int i = 0; i < V; ++i) in[k][i] = input_at<T, K>(a, b, c + i, t);
        }
        for (int t0 = first; t0 < stop; t0 += AHEAD) {
#pragma unroll
            for (int j = 0; j < AHEAD; ++j)
                if (t0 + j < stop) load_vec<T, V>(x + (t0 + j) * a.x.row, in[K - 1 + j]);
#pragma unroll
            for (int j = 0; j < AHEAD; ++j) {
                if (t0 + j >= stop) break;
                float v[V];
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    v[i] = bias[i];
#pragma unroll
                    for (int k = 0; k < K; ++k) v[i] = fmaf(w[k][i], in[j + k][i], v[i]);
                    v[i] = causal_f(v[i], a.s.silu);
                }
                store_vec<T, V>(y + (t0 + j) * a.y.row, v);
            }
#pragma unroll
            for (int k = 0; k < K - 1; ++k)
#pragma unroll
                for (int i = 0; i < V; ++i) in[k][i] = in[AHEAD + k][i];
        }
    }
    const float zero[V] = {};
    for (int t = max(first, length); t < end; ++t) store_vec<T, V>(y + t * a.y.row, zero);
}

// The strip's K-1 following positions are computed too, for the gradients of its own inputs; dw and d_bias count
// the strip's own positions.
template <typename T, int K, int V> __global__ void __launch_bounds__(256) causal_tokens_backward_kernel(const __grid_constant__ CausalArgs a) {
    __shared__ float meet[8][32 * V];
    constexpr int AHEAD = 4;
    begin_kernel();
    const int columns = (a.s.C + 32 * V - 1) / (32 * V), groups = (a.strips + 7) / 8;
    const unsigned main = (unsigned)a.s.B * groups * columns;
    if (blockIdx.x >= main) return write_d_state<T, K>(a, (long long)(blockIdx.x - main) * 256 + threadIdx.x);
    const int column = blockIdx.x % columns, part = blockIdx.x / columns, b = part / groups, warp = threadIdx.x / 32;
    const int strip = part % groups * 8 + warp, c = (column * 32 + threadIdx.x % 32) * V;
    float dw[K][V] = {}, db[V] = {};
    if (strip < a.strips && c < a.s.C) {
        const int first = strip * a.strip, end = min(first + a.strip, a.s.T), length = length_of(a, b);
        const int stop = min(end, length), beyond = min(end + K - 1, length);  // last position that reaches the strip
        const T *x = static_cast<const T *>(a.x.p) + b * a.x.batch + c, *dy = static_cast<const T *>(a.dy.p) + b * a.dy.batch + c;
        T *dx = static_cast<T *>(a.dx.p) + b * a.dx.batch + c;
        const long long row = (long long)b * a.s.C + c;
        if (first < stop) {
            float w[K][V], bias[V], in[K - 1 + AHEAD][V], slope[K - 1 + AHEAD][V];
#pragma unroll
            for (int i = 0; i < V; ++i) {
                bias[i] = a.bias == nullptr ? 0.f : a.bias[c + i];
#pragma unroll
                for (int k = 0; k < K; ++k) w[k][i] = a.w[(long long)(c + i) * K + k];
            }
#pragma unroll
            for (int k = 0; k < K - 1; ++k) {
                const int t = first - K + 1 + k;
                if (t >= 0) load_vec<T, V>(x + t * a.x.row, in[k]);
                else
#pragma unroll
                    for (int i = 0; i < V; ++i) in[k][i] = input_at<T, K>(a, b, c + i, t);
#pragma unroll
                for (int i = 0; i < V; ++i) slope[k][i] = 0.f;
            }
            for (int t0 = first; t0 < stop + K - 1; t0 += AHEAD) {
                float g[AHEAD][V];
#pragma unroll
                for (int j = 0; j < AHEAD; ++j) {
                    if (t0 + j < beyond) {
                        load_vec<T, V>(x + (t0 + j) * a.x.row, in[K - 1 + j]);
                        load_vec<T, V>(dy + (t0 + j) * a.dy.row, g[j]);
                    }
                }
#pragma unroll
                for (int j = 0; j < AHEAD; ++j) {
                    const int t = t0 + j, own = t - K + 1;  // the input whose last reader t is
                    if (t < beyond) {
#pragma unroll
                        for (int i = 0; i < V; ++i) {
                            float pre = bias[i];
#pragma unroll
                            for (int k = 0; k < K; ++k) pre = fmaf(w[k][i], in[j + k][i], pre);
                            const float s = g[j][i] * causal_slope(pre, a.s.silu);
                            slope[K - 1 + j][i] = s;
                            if (t < stop) {
                                db[i] += s;
#pragma unroll
                                for (int k = 0; k < K; ++k) dw[k][i] = fmaf(s, in[j + k][i], dw[k][i]);
                            }
                        }
                    } else {
#pragma unroll
                        for (int i = 0; i < V; ++i) slope[K - 1 + j][i] = 0.f;
                    }
                    if (own >= first && own < stop) {
                        float v[V] = {};
#pragma unroll
                        for (int i = 0; i < V; ++i)
#pragma unroll
                            for (int k = 0; k < K; ++k) v[i] = fmaf(w[K - 1 - k][i], slope[j + k][i], v[i]);
                        if (a.d_last != nullptr && own >= length - K + 1) {
#pragma unroll
                            for (int i = 0; i < V; ++i)
                                v[i] += to_f32(static_cast<const T *>(a.d_last)[(row + i) * (K - 1) + own - (length - K + 1)]);
                        }
                        store_vec<T, V>(dx + own * a.dx.row, v);
                    }
                }
#pragma unroll
                for (int k = 0; k < K - 1; ++k)
#pragma unroll
                    for (int i = 0; i < V; ++i) in[k][i] = in[AHEAD + k][i], slope[k][i] = slope[AHEAD + k][i];
            }
        }
        const float zero[V] = {};
        for (int t = max(first, length); t < end; ++t) store_vec<T, V>(dx + t * a.dx.row, zero);
    }
    // over the CTA's strips
#pragma unroll
    for (int k = 0; k <= K; ++k) {
#pragma unroll
        for (int i = 0; i < V; ++i) meet[warp][i * 32 + threadIdx.x % 32] = k == K ? db[i] : dw[k == K ? 0 : k][i];
        __syncthreads();
        for (int e = threadIdx.x; e < 32 * V; e += 256) {
            float v = 0.f;
#pragma unroll
            for (int m = 0; m < 8; ++m) v += meet[m][e];
            const int to = (column * 32 + e % 32) * V + e / 32;
            if (to < a.s.C) {
                if (k == K) a.part_b[(long long)part * a.s.C + to] = v;
                else a.part_w[((long long)part * a.s.C + to) * K + k] = v;
            }
        }
        __syncthreads();
    }
}

// --------------------------------------------------------------------------------------- planes

// 2^row_bits neighbouring lanes go along a strip of a row, a vector of positions each; inputs beside it come from
// the first-level cache.
template <typename T, int K, int V> __global__ void __launch_bounds__(256) causal_planes_forward_kernel(const __grid_constant__ CausalArgs a) {
    begin_kernel();
    const int lanes = 1 << a.row_bits, per = 256 >> a.row_bits;  // strips of a CTA
    const long long all = (long long)a.s.B * a.s.C * a.strips;
    const unsigned main = (unsigned)((all + per - 1) / per);
    if (blockIdx.x >= main) return write_state_last<T, K>(a, (long long)(blockIdx.x - main) * 256 + threadIdx.x);
    const long long unit = (long long)blockIdx.x * per + (threadIdx.x >> a.row_bits);
    if (unit >= all) return;
    const int row = unit / a.strips, strip = unit % a.strips, b = row / a.s.C, c = row % a.s.C, length = length_of(a, b);
    const int first = strip * a.strip, end = min(first + a.strip, a.s.T), lane = threadIdx.x & (lanes - 1);
    const T *x = static_cast<const T *>(a.x.p) + b * a.x.batch + c * a.x.row;
    T *y = static_cast<T *>(a.y.p) + b * a.y.batch + c * a.y.row;
    float w[K];
#pragma unroll
    for (int k = 0; k < K; ++k) w[k] = a.w[(long long)c * K + k];
    const float bias = a.bias == nullptr ? 0.f : a.bias[c];
    for (int t0 = first + lane * V; t0 < end; t0 += lanes * V) {
        float in[V + K - 1], v[V];
        const bool whole = t0 + V <= a.s.T;
        if (t0 + V <= length) {
            float q[V];
            load_vec<T, V>(x + t0, q);
#pragma unroll
            for (int i = 0; i < V; ++i) in[K - 1 + i] = q[i];
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) in[K - 1 + i] = t0 + i < length ? to_f32(x[t0 + i]) : 0.f;
        }
#pragma unroll
        for (int k = 0; k < K - 1; ++k) {
            const int t = t0 - K + 1 + k;
            in[k] = t >= 0 ? (t < length ? to_f32(x[t]) : 0.f) : input_at<T, K>(a, b, c, t);
        }
#pragma unroll
        for (int i = 0; i < V; ++i) {
            v[i] = bias;
#pragma unroll
            for (int k = 0; k < K; ++k) v[i] = fmaf(w[k], in[i + k], v[i]);
            v[i] = t0 + i < length ? causal_f(v[i], a.s.silu) : 0.f;
        }
        if (whole) store_vec<T, V>(y + t0, v);
        else
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (t0 + i < a.s.T) y[t0 + i] = from_f32<T>(v[i]);
    }
}

template <typename T, int K, int V> __global__ void __launch_bounds__(256) causal_planes_backward_kernel(const __grid_constant__ CausalArgs a) {
    begin_kernel();
    const int lanes = 1 << a.row_bits, per = 256 >> a.row_bits;
    const long long all = (long long)a.s.B * a.s.C * a.strips;
    const unsigned main = (unsigned)((all + per - 1) / per);
    if (blockIdx.x >= main) return write_d_state<T, K>(a, (long long)(blockIdx.x - main) * 256 + threadIdx.x);
    const long long unit = (long long)blockIdx.x * per + (threadIdx.x >> a.row_bits);
    const bool used = unit < all;
    const int row = used ? unit / a.strips : 0, strip = used ? unit % a.strips : 0, b = row / a.s.C, c = row % a.s.C;
    const int length = length_of(a, b), lane = threadIdx.x & (lanes - 1);
    const int first = strip * a.strip, end = used ? min(first + a.strip, a.s.T) : 0;
    const T *x = static_cast<const T *>(a.x.p) + b * a.x.batch + c * a.x.row, *dy = static_cast<const T *>(a.dy.p) + b * a.dy.batch + c * a.dy.row;
    T *dx = static_cast<T *>(a.dx.p) + b * a.dx.batch + c * a.dx.row;
    float w[K], dw[K] = {}, db = 0.f;
#pragma unroll
    for (int k = 0; k < K; ++k) w[k] = a.w[(long long)c * K + k];
    const float bias = a.bias == nullptr ? 0.f : a.bias[c];
    for (int t0 = first + lane * V; t0 < end; t0 += lanes * V) {
        float in[V + 2 * (K - 1)], g[V + K - 1], v[V];  // inputs t0 - (K-1) ..., dy t0 ...
        if (t0 + V <= length) {
            float q[V], r[V];
            load_vec<T, V>(x + t0, q), load_vec<T, V>(dy + t0, r);
#pragma unroll
            for (int i = 0; i < V; ++i) in[K - 1 + i] = q[i], g[i] = r[i];
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) in[K - 1 + i] = t0 + i < length ? to_f32(x[t0 + i]) : 0.f, g[i] = t0 + i < length ? to_f32(dy[t0 + i]) : 0.f;
        }
#pragma unroll
        for (int k = 0; k < K - 1; ++k) {
            const int t = t0 - K + 1 + k, u = t0 + V + k;
            in[k] = t >= 0 ? (t < length ? to_f32(x[t]) : 0.f) : input_at<T, K>(a, b, c, t);
            in[V + K - 1 + k] = u < length ? to_f32(x[u]) : 0.f, g[V + k] = u < length ? to_f32(dy[u]) : 0.f;
        }
#pragma unroll
        for (int i = 0; i < V + K - 1; ++i) {  // g: the gradient before f
            float pre = bias;
#pragma unroll
            for (int k = 0; k < K; ++k) pre = fmaf(w[k], in[i + k], pre);
            g[i] = t0 + i < length ? g[i] * causal_slope(pre, a.s.silu) : 0.f;
            if (i < V) {
                db += g[i];
#pragma unroll
                for (int k = 0; k < K; ++k) dw[k] = fmaf(g[i], in[i + k], dw[k]);
            }
        }
#pragma unroll
        for (int i = 0; i < V; ++i) {
            v[i] = 0.f;
#pragma unroll
            for (int k = 0; k < K; ++k) v[i] = fmaf(w[K - 1 - k], g[i + k], v[i]);
            const int t = t0 + i;
            if (t >= length) v[i] = 0.f;
            else if (a.d_last != nullptr && t >= length - K + 1)
                v[i] += to_f32(static_cast<const T *>(a.d_last)[(long long)row * (K - 1) + t - (length - K + 1)]);
        }
        if (t0 + V <= a.s.T) store_vec<T, V>(dx + t0, v);
        else
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (t0 + i < a.s.T) dx[t0 + i] = from_f32<T>(v[i]);
    }
    const long long part = (long long)b * a.strips + strip;
#pragma unroll
    for (int k = 0; k <= K; ++k) {
        float s = k == K ? db : dw[k == K ? 0 : k];
        for (int m = lanes / 2; m >= 1; m /= 2) s += __shfl_xor_sync(0xffffffffu, s, m);
        if (used && lane == 0) {
            if (k == K) a.part_b[part * a.s.C + c] = s;
            else a.part_w[(part * a.s.C + c) * K + k] = s;
        }
    }
}

// ---------------------------------------------------------------------------------------- launch

template <bool BACKWARD, typename T, int K, int V> cudaError_t launch_causal_as(const CausalArgs &a, cudaStream_t st) {
    const bool planes = a.s.layout == WTCONV_SCAN_PLANES, ends = BACKWARD ? a.d_state != nullptr : a.state_last != nullptr;
    const long long rows = (long long)a.s.B * a.s.C;
    long long grid = planes ? (rows * a.strips + (256 >> a.row_bits) - 1) / (256 >> a.row_bits)
                            : (long long)a.s.B * ceil_div(a.strips, 8) * ceil_div(a.s.C, 32 * V);
    if (ends) grid += (rows + 255) / 256;
    if (grid > 0x7fffffffll) return cudaErrorInvalidValue;
    if constexpr (BACKWARD)
        return planes ? launch_kernel(causal_planes_backward_kernel<T, K, V>, (unsigned)grid, 256, 0, st, 1, a)
                      : launch_kernel(causal_tokens_backward_kernel<T, K, V>, (unsigned)grid, 256, 0, st, 1, a);
    else
        return planes ? launch_kernel(causal_planes_forward_kernel<T, K, V>, (unsigned)grid, 256, 0, st, 1, a)
                      : launch_kernel(causal_tokens_forward_kernel<T, K, V>, (unsigned)grid, 256, 0, st, 1, a);
}
template <bool BACKWARD, typename T, int V> cudaError_t launch_causal_taps(const CausalArgs &a, cudaStream_t st) {
    return a.s.K == 2   ? launch_causal_as<BACKWARD, T, 2, V>(a, st)
           : a.s.K == 3 ? launch_causal_as<BACKWARD, T, 3, V>(a, st)
                        : launch_causal_as<BACKWARD, T, 4, V>(a, st);
}

template <typename T> cudaError_t launch_causal_forward(const CausalArgs &a, cudaStream_t st) {
    return a.wide > 1 ? launch_causal_taps<false, T, 16 / sizeof(T)>(a, st) : launch_causal_taps<false, T, 1>(a, st);
}
template <typename T> cudaError_t launch_causal_backward(const CausalArgs &a, cudaStream_t st) {
    const cudaError_t e = a.wide > 1 ? launch_causal_taps<true, T, 4>(a, st) : launch_causal_taps<true, T, 1>(a, st);
    if (e != cudaSuccess) return e;
    ColumnSums s = {};
    s.parts = a.parts;
    s.part[0] = a.part_w, s.part[1] = a.part_b, s.out[0] = a.dw, s.out[1] = a.d_bias;
    s.width[0] = a.s.C * a.s.K, s.width[1] = a.s.C;
    return launch_column_sums(s, st);
}

// One position of every sequence, a thread to a channel.
template <typename T, int K>
__global__ void __launch_bounds__(128) causal_step_kernel(const __grid_constant__ CausalArgs a, T *pool, int n_states, const int *slots) {
    begin_kernel();
    const int blocks = (a.s.C + 127) / 128, b = blockIdx.x / blocks, c = blockIdx.x % blocks * 128 + threadIdx.x;
    if (c >= a.s.C) return;
    const int slot = slots == nullptr ? b : slots[b];
    float v = 0.f;
    if (slot >= 0 && slot < n_states) {
        T *state = pool + ((long long)slot * a.s.C + c) * (K - 1), in[K];
#pragma unroll
        for (int k = 0; k < K - 1; ++k) in[k] = state[k];
        in[K - 1] = static_cast<const T *>(a.x.p)[b * a.x.row + c];
        v = a.bias == nullptr ? 0.f : a.bias[c];
#pragma unroll
        for (int k = 0; k < K; ++k) v = fmaf(a.w[(long long)c * K + k], to_f32(in[k]), v);
        v = causal_f(v, a.s.silu);
#pragma unroll
        for (int k = 0; k < K - 1; ++k) state[k] = in[k + 1];
    }
    static_cast<T *>(a.y.p)[b * a.y.row + c] = from_f32<T>(v);
}
template <typename T> cudaError_t launch_causal_step(const CausalArgs &a, void *pool, int n_states, const int *slots, cudaStream_t st) {
    const unsigned grid = (unsigned)a.s.B * ceil_div(a.s.C, 128);
    T *const p = static_cast<T *>(pool);
    return a.s.K == 2   ? launch_kernel(causal_step_kernel<T, 2>, grid, 128, 0, st, 1, a, p, n_states, slots)
           : a.s.K == 3 ? launch_kernel(causal_step_kernel<T, 3>, grid, 128, 0, st, 1, a, p, n_states, slots)
                        : launch_kernel(causal_step_kernel<T, 4>, grid, 128, 0, st, 1, a, p, n_states, slots);
}

}  // namespace wtconv
