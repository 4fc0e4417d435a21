// Short causal convolution of every channel along its sequence (wtconv_ssm.h).  Bound by memory: each activation
// is read once (a strip's first K-1 inputs twice) and each result written once.  Where addresses allow it, a thread of
// planes takes 16 bytes at once (8 in the backward of 16-bit types), one of tokens a pair of channels.
#pragma once

#include "causal.h"
#include "column_sums.cuh"
#include "train_device.cuh"

namespace wtconv {

constexpr float kCausalLog2E = 1.4426950408889634f;

__device__ __forceinline__ Pair causal_sigmoid(Pair v) {
    const Pair w = mul(v, Pair(-kCausalLog2E));
    float a, b;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(a) : "f"(w.lo()));
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(b) : "f"(w.hi()));
    const Pair s = add(Pair(a, b), Pair(1.f));
    return {reciprocal(s.lo()), reciprocal(s.hi())};
}
template <bool SILU> __device__ __forceinline__ Pair causal_f(Pair pre) { return SILU ? mul(pre, causal_sigmoid(pre)) : pre; }
template <bool SILU> __device__ __forceinline__ Pair causal_slope(Pair pre) {
    if (!SILU) return Pair(1.f);
    const Pair p = causal_sigmoid(pre);
    return mul(p, fma(pre, sub(Pair(1.f), p), Pair(1.f)));
}
__device__ __forceinline__ float causal_f(float pre, int silu) { return silu ? causal_f<true>(Pair(pre)).lo() : pre; }
__device__ __forceinline__ float causal_slope(float pre, int silu) { return silu ? causal_slope<true>(Pair(pre)).lo() : 1.f; }
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

// A pair of neighbouring channels: at once where WIDE, else one at a time; `both`: the second is one of the tensor's.
template <typename T, bool WIDE> __device__ __forceinline__ typename Raw<T>::Two load_two(const T *p, bool both) {
    if (WIDE) return *reinterpret_cast<const typename Raw<T>::Two *>(p);
    return two_of<T>(load_one(p), both ? load_one(p + 1) : 0);
}
template <typename T, bool WIDE> __device__ __forceinline__ void store_two(T *p, bool both, Pair v) {
    if (WIDE) {
        Vec<T, 2> q;
        q.v[0] = from_f32<T>(v.lo()), q.v[1] = from_f32<T>(v.hi());
        *reinterpret_cast<Vec<T, 2> *>(p) = q;
        return;
    }
    p[0] = from_f32<T>(v.lo());
    if (both) p[1] = from_f32<T>(v.hi());
}

// A warp's lanes take neighbouring pairs of channels, a thread goes along its strip of positions with the last K inputs
// in registers.  What bounds it is how much is on its way from memory: loads run a batch of eight positions ahead, and
// two channels a thread leave registers for many warps (8 x 4096 x 2048 in bf16, K = 4: with eight channels a thread and
// four positions ahead the forward took 86 us, with four channels the backward 247 us).
constexpr int kCausalAhead = 8;

// What a thread of the tokens' kernels works on.
template <typename T, int K> struct Strip {
    int b, c, first, end, length, stop;
    bool both;  // whether the pair's second channel is one
    Pair w[K], bias;
    // false: nothing
    __device__ __forceinline__ bool find(const CausalArgs &a) {
        const int columns = (a.s.C + 63) / 64, groups = (a.strips + 7) / 8;
        const int strip = blockIdx.x / columns % groups * 8 + threadIdx.x / 32;
        b = blockIdx.x / columns / groups, c = (blockIdx.x % columns * 32 + threadIdx.x % 32) * 2;
        both = c + 1 < a.s.C;
        if (strip >= a.strips || c >= a.s.C) return false;
        first = strip * a.strip, end = min(first + a.strip, a.s.T), length = length_of(a, b), stop = min(end, length);
        const int c1 = both ? c + 1 : c;
        bias = a.bias == nullptr ? Pair(0.f) : Pair(a.bias[c], a.bias[c1]);
#pragma unroll
        for (int k = 0; k < K; ++k) w[k] = Pair(a.w[(long long)c * K + k], a.w[(long long)c1 * K + k]);
        return true;
    }
    __device__ __forceinline__ Pair sum(const Pair *in) const {
        Pair v = bias;
#pragma unroll
        for (int k = 0; k < K; ++k) v = fma(w[k], in[k], v);
        return v;
    }
    // the K-1 inputs before the strip
    __device__ __forceinline__ void before(const CausalArgs &a, Pair (&in)[K - 1]) const {
#pragma unroll
        for (int k = 0; k < K - 1; ++k) {
            const int t = first - K + 1 + k;
            in[k] = Pair(input_at<T, K>(a, b, c, t), both ? input_at<T, K>(a, b, c + 1, t) : 0.f);
        }
    }
};

template <typename T, int K, bool WIDE, bool SILU> __global__ void __launch_bounds__(256) causal_tokens_forward_kernel(const __grid_constant__ CausalArgs a) {
    constexpr int AHEAD = kCausalAhead;
    using Two = typename Raw<T>::Two;
    begin_kernel();
    const unsigned main = (unsigned)a.s.B * ((a.strips + 7) / 8) * ((a.s.C + 63) / 64);
    if (blockIdx.x >= main) return write_state_last<T, K>(a, (long long)(blockIdx.x - main) * 256 + threadIdx.x);
    Strip<T, K> s;
    if (!s.find(a)) return;
    const T *const x = static_cast<const T *>(a.x.p) + s.b * a.x.batch + s.c;
    T *const y = static_cast<T *>(a.y.p) + s.b * a.y.batch + s.c;
    if (s.first < s.stop) {
        // (all of a batch's positions at once where they are the strip's: its checks are a third of the instructions)
        const auto fetch = [&](int t0, Two(&v)[AHEAD]) {
            const T *p = x + t0 * a.x.row;
            if (t0 + AHEAD <= s.stop) {
#pragma unroll
                for (int j = 0; j < AHEAD; ++j) v[j] = load_two<T, WIDE>(p + j * a.x.row, s.both);
            } else {
#pragma unroll
                for (int j = 0; j < AHEAD; ++j)
                    if (t0 + j < s.stop) v[j] = load_two<T, WIDE>(p + j * a.x.row, s.both);
            }
        };
        Two even[AHEAD] = {}, odd[AHEAD] = {};
        fetch(s.first, even);
        Pair window[K - 1];
        s.before(a, window);
        const auto batch = [&](int t0, Two(&now)[AHEAD], Two(&next)[AHEAD]) {
            fetch(t0 + AHEAD, next);
            arrived(now);
            Pair in[K - 1 + AHEAD];
#pragma unroll
            for (int k = 0; k < K - 1; ++k) in[k] = window[k];
#pragma unroll
            for (int j = 0; j < AHEAD; ++j) in[K - 1 + j] = pair_of<T>(now[j]);
            T *const to = y + t0 * a.y.row;
            if (t0 + AHEAD <= s.stop) {
#pragma unroll
                for (int j = 0; j < AHEAD; ++j) store_two<T, WIDE>(to + j * a.y.row, s.both, causal_f<SILU>(s.sum(in + j)));
            } else {
#pragma unroll
                for (int j = 0; j < AHEAD; ++j)
                    if (t0 + j < s.stop) store_two<T, WIDE>(to + j * a.y.row, s.both, causal_f<SILU>(s.sum(in + j)));
            }
#pragma unroll
            for (int k = 0; k < K - 1; ++k) window[k] = in[AHEAD + k];
        };
        for (int t0 = s.first; t0 < s.stop; t0 += 2 * AHEAD) {
            batch(t0, even, odd);
            if (t0 + AHEAD < s.stop) batch(t0 + AHEAD, odd, even);
        }
    }
    for (int t = max(s.first, s.length); t < s.end; ++t) store_two<T, WIDE>(y + t * a.y.row, s.both, Pair(0.f));
}

// The strip's K-1 following positions are computed too, for the gradients of its own inputs; dw and d_bias count
// the strip's own positions.
template <typename T, int K, bool WIDE, bool SILU> __global__ void __launch_bounds__(256) causal_tokens_backward_kernel(const __grid_constant__ CausalArgs a) {
    constexpr int AHEAD = kCausalAhead;
    using Two = typename Raw<T>::Two;
    __shared__ float meet[8][K + 1][64];
    begin_kernel();
    const int columns = (a.s.C + 63) / 64;
    const unsigned main = (unsigned)a.s.B * ((a.strips + 7) / 8) * columns;
    if (blockIdx.x >= main) return write_d_state<T, K>(a, (long long)(blockIdx.x - main) * 256 + threadIdx.x);
    Pair dw[K], db(0.f);
#pragma unroll
    for (int k = 0; k < K; ++k) dw[k] = Pair(0.f);
    Strip<T, K> s;
    if (s.find(a)) {
        const int beyond = min(s.end + K - 1, s.length);  // the last position that reaches the strip
        const T *const x = static_cast<const T *>(a.x.p) + s.b * a.x.batch + s.c, *const dy = static_cast<const T *>(a.dy.p) + s.b * a.dy.batch + s.c;
        T *const dx = static_cast<T *>(a.dx.p) + s.b * a.dx.batch + s.c;
        if (s.first < s.stop) {
            struct Fetched {
                Two x[AHEAD], dy[AHEAD];
            } even = {}, odd = {};
            const auto fetch = [&](int t0, Fetched &f) {
                const T *const p = x + t0 * a.x.row, *const q = dy + t0 * a.dy.row;
                if (t0 + AHEAD <= beyond) {
#pragma unroll
                    for (int j = 0; j < AHEAD; ++j) f.x[j] = load_two<T, WIDE>(p + j * a.x.row, s.both), f.dy[j] = load_two<T, WIDE>(q + j * a.dy.row, s.both);
                    return;
                }
#pragma unroll
                for (int j = 0; j < AHEAD; ++j)
                    if (t0 + j < beyond) f.x[j] = load_two<T, WIDE>(p + j * a.x.row, s.both), f.dy[j] = load_two<T, WIDE>(q + j * a.dy.row, s.both);
            };
            fetch(s.first, even);
            Pair window[K - 1], slopes[K - 1];
            s.before(a, window);
#pragma unroll
            for (int k = 0; k < K - 1; ++k) slopes[k] = Pair(0.f);
            const auto batch = [&](int t0, Fetched &now, Fetched &next) {
                fetch(t0 + AHEAD, next);
                arrived(now.x), arrived(now.dy);
                Pair in[K - 1 + AHEAD], slope[K - 1 + AHEAD];
#pragma unroll
                for (int k = 0; k < K - 1; ++k) in[k] = window[k], slope[k] = slopes[k];
                T *const to = dx + (t0 - K + 1) * a.dx.row;
                const auto positions = [&](auto full) {
                    constexpr bool FULL = decltype(full)::value;
#pragma unroll
                    for (int j = 0; j < AHEAD; ++j) {
                        const int t = t0 + j, own = t - K + 1;  // the input whose last reader t is
                        in[K - 1 + j] = pair_of<T>(now.x[j]);
                        const Pair g = mul(pair_of<T>(now.dy[j]), causal_slope<SILU>(s.sum(in + j)));
                        slope[K - 1 + j] = FULL || t < beyond ? g : Pair(0.f);
                        if (FULL || t < s.stop) {
                            db = add(db, g);
#pragma unroll
                            for (int k = 0; k < K; ++k) dw[k] = fma(g, in[j + k], dw[k]);
                        }
                        if (!FULL && (own < s.first || own >= s.stop)) continue;
                        Pair v(0.f);
#pragma unroll
                        for (int k = 0; k < K; ++k) v = fma(s.w[K - 1 - k], slope[j + k], v);
                        if (!FULL && a.d_last != nullptr && own >= s.length - K + 1) {
                            const T *const last = static_cast<const T *>(a.d_last) + ((long long)s.b * a.s.C + s.c) * (K - 1) + own - (s.length - K + 1);
                            v = add(v, Pair(to_f32(last[0]), s.both ? to_f32(last[K - 1]) : 0.f));
                        }
                        store_two<T, WIDE>(to + j * a.dx.row, s.both, v);
                    }
                };
                // whole batches of the strip's own positions whose inputs are its own too; the last state's inputs (K-1 before
                // the end) come with the batch after them
                if (t0 >= s.first + K - 1 && t0 + AHEAD <= s.stop) positions(std::true_type{});
                else positions(std::false_type{});
#pragma unroll
                for (int k = 0; k < K - 1; ++k) window[k] = in[AHEAD + k], slopes[k] = slope[AHEAD + k];
            };
            for (int t0 = s.first; t0 < s.stop + K - 1; t0 += 2 * AHEAD) {
                batch(t0, even, odd);
                if (t0 + AHEAD < s.stop + K - 1) batch(t0 + AHEAD, odd, even);
            }
        }
        for (int t = max(s.first, s.length); t < s.end; ++t) store_two<T, WIDE>(dx + t * a.dx.row, s.both, Pair(0.f));
    }
    // over the CTA's strips
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, part = blockIdx.x / columns;
#pragma unroll
    for (int k = 0; k <= K; ++k) {
        const Pair v = k == K ? db : dw[k == K ? 0 : k];
        meet[warp][k][2 * lane] = v.lo(), meet[warp][k][2 * lane + 1] = v.hi();
    }
    __syncthreads();
    for (int e = threadIdx.x; e < 64 * (K + 1); e += 256) {
        const int k = e / 64, to = blockIdx.x % columns * 64 + e % 64;
        float v = 0.f;
#pragma unroll
        for (int m = 0; m < 8; ++m) v += meet[m][k][e % 64];
        if (to >= a.s.C) continue;
        if (k == K) a.part_b[(long long)part * a.s.C + to] = v;
        else a.part_w[((long long)part * a.s.C + to) * K + k] = v;
    }
}

// --------------------------------------------------------------------------------------- planes

// f or its slope of COUNT values, two at a time.
template <bool SLOPE, bool SILU, int COUNT> __device__ __forceinline__ void causal_map(float (&v)[COUNT]) {
#pragma unroll
    for (int i = 0; i < COUNT; i += 2) {
        const Pair p(v[i], v[i + 1 < COUNT ? i + 1 : i]), q = SLOPE ? causal_slope<SILU>(p) : causal_f<SILU>(p);
        v[i] = q.lo();
        if (i + 1 < COUNT) v[i + 1] = q.hi();
    }
}

// Positions [t0 - BEFORE, t0 + V + AFTER) of a row, 0 past `length`, the state before position 0.  Inside the row the
// vectors beside t0's come whole, from the first-level cache.
template <typename T, int K, int V, int BEFORE, int AFTER>
__device__ __forceinline__ void load_around(const CausalArgs &a, const T *row, int b, int c, int t0, int length, float (&v)[BEFORE + V + AFTER]) {
    if (V > 1 && (BEFORE == 0 || t0 >= V) && t0 + V + (AFTER > 0 ? V : 0) <= length) {
        float q[V];
        if (BEFORE > 0) {
            load_vec<T, V>(row + t0 - V, q);
#pragma unroll
            for (int i = 0; i < BEFORE; ++i) v[i] = q[V - BEFORE + i];
        }
        load_vec<T, V>(row + t0, q);
#pragma unroll
        for (int i = 0; i < V; ++i) v[BEFORE + i] = q[i];
        if (AFTER > 0) {
            load_vec<T, V>(row + t0 + V, q);
#pragma unroll
            for (int i = 0; i < AFTER; ++i) v[BEFORE + V + i] = q[i];
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < BEFORE + V + AFTER; ++i) {
        const int t = t0 - BEFORE + i;
        v[i] = t >= 0 ? (t < length ? to_f32(row[t]) : 0.f) : input_at<T, K>(a, b, c, t);
    }
}
template <typename T, int V> __device__ __forceinline__ void store_some(T *row, int t0, int T_, const float (&v)[V]) {
    if (t0 + V <= T_) return store_vec<T, V>(row + t0, v);
#pragma unroll
    for (int i = 0; i < V; ++i)
        if (t0 + i < T_) row[t0 + i] = from_f32<T>(v[i]);
}

// 2^row_bits neighbouring lanes go along a strip of a row, a vector of positions each.
struct RowStrip {
    bool used;
    int b, c, row, strip, lane, lanes, length, first, end;
    __device__ __forceinline__ explicit RowStrip(const CausalArgs &a) {
        const int per = 256 >> a.row_bits;  // strips of a CTA
        const long long unit = (long long)blockIdx.x * per + (threadIdx.x >> a.row_bits);
        used = unit < (long long)a.s.B * a.s.C * a.strips;
        lanes = 1 << a.row_bits, lane = threadIdx.x & (lanes - 1);
        row = used ? (int)(unit / a.strips) : 0, strip = used ? (int)(unit % a.strips) : 0;
        b = row / a.s.C, c = row % a.s.C, length = length_of(a, b);
        first = strip * a.strip, end = used ? min(first + a.strip, a.s.T) : 0;
    }
    static __device__ __forceinline__ unsigned ctas(const CausalArgs &a) {
        const int per = 256 >> a.row_bits;
        return (unsigned)(((long long)a.s.B * a.s.C * a.strips + per - 1) / per);
    }
};

template <typename T, int K, int V, bool SILU> __global__ void __launch_bounds__(256) causal_planes_forward_kernel(const __grid_constant__ CausalArgs a) {
    begin_kernel();
    const unsigned main = RowStrip::ctas(a);
    if (blockIdx.x >= main) return write_state_last<T, K>(a, (long long)(blockIdx.x - main) * 256 + threadIdx.x);
    const RowStrip s(a);
    const T *x = static_cast<const T *>(a.x.p) + s.b * a.x.batch + s.c * a.x.row;
    T *y = static_cast<T *>(a.y.p) + s.b * a.y.batch + s.c * a.y.row;
    float w[K];
#pragma unroll
    for (int k = 0; k < K; ++k) w[k] = a.w[(long long)s.c * K + k];
    const float bias = a.bias == nullptr ? 0.f : a.bias[s.c];
    for (int t0 = s.first + s.lane * V; t0 < s.end; t0 += s.lanes * V) {
        float v[V] = {};
        if (t0 < s.length) {
            float in[K - 1 + V];
            load_around<T, K, V, K - 1, 0>(a, x, s.b, s.c, t0, s.length, in);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                v[i] = bias;
#pragma unroll
                for (int k = 0; k < K; ++k) v[i] = fmaf(w[k], in[i + k], v[i]);
            }
            causal_map<false, SILU>(v);
#pragma unroll
            for (int i = 0; i < V; ++i) v[i] = t0 + i < s.length ? v[i] : 0.f;
        }
        store_some<T, V>(y, t0, a.s.T, v);
    }
}

template <typename T, int K, int V, bool SILU> __global__ void __launch_bounds__(256) causal_planes_backward_kernel(const __grid_constant__ CausalArgs a) {
    begin_kernel();
    const unsigned main = RowStrip::ctas(a);
    if (blockIdx.x >= main) return write_d_state<T, K>(a, (long long)(blockIdx.x - main) * 256 + threadIdx.x);
    const RowStrip s(a);
    const T *x = static_cast<const T *>(a.x.p) + s.b * a.x.batch + s.c * a.x.row, *dy = static_cast<const T *>(a.dy.p) + s.b * a.dy.batch + s.c * a.dy.row;
    T *dx = static_cast<T *>(a.dx.p) + s.b * a.dx.batch + s.c * a.dx.row;
    float w[K], dw[K] = {}, db = 0.f;
#pragma unroll
    for (int k = 0; k < K; ++k) w[k] = a.w[(long long)s.c * K + k];
    const float bias = a.bias == nullptr ? 0.f : a.bias[s.c];
    for (int t0 = s.first + s.lane * V; t0 < s.end; t0 += s.lanes * V) {
        float v[V] = {};
        if (t0 < s.length) {
            float in[V + 2 * (K - 1)], g[V + K - 1], slope[V + K - 1];  // inputs from t0 - (K-1) on, gradients from t0 on
            load_around<T, K, V, K - 1, K - 1>(a, x, s.b, s.c, t0, s.length, in);
            load_around<T, K, V, 0, K - 1>(a, dy, s.b, s.c, t0, s.length, g);
#pragma unroll
            for (int i = 0; i < V + K - 1; ++i) {
                slope[i] = bias;
#pragma unroll
                for (int k = 0; k < K; ++k) slope[i] = fmaf(w[k], in[i + k], slope[i]);
            }
            causal_map<true, SILU>(slope);
#pragma unroll
            for (int i = 0; i < V + K - 1; ++i) {
                g[i] = t0 + i < s.length ? g[i] * slope[i] : 0.f;
                if (i >= V || t0 + i >= s.length) continue;  // (past the length: inputs before it may be infinite, 0 times them is not 0)
                db += g[i];
#pragma unroll
                for (int k = 0; k < K; ++k) dw[k] = fmaf(g[i], in[i + k], dw[k]);
            }
#pragma unroll
            for (int i = 0; i < V; ++i)
#pragma unroll
                for (int k = 0; k < K; ++k) v[i] = fmaf(w[K - 1 - k], g[i + k], v[i]);
            if (t0 + V > s.length - K + 1) {  // the end: inputs that the last state holds, and none past it
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const int t = t0 + i;
                    if (t >= s.length) v[i] = 0.f;
                    else if (a.d_last != nullptr && t >= s.length - K + 1)
                        v[i] += to_f32(static_cast<const T *>(a.d_last)[(long long)s.row * (K - 1) + t - (s.length - K + 1)]);
                }
            }
        }
        store_some<T, V>(dx, t0, a.s.T, v);
    }
    const long long part = (long long)s.b * a.strips + s.strip;
#pragma unroll
    for (int k = 0; k <= K; ++k) {
        float v = k == K ? db : dw[k == K ? 0 : k];
        for (int m = s.lanes / 2; m >= 1; m /= 2) v += __shfl_xor_sync(0xffffffffu, v, m);
        if (s.used && s.lane == 0) {
            if (k == K) a.part_b[part * a.s.C + s.c] = v;
            else a.part_w[(part * a.s.C + s.c) * K + k] = v;
        }
    }
}

// ---------------------------------------------------------------------------------------- launch

template <bool BACKWARD, typename T, int K, bool WIDE> cudaError_t launch_causal_as(const CausalArgs &a, cudaStream_t st) {
    const bool planes = a.s.layout == WTCONV_SCAN_PLANES, ends = BACKWARD ? a.d_state != nullptr : a.state_last != nullptr;
    const long long rows = (long long)a.s.B * a.s.C;
    long long grid = planes ? (rows * a.strips + (256 >> a.row_bits) - 1) / (256 >> a.row_bits)
                            : (long long)a.s.B * ceil_div(a.strips, 8) * ceil_div(a.s.C, 64);
    if (ends) grid += (rows + 255) / 256;
    if (grid > 0x7fffffffll) return cudaErrorInvalidValue;
    const auto launch = [&](auto kernel) { return launch_kernel(kernel, (unsigned)grid, 256, 0, st, 1, a); };
    if constexpr (BACKWARD) {
        constexpr int V = WIDE ? 4 : 1;
        if (planes) return a.s.silu ? launch(causal_planes_backward_kernel<T, K, V, true>) : launch(causal_planes_backward_kernel<T, K, V, false>);
        return a.s.silu ? launch(causal_tokens_backward_kernel<T, K, WIDE, true>) : launch(causal_tokens_backward_kernel<T, K, WIDE, false>);
    } else {
        constexpr int V = WIDE ? 16 / sizeof(T) : 1;
        if (planes) return a.s.silu ? launch(causal_planes_forward_kernel<T, K, V, true>) : launch(causal_planes_forward_kernel<T, K, V, false>);
        return a.s.silu ? launch(causal_tokens_forward_kernel<T, K, WIDE, true>) : launch(causal_tokens_forward_kernel<T, K, WIDE, false>);
    }
}
template <bool BACKWARD, typename T, bool WIDE> cudaError_t launch_causal_taps(const CausalArgs &a, cudaStream_t st) {
    return a.s.K == 2   ? launch_causal_as<BACKWARD, T, 2, WIDE>(a, st)
           : a.s.K == 3 ? launch_causal_as<BACKWARD, T, 3, WIDE>(a, st)
                        : launch_causal_as<BACKWARD, T, 4, WIDE>(a, st);
}

template <typename T> cudaError_t launch_causal_forward(const CausalArgs &a, cudaStream_t st) {
    return a.wide ? launch_causal_taps<false, T, true>(a, st) : launch_causal_taps<false, T, false>(a, st);
}
template <typename T> cudaError_t launch_causal_backward(const CausalArgs &a, cudaStream_t st) {
    const cudaError_t e = a.wide ? launch_causal_taps<true, T, true>(a, st) : launch_causal_taps<true, T, false>(a, st);
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
