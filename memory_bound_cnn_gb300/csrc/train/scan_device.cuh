// Arithmetic of the gated scan (wtconv_scan.h) and its loads and stores.
#pragma once

#include "scan.h"
#include "train_device.cuh"

namespace wtconv {

// Gates of two elements: a = sigmoid(z) and b = 1 - a, both to a few units of their own last place.
// With e = exp(-z), a = 1 / (1 + e) and b = e a: nothing cancels.  e is held below 2^100, where a has
// long been 0 to fp32's eyes beside any h that matters (2^-100) and b is 1.  A NaN comes through.
struct Gates {
    Pair a, b;
};
constexpr float kLog2E = 1.4426950408889634f;
__device__ __forceinline__ float exp2_of(float v) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}
__device__ __forceinline__ float capped(float e) {  // min(e, 2^100), or NaN
    float r;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(e), "f"(1.2676506002282294e30f));
    return r;
}
__device__ __forceinline__ Gates gates_of_exp(Pair e) {
    const Pair d = add(e, Pair(1.f));
    Gates g;
    g.a = Pair(reciprocal(d.lo()), reciprocal(d.hi()));
    g.b = mul(e, g.a);
    return g;
}
// bias: minus the channels' gate_bias, times log2 e
__device__ __forceinline__ Gates gates_of(Pair gate, Pair bias) {
    const Pair w = fma(gate, Pair(-kLog2E), bias);
    return gates_of_exp(Pair(capped(exp2_of(w.lo())), capped(exp2_of(w.hi()))));
}

// Two 16-bit elements of a word as fp32, and back (rounded to nearest).
template <typename T> __device__ __forceinline__ Pair widen(uint32_t w);
template <> __device__ __forceinline__ Pair widen<__nv_bfloat16>(uint32_t w) {
    return {__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u)};
}
template <> __device__ __forceinline__ Pair widen<__half>(uint32_t w) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w));
    return {f.x, f.y};
}
template <typename T> __device__ __forceinline__ uint32_t narrow(Pair v);
template <> __device__ __forceinline__ uint32_t narrow<__nv_bfloat16>(Pair v) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(v.lo(), v.hi());
    return *reinterpret_cast<const uint32_t *>(&h);
}
template <> __device__ __forceinline__ uint32_t narrow<__half>(Pair v) {
    const __half2 h = __floats2half2_rn(v.lo(), v.hi());
    return *reinterpret_cast<const uint32_t *>(&h);
}

// length of sequence b, clipped to [0, T]
__device__ __forceinline__ int scan_length(const int *lengths, int b, int T) {
    if (lengths == nullptr) return T;
    const int n = lengths[b];
    return n < 0 ? 0 : (n < T ? n : T);
}

// A stretch of the recurrence as the map h -> a h + u of the state before it; `then` appends the
// stretch that follows.
struct Span {
    float a, u;
    __device__ __forceinline__ Span then(Span next) const { return {a * next.a, fmaf(next.a, u, next.u)}; }
    __device__ __forceinline__ float of(float h) const { return fmaf(a, h, u); }
};

// Inclusive scan of spans over groups of WIDTH lanes: forward (lane l ends with lanes 0..l), or
// backward (lanes WIDTH-1 down to l).
template <int WIDTH, bool BACKWARD> __device__ __forceinline__ Span warp_scan(Span s, int lane) {
#pragma unroll
    for (int d = 1; d < WIDTH; d <<= 1) {
        Span o;
        o.a = BACKWARD ? __shfl_down_sync(0xffffffffu, s.a, d, WIDTH) : __shfl_up_sync(0xffffffffu, s.a, d, WIDTH);
        o.u = BACKWARD ? __shfl_down_sync(0xffffffffu, s.u, d, WIDTH) : __shfl_up_sync(0xffffffffu, s.u, d, WIDTH);
        const int l = lane & (WIDTH - 1);
        if (BACKWARD ? l + d < WIDTH : l >= d) s = o.then(s);
    }
    return s;
}
// The scan's result of the lane before (after, if BACKWARD): the identity for the first.
template <int WIDTH, bool BACKWARD> __device__ __forceinline__ Span lane_before(Span s, int lane) {
    Span o;
    o.a = BACKWARD ? __shfl_down_sync(0xffffffffu, s.a, 1, WIDTH) : __shfl_up_sync(0xffffffffu, s.a, 1, WIDTH);
    o.u = BACKWARD ? __shfl_down_sync(0xffffffffu, s.u, 1, WIDTH) : __shfl_up_sync(0xffffffffu, s.u, 1, WIDTH);
    const int l = lane & (WIDTH - 1);
    if (BACKWARD ? l == WIDTH - 1 : l == 0) o = {1.f, 0.f};
    return o;
}

// Eight consecutive elements as raw words, and as fp32.
template <typename T> struct Eight {
    uint32_t w[2 * sizeof(T)];
    __device__ __forceinline__ float get(int j) const {
        if constexpr (sizeof(T) == 4) return __uint_as_float(w[j]);
        else {
            const uint16_t h = (uint16_t)(w[j >> 1] >> (16 * (j & 1)));
            return to_f32(*reinterpret_cast<const T *>(&h));
        }
    }
    __device__ __forceinline__ void set(int j, float a, float b) {  // elements j (even) and j + 1
        if constexpr (sizeof(T) == 4) {
            w[j] = __float_as_uint(a), w[j + 1] = __float_as_uint(b);
        } else {
            const T lo = from_f32<T>(a), hi = from_f32<T>(b);
            w[j >> 1] = (uint32_t)*reinterpret_cast<const uint16_t *>(&lo) |
                        (uint32_t)*reinterpret_cast<const uint16_t *>(&hi) << 16;
        }
    }
    // elements 0 .. valid-1 from p (all of them: vectors if VEC); the rest zeros
    template <bool VEC> __device__ __forceinline__ void load(const T *p, int valid) {
        if (VEC && valid >= 8) {
#pragma unroll
            for (int k = 0; k < (int)sizeof(T) / 2; ++k) {
                const uint4 q = __ldg(reinterpret_cast<const uint4 *>(p) + k);
                w[4 * k] = q.x, w[4 * k + 1] = q.y, w[4 * k + 2] = q.z, w[4 * k + 3] = q.w;
            }
            return;
        }
#pragma unroll
        for (int k = 0; k < 2 * (int)sizeof(T); ++k) w[k] = 0;
        if (valid <= 0) return;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            if (j >= valid) continue;
            if constexpr (sizeof(T) == 4) w[j] = __float_as_uint(p[j]);
            else w[j >> 1] |= (uint32_t)*reinterpret_cast<const uint16_t *>(p + j) << (16 * (j & 1));
        }
    }
    template <bool VEC> __device__ __forceinline__ void store(T *p, int valid) const {
        if (VEC && valid >= 8) {
#pragma unroll
            for (int k = 0; k < (int)sizeof(T) / 2; ++k)
                reinterpret_cast<uint4 *>(p)[k] = make_uint4(w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]);
            return;
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            if (j >= valid) continue;
            if constexpr (sizeof(T) == 4) p[j] = __uint_as_float(w[j]);
            else *reinterpret_cast<uint16_t *>(p + j) = (uint16_t)(w[j >> 1] >> (16 * (j & 1)));
        }
    }
};

}  // namespace wtconv
