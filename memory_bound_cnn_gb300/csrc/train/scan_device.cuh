// Arithmetic of the gated scan (wtconv_scan.h) and its loads and stores.
#pragma once

#include "scan.h"
#include "train_device.cuh"

namespace wtconv {

// Gates of two elements: a = sigmoid(z) and b = 1 - a.  With e = exp(-z), a = 1 / (1 + e) and b = e a:
// nothing cancels.  In units of 2^-24 of its own value e is off by up to 2.2 |z| + 4 (z is rounded, and so
// is its product with a rounded log2 e; the exponential itself: 4), which reaches a times b and b times a;
// the other operations add up to 4.  e is held below 2^100, where a has long been 0 to fp32's eyes beside
// any h that matters (2^-100) and b is 1.  A NaN comes through.
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
    const Pair d = fma(e, Pair(-1.f), Pair(-1.f));  // -(1 + e)
    Gates g;
    g.a = Pair(reciprocal(-d.lo()), reciprocal(-d.hi()));
    // one Newton step: a bias of the approximation would grow with the hundreds of positions that a
    // state remembers (a^n)
    g.a = fma(g.a, fma(d, g.a, Pair(1.f)), g.a);
    g.b = mul(e, g.a);
    return g;
}
// (The sum comes first: a bias scaled beforehand saves an instruction, but is rounded at its own size, the
// same way at every position.  With gates and biases of 20 to 60 that cancel, b was off by 58 units.)
__device__ __forceinline__ Gates gates_of(Pair gate, Pair bias) {
    const Pair w = mul(add(gate, bias), Pair(-kLog2E));
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

// Asynchronous copies of 16 or 4 bytes to shared memory, of which the first `bytes` are read and the
// rest come out as zeros.
template <int CP> __device__ __forceinline__ void copy_async(void *to, const void *from, int bytes) {
    const unsigned dst = (unsigned)__cvta_generic_to_shared(to);
    if constexpr (CP == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(from), "r"(bytes) : "memory");
    else asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(from), "r"(bytes) : "memory");
}
__device__ __forceinline__ void commit_copies() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int PENDING> __device__ __forceinline__ void wait_copies() {
    asm volatile("cp.async.wait_group %0;" ::"n"(PENDING) : "memory");
}

// A stretch of the recurrence as the map h -> a h + u of the state before it; `then` appends the
// stretch that follows.
struct Span {
    float a, u;
    __device__ __forceinline__ Span then(Span next) const { return {a * next.a, fmaf(next.a, u, next.u)}; }
    __device__ __forceinline__ float of(float h) const { return fmaf(a, h, u); }
};

// s gets the span of the lane `d` before (after, if BACKWARD) in its group of lanes put before it, if
// there is one.  The shuffle's own predicate guards the two products.  clamp: the shuffle's bounds.
template <bool BACKWARD> __device__ __forceinline__ void scan_step(Span &s, int d, int clamp) {
    if (BACKWARD)
        asm volatile("{\n\t.reg .f32 a, u;\n\t.reg .pred p;\n\t"
                     "shfl.sync.down.b32 a|p, %0, %2, %3, 0xffffffff;\n\t"
                     "shfl.sync.down.b32 u, %1, %2, %3, 0xffffffff;\n\t"
                     "@p fma.rn.f32 %1, %0, u, %1;\n\t@p mul.f32 %0, %0, a;\n\t}"
                     : "+f"(s.a), "+f"(s.u) : "r"(d), "r"(clamp));
    else
        asm volatile("{\n\t.reg .f32 a, u;\n\t.reg .pred p;\n\t"
                     "shfl.sync.up.b32 a|p, %0, %2, %3, 0xffffffff;\n\t"
                     "shfl.sync.up.b32 u, %1, %2, %3, 0xffffffff;\n\t"
                     "@p fma.rn.f32 %1, %0, u, %1;\n\t@p mul.f32 %0, %0, a;\n\t}"
                     : "+f"(s.a), "+f"(s.u) : "r"(d), "r"(clamp));
}
template <bool BACKWARD> __device__ __forceinline__ int scan_clamp(int width) {
    return (32 - width) << 8 | (BACKWARD ? 31 : 0);
}
// Inclusive scan of spans over groups of `width` lanes (a power of two): forward (lane l ends with
// lanes 0..l), or backward (lanes width-1 down to l).
template <bool BACKWARD> __device__ __forceinline__ Span warp_scan(Span s, int width) {
    const int clamp = scan_clamp<BACKWARD>(width);
#pragma unroll
    for (int d = 1; d < 32; d <<= 1)
        if (d < width) scan_step<BACKWARD>(s, d, clamp);
    return s;
}
// The scan's result of the lane before (after, if BACKWARD) in the group: the identity for the first.
template <bool BACKWARD> __device__ __forceinline__ Span lane_before(Span s, int width) {
    Span o = {1.f, 0.f};
    const int clamp = scan_clamp<BACKWARD>(width);
    if (BACKWARD)
        asm volatile("{\n\t.reg .f32 a, u;\n\t.reg .pred p;\n\t"
                     "shfl.sync.down.b32 a|p, %2, 1, %4, 0xffffffff;\n\t"
                     "shfl.sync.down.b32 u, %3, 1, %4, 0xffffffff;\n\t"
                     "@p mov.f32 %0, a;\n\t@p mov.f32 %1, u;\n\t}"
                     : "+f"(o.a), "+f"(o.u) : "f"(s.a), "f"(s.u), "r"(clamp));
    else
        asm volatile("{\n\t.reg .f32 a, u;\n\t.reg .pred p;\n\t"
                     "shfl.sync.up.b32 a|p, %2, 1, %4, 0xffffffff;\n\t"
                     "shfl.sync.up.b32 u, %3, 1, %4, 0xffffffff;\n\t"
                     "@p mov.f32 %0, a;\n\t@p mov.f32 %1, u;\n\t}"
                     : "+f"(o.a), "+f"(o.u) : "f"(s.a), "f"(s.u), "r"(clamp));
    return o;
}

}  // namespace wtconv
