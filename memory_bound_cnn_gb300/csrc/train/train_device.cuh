// Element types and warp sums of the operators beside the WTConv layer.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace wtconv {

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }

template <typename T> __device__ __forceinline__ T from_f32(float v);
template <> __device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <> __device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }

// Two fp32 values that one instruction works on (each lane rounded as the plain instruction would).
struct Pair {
    unsigned long long q;
    __device__ __forceinline__ Pair() {}
    __device__ __forceinline__ Pair(float lo, float hi) { asm("mov.b64 %0, {%1, %2};" : "=l"(q) : "f"(lo), "f"(hi)); }
    __device__ __forceinline__ explicit Pair(float v) : Pair(v, v) {}
    __device__ __forceinline__ float lo() const {
        float a;
        asm("mov.b64 {%0, _}, %1;" : "=f"(a) : "l"(q));
        return a;
    }
    __device__ __forceinline__ float hi() const {
        float b;
        asm("mov.b64 {_, %0}, %1;" : "=f"(b) : "l"(q));
        return b;
    }
};
__device__ __forceinline__ Pair mul(Pair a, Pair b) {
    Pair r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.q) : "l"(a.q), "l"(b.q));
    return r;
}
__device__ __forceinline__ Pair add(Pair a, Pair b) {
    Pair r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.q) : "l"(a.q), "l"(b.q));
    return r;
}
__device__ __forceinline__ Pair sub(Pair a, Pair b) {
    Pair r;
    asm("sub.rn.f32x2 %0, %1, %2;" : "=l"(r.q) : "l"(a.q), "l"(b.q));
    return r;
}
__device__ __forceinline__ Pair add_down(Pair a, Pair b) {  // rounded towards minus infinity
    Pair r;
    asm("add.rm.f32x2 %0, %1, %2;" : "=l"(r.q) : "l"(a.q), "l"(b.q));
    return r;
}
__device__ __forceinline__ Pair fma(Pair a, Pair b, Pair c) {
    Pair r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.q) : "l"(a.q), "l"(b.q), "l"(c.q));
    return r;
}
// The product, rounded also where a sum follows: `add` of a `mul` is compiled to one fused
// multiply-add, whose product is not rounded.  zero holds -0, which changes no product, in a form
// the compiler cannot see through (a kernel's argument).
__device__ __forceinline__ Pair product(Pair a, Pair b, Pair zero) { return fma(a, b, zero); }
__device__ __forceinline__ Pair abs(Pair a) {
    Pair r;
    r.q = a.q & 0x7fffffff7fffffffull;
    return r;
}

__device__ __forceinline__ float reciprocal(float v) {  // to about one unit of the last place
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}
__device__ __forceinline__ float root_of(float v) {  // the same; below the least normal number: 0
    float r;
    asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

// First of all in every kernel: lets the next launch of the stream be set up, and waits until the one
// before has ended and its memory is visible.
__device__ __forceinline__ void begin_kernel() {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
}

template <typename V> __device__ __forceinline__ V warp_sum(V v) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
    return v;
}

}  // namespace wtconv
