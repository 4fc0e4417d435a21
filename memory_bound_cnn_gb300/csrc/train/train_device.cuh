// Element types and warp sums of the operators beside the WTConv layer.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <type_traits>

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
    __device__ __forceinline__ explicit Pair(unsigned long long both) : q(both) {}
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
// A pair of neighbours, and a single element, as they lie in memory.  What is fetched ahead stays a whole register in
// this form until it is used: packed or converted, it would have to arrive first.
template <typename T> struct Raw {
    using Two = typename std::conditional<sizeof(T) == 2, uint32_t, unsigned long long>::type;
};
template <typename T> __device__ __forceinline__ uint32_t load_one(const T *p) {
    if constexpr (sizeof(T) == 2) return *reinterpret_cast<const unsigned short *>(p);
    else return *reinterpret_cast<const uint32_t *>(p);
}
template <typename T> __device__ __forceinline__ typename Raw<T>::Two two_of(uint32_t first, uint32_t second) {
    if constexpr (sizeof(T) == 2) return first | second << 16;
    else return first | (unsigned long long)second << 32;
}
template <typename T> __device__ __forceinline__ Pair pair_of(typename Raw<T>::Two v) {
    if constexpr (std::is_same<T, float>::value) return Pair(v);
    else if constexpr (std::is_same<T, __half>::value) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&v));
        return {f.x, f.y};
    } else return {__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u)};
}
template <typename T> __device__ __forceinline__ float f32_of(uint32_t v) {
    if constexpr (std::is_same<T, float>::value) return __uint_as_float(v);
    else if constexpr (std::is_same<T, __half>::value) return __half2float(__ushort_as_half((unsigned short)v));
    else return __uint_as_float(v << 16);
}
// Where a fetched value is first used: the compiler would otherwise move what is done with it up to the load.
__device__ __forceinline__ void arrived(uint32_t &v) { asm volatile("" : "+r"(v)); }
__device__ __forceinline__ void arrived(unsigned long long &v) { asm volatile("" : "+l"(v)); }
template <typename V, int COUNT> __device__ __forceinline__ void arrived(V (&v)[COUNT]) {
#pragma unroll
    for (int i = 0; i < COUNT; ++i) arrived(v[i]);
}

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

// V neighbouring elements, in one access of up to 16 bytes (several where they are more).
template <typename T, int V> struct alignas(sizeof(T) * V > 16 ? 16 : sizeof(T) * V) Vec {
    T v[V];
};
template <typename T, int V> __device__ __forceinline__ void load_vec(const T *p, float (&to)[V]) {
    const Vec<T, V> q = *reinterpret_cast<const Vec<T, V> *>(p);
#pragma unroll
    for (int i = 0; i < V; ++i) to[i] = to_f32(q.v[i]);
}
template <typename T, int V> __device__ __forceinline__ void store_vec(T *p, const float (&from)[V]) {
    Vec<T, V> q;
#pragma unroll
    for (int i = 0; i < V; ++i) q.v[i] = from_f32<T>(from[i]);
    *reinterpret_cast<Vec<T, V> *>(p) = q;
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
