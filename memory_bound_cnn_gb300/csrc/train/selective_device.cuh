// Arithmetic and tiles of the selective scan (wtconv_ssm.h).
#pragma once

#include "selective.h"
#include "train_device.cuh"

namespace wtconv {

constexpr float kSelLog2E = 1.4426950408889634f, kSelLn2 = 0.6931471805599453f;

__device__ __forceinline__ float exp2_fast(float v) {  // to about two units of the last place
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}
// The same, computed where it stands: otherwise the compiler keeps a block's 64 decays from the way forward for
// the way back, more registers than there are.
__device__ __forceinline__ float exp2_again(float v) {
    float r;
    asm volatile("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}
__device__ __forceinline__ Pair exp2_again(Pair v) { return {exp2_again(v.lo()), exp2_again(v.hi())}; }
__device__ __forceinline__ Pair exp2_fast(Pair v) { return {exp2_fast(v.lo()), exp2_fast(v.hi())}; }

// softplus(v) = max(v, 0) + log(1 + e) with e = exp(-|v|) in (0, 1]: nothing cancels.  With s = e / (2 + e)
// <= 1/3, log(1 + e) = 2 artanh s = 2 (s + s^3/3 + ... + s^13/13); the next term is 1.4e-8 of the value.
// slope: sigmoid(v), from the same e.
struct Softplus {
    float value, slope;
};
__device__ __forceinline__ Softplus softplus_of(float v) {
    const float e = exp2_fast(-kSelLog2E * fabsf(v));
    const float s = e * reciprocal(2.f + e), q = s * s;
    float p = 1.f / 13;
    p = fmaf(p, q, 1.f / 11), p = fmaf(p, q, 1.f / 9), p = fmaf(p, q, 1.f / 7);
    p = fmaf(p, q, 1.f / 5), p = fmaf(p, q, 1.f / 3), p = fmaf(p, q, 1.f);
    const float r = reciprocal(1.f + e);
    return {fmaxf(v, 0.f) + 2.f * s * p, v >= 0.f ? r : e * r};
}
__device__ __forceinline__ float sigmoid_of(float v) { return reciprocal(1.f + exp2_fast(-kSelLog2E * v)); }

// Element (position, channel) of an activation.
template <typename T, bool PLANES>
__device__ __forceinline__ T *at(const wtconv_ssm_tensor &t, int b, int position, int channel) {
    const long long outer = PLANES ? channel : position, inner = PLANES ? position : channel;
    return static_cast<T *>(t.p) + b * t.batch + outer * t.row + inner;
}

// Sums v[0..COUNT) over the lanes that differ in the COUNT * FIRST ... bits: lanes FIRST, 2 FIRST, ... apart
// exchange halves, so that COUNT sums over COUNT lanes take COUNT - 1 exchanges.  A lane ends with the sum
// of v[i] in v[0], i its index among the COUNT lanes.
template <int COUNT, int FIRST> __device__ __forceinline__ void sum_exchange(float (&v)[COUNT], int index) {
#pragma unroll
    for (int w = COUNT / 2; w >= 1; w /= 2) {
        const bool upper = index & w;
#pragma unroll
        for (int j = 0; j < w; ++j) {
            const float send = upper ? v[j] : v[j + w], keep = upper ? v[j + w] : v[j];
            v[j] = keep + __shfl_xor_sync(0xffffffffu, send, w * FIRST);
        }
    }
}

// What a CTA works on: a tile of channels of one group, a segment of one sequence.
struct Place {
    int b, group, c0, channels, tile, segment, first, end, length;
    __device__ __forceinline__ Place(const SelectiveArgs &a, unsigned block) {
        // (tiles innermost: the CTAs that read the same B and C run together)
        tile = block % (a.s.G * a.tiles);
        const unsigned rest = block / (a.s.G * a.tiles);
        segment = rest % a.segments, b = rest / a.segments;
        group = tile / a.tiles;
        const int c = tile % a.tiles * kSelTile;
        c0 = group * a.channels + c, channels = min(kSelTile, a.channels - c);
        length = a.in.lengths == nullptr ? a.s.T : min(max(a.in.lengths[b], 0), a.s.T);
        first = segment * a.segment;
        end = min(first + a.segment, a.s.T);  // (segment * segments < 2^31: segments are at most 256 rounds more than T)
    }
};

// Four neighbouring states of a channel's N in memory of fp32: the lane's are n0 to n0 + 3; those past N are 0.
struct Quad {
    Pair a, b;
};
__device__ __forceinline__ Quad load_quad(const float *row, int n0, int N) {
    const float v0 = n0 < N ? row[n0] : 0.f, v1 = n0 + 1 < N ? row[n0 + 1] : 0.f;
    const float v2 = n0 + 2 < N ? row[n0 + 2] : 0.f, v3 = n0 + 3 < N ? row[n0 + 3] : 0.f;
    return {Pair(v0, v1), Pair(v2, v3)};
}
__device__ __forceinline__ void store_quad(float *row, int n0, int N, const Quad &q) {
    if (n0 < N) row[n0] = q.a.lo();
    if (n0 + 1 < N) row[n0 + 1] = q.a.hi();
    if (n0 + 2 < N) row[n0 + 2] = q.b.lo();
    if (n0 + 3 < N) row[n0 + 3] = q.b.hi();
}
__device__ __forceinline__ Quad quad_of(const float4 &v) { return {Pair(v.x, v.y), Pair(v.z, v.w)}; }
__device__ __forceinline__ float4 float4_of(const Quad &q) { return make_float4(q.a.lo(), q.a.hi(), q.b.lo(), q.b.hi()); }
__device__ __forceinline__ float sum_of(const Quad &q) {
    const Pair s = add(q.a, q.b);
    return s.lo() + s.hi();
}

}  // namespace wtconv
