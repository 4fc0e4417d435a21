// AdamW step over a table of tensors (wtconv_optim.h).
//
// One CTA per chunk of 2048 elements of one tensor, one warp per 256 of them (a block of the 8-bit
// states), eight elements per lane in registers between the one read and the one write of each
// array.  With 32-bit states the step runs at the rate of a copy (100 M elements with bf16 gradients and
// a bf16 copy, 28 bytes each: 409 us, 6.8 TB/s).  With 8-bit states (130 M elements 451 us, 4.6 TB/s) neither
// HBM nor one unit is full: 102 instructions an element take 77 % of the issue slots, and the 64 registers
// that they need leave 45 % of an SM's warps to cover the loads, the largest stall.  A form with 88
// instructions and the same registers took as long (454 us), so issue alone does not bound it.
#include <cooperative_groups.h>
#include <float.h>

#include <utility>

#include "optim.h"
#include "train_device.cuh"

namespace wtconv {

namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 256, kNormThreads = 512, kNormCluster = 8;
constexpr uint32_t kIndexStride = 3242174889u;  // 2^32 / p, p^3 = p + 1
constexpr float kLeastMax = 8.077935669463161e-28f;  // 2^-90

// the table's tensor that holds chunk `chunk`
template <int CAP> __device__ __forceinline__ int find_tensor(const TensorTable<CAP> &table, int chunk) {
    int lo = 0, hi = table.count;  // first[lo] <= chunk < first[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (table.first[mid] <= chunk) lo = mid;
        else hi = mid;
    }
    return lo;
}

// Four consecutive elements from i on, those at or past n as zeros; vectors where VEC.
template <bool VEC> __device__ __forceinline__ void load4(const float *p, long long i, long long n, float (&v)[4]) {
    if (VEC && i + 4 <= n) {
        const float4 q = *reinterpret_cast<const float4 *>(p + i);
        v[0] = q.x, v[1] = q.y, v[2] = q.z, v[3] = q.w;
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = i + j < n ? p[i + j] : 0.f;
    }
}
template <bool VEC, typename T> __device__ __forceinline__ void load4(const T *p, long long i, long long n, float (&v)[4]) {
    if (VEC && i + 4 <= n) {
        uint2 q = *reinterpret_cast<const uint2 *>(p + i);
        const T *e = reinterpret_cast<const T *>(&q);
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = to_f32(e[j]);
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = i + j < n ? to_f32(p[i + j]) : 0.f;
    }
}
template <bool VEC> __device__ __forceinline__ void store4(float *p, long long i, long long n, const float (&v)[4]) {
    if (VEC && i + 4 <= n) *reinterpret_cast<float4 *>(p + i) = make_float4(v[0], v[1], v[2], v[3]);
    else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (i + j < n) p[i + j] = v[j];
    }
}
template <bool VEC, typename T> __device__ __forceinline__ void store4(T *p, long long i, long long n, const float (&v)[4]) {
    if (VEC && i + 4 <= n) {
        uint2 q;
        T *e = reinterpret_cast<T *>(&q);
#pragma unroll
        for (int j = 0; j < 4; ++j) e[j] = from_f32<T>(v[j]);
        *reinterpret_cast<uint2 *>(p + i) = q;
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (i + j < n) p[i + j] = from_f32<T>(v[j]);
    }
}
template <bool VEC> __device__ __forceinline__ uint32_t load_codes(const uint8_t *p, long long i, long long n) {
    if (VEC && i + 4 <= n) return *reinterpret_cast<const uint32_t *>(p + i);
    uint32_t q = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j)
        if (i + j < n) q |= (uint32_t)p[i + j] << (8 * j);
    return q;
}
template <bool VEC> __device__ __forceinline__ void store_codes(uint8_t *p, long long i, long long n, uint32_t q) {
    if (VEC && i + 4 <= n) *reinterpret_cast<uint32_t *>(p + i) = q;
    else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (i + j < n) p[i + j] = (uint8_t)(q >> (8 * j));
    }
}

// ------------------------------------------------------------------------- 8-bit states
// Products and sums that decide a code are rounded one by one (no fused multiply-add: `product`), so
// that a code is a function of its inputs that any fp32 program can follow.  Elements are worked on in pairs
// (Pair: one instruction for two), and bytes become fp32 and back through 2^23 + n, whose last bits are n:
// a conversion instruction runs at an eighth of the rate of an add, and the threshold's is the one that is
// left for an element.  130 M elements took 787 us one by one with conversions and exact square roots, 551 us
// without those.

constexpr float kTwo23 = 8388608.f;

// bytes j and j + 1 of a word, plus 2^23, as fp32
__device__ __forceinline__ Pair bytes_of(uint32_t q, int j) {
    return {__uint_as_float(__byte_perm(q, 0x4b000000u, 0x7540 | j)), __uint_as_float(__byte_perm(q, 0x4b000000u, 0x7541 + j))};
}
// values of codes j, j + 1: m from bytes plus 128; the unit is M / 127^2 or M / 255^4
__device__ __forceinline__ Pair m_values(uint32_t q, int j, Pair unit) {
    const Pair c = add(bytes_of(q, j), Pair(-(kTwo23 + 128.f)));
    return mul(mul(c, abs(c)), unit);
}
__device__ __forceinline__ Pair fourth(Pair c, Pair zero) {
    const Pair q = mul(c, c);
    return product(q, q, zero);
}
__device__ __forceinline__ Pair v_values(uint32_t q, int j, Pair unit) {
    const Pair c = add(bytes_of(q, j), Pair(-kTwo23)), c2 = mul(c, c);
    return mul(mul(c2, c2), unit);
}
__device__ __forceinline__ float m_unit(float most) { return __fmul_rn(most, (float)(1.0 / (127.0 * 127.0))); }
__device__ __forceinline__ float v_unit(float most) { return __fmul_rn(most, (float)(1.0 / (255.0 * 255.0 * 255.0 * 255.0))); }

// Largest magnitude of a warp's block; magnitudes compare as their bit patterns, NaN above all.
__device__ __forceinline__ float block_max(uint32_t mine) { return __uint_as_float(__reduce_max_sync(0xffffffffu, mine)); }
__device__ __forceinline__ uint32_t larger(uint32_t most, Pair size) {
    return max(most, max(__float_as_uint(size.lo()), __float_as_uint(size.hi())));
}
__device__ __forceinline__ float at_least_normal(float v) {  // max(v, 2^-126), or NaN
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(v), "f"(FLT_MIN));
    return r;
}
// levels per unit of magnitude: top^power / max (0 where the block is held as zeros)
__device__ __forceinline__ float inverse_unit(float most, float top_power) {
    return most > 0.f ? __fmul_rn(__fdiv_rn(1.f, most), top_power) : most;
}
// thresholds of two elements from their Weyl integers
__device__ __forceinline__ Pair thresholds(uint32_t w) {
    return mul(Pair((float)(w >> 8), (float)((w + kIndexStride) >> 8)), Pair(5.9604644775390625e-8f));
}
// Codes of two magnitudes at y levels: the one below (the floor of `root`, the value's place on the
// scale of codes) or the one above, by the share of the way against u.  far: a root was not exact
// enough and its y does not lie between the two codes.
struct Codes {
    uint32_t lo, hi;
};
template <bool FOURTH> __device__ __forceinline__ Codes codes_of(Pair y, float root_lo, float root_hi, Pair u, Pair zero, bool &far) {
    constexpr float top = FOURTH ? 255.f : 127.f;
    const Pair r = add_down(Pair(fminf(root_lo, top - 0.5f), fminf(root_hi, top - 0.5f)), Pair(kTwo23));  // last bits: the floor
    const Pair low = add(r, Pair(-kTwo23)), next = add(low, Pair(1.f));
    const Pair below = FOURTH ? fourth(low, zero) : product(low, low, zero), above = FOURTH ? fourth(next, zero) : product(next, next, zero);
    const Pair past = sub(y, below), limit = mul(u, sub(above, below));
    far |= past.lo() < 0.f || (y.lo() > above.lo() && next.lo() < top);
    far |= past.hi() < 0.f || (y.hi() > above.hi() && next.hi() < top);
    // r's bits are 0x4b000000 + the floor; the caller takes the last byte
    return {__float_as_uint(r.lo()) + (past.lo() > limit.lo()), __float_as_uint(r.hi()) + (past.hi() > limit.hi())};
}
// -c where the value is negative (in the last byte)
__device__ __forceinline__ uint32_t with_sign(uint32_t c, float value) { return value < 0.f ? 0u - c : c; }
// a positive v does not take code 0
__device__ __forceinline__ uint32_t not_zero(uint32_t c, float y) { return y > 0.f ? max(c, 0x4b000001u) : c; }
__device__ __forceinline__ uint32_t last_bytes(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    return __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410);
}

// Codes of four consecutive elements (the first with Weyl integer w) as words.  ROOTS: how exact the
// square roots are; `roots` holds approximate ones of v.
template <bool EXACT>
__device__ __forceinline__ bool four_codes(const Pair (&m)[2], const Pair (&v)[2], const Pair (&roots)[2], float mi, float vi,
                                           float v_scale, uint32_t w, Pair zero, uint32_t &m_word, uint32_t &v_word) {
    bool far = false;
    Codes mc[2], vc[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const Pair u = thresholds(w + 2 * k * kIndexStride);
        const Pair my = product(abs(m[k]), Pair(mi), zero), vy = product(v[k], Pair(vi), zero);
        if (EXACT) {
            mc[k] = codes_of<false>(my, __fsqrt_rn(my.lo()), __fsqrt_rn(my.hi()), u, zero, far);
            vc[k] = codes_of<true>(vy, __fsqrt_rn(__fsqrt_rn(vy.lo())), __fsqrt_rn(__fsqrt_rn(vy.hi())), u, zero, far);
        } else {
            const Pair root = mul(roots[k], Pair(v_scale));  // sqrt(vy) = sqrt(v) sqrt(vi)
            mc[k] = codes_of<false>(my, root_of(my.lo()), root_of(my.hi()), u, zero, far);
            vc[k] = codes_of<true>(vy, root_of(root.lo()), root_of(root.hi()), u, zero, far);
        }
        mc[k].lo = with_sign(mc[k].lo, m[k].lo()), mc[k].hi = with_sign(mc[k].hi, m[k].hi());
        vc[k].lo = not_zero(vc[k].lo, vy.lo()), vc[k].hi = not_zero(vc[k].hi, vy.hi());
    }
    m_word = last_bytes(mc[0].lo, mc[0].hi, mc[1].lo, mc[1].hi);
    v_word = last_bytes(vc[0].lo, vc[0].hi, vc[1].lo, vc[1].hi);
    return far;
}
struct FourCodes {
    uint32_t m, v;
};
__device__ __noinline__ FourCodes exact_codes(Pair m0, Pair m1, Pair v0, Pair v1, float mi, float vi, uint32_t w, Pair zero) {
    const Pair m[2] = {m0, m1}, v[2] = {v0, v1};
    FourCodes c;
    four_codes<true>(m, v, v, mi, vi, 0.f, w, zero, c.m, c.v);
    return c;
}

// ------------------------------------------------------------------------------- the step

template <typename G, int BITS, bool VEC>
__device__ __forceinline__ void update(const wtconv_optim_tensor &t, const StepScalars &s, float clip, long long start) {
    const int lane = threadIdx.x & 31;
    const long long n = t.n;
    const long long first = start + (threadIdx.x >> 5) * 256;
    if (first >= n) return;
    Pair m[2][2], v[2][2], roots[2][2];  // [half of the block][pair]
    float p[2][4], g[2][4], mf[2][4], vf[2][4];
    const long long blk = first / WTCONV_ADAMW_BLOCK;
    uint32_t mq[2], vq[2];
    float mu = 0.f, vu = 0.f;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const long long i = first + h * 128 + lane * 4;
        if (BITS == 8) {
            mq[h] = load_codes<VEC>(static_cast<const uint8_t *>(t.m), i, n) ^ 0x80808080u;
            vq[h] = load_codes<VEC>(static_cast<const uint8_t *>(t.v), i, n);
        } else {
            load4<VEC>(static_cast<const float *>(t.m), i, n, mf[h]);
            load4<VEC>(static_cast<const float *>(t.v), i, n, vf[h]);
        }
        load4<VEC>(t.param, i, n, p[h]);
        load4<VEC>(static_cast<const G *>(t.grad), i, n, g[h]);
    }
    if (BITS == 8) mu = m_unit(t.m_max[blk]), vu = v_unit(t.v_max[blk]);
    if (!(fabsf(clip) <= FLT_MAX)) return;  // a step over gradients without a norm is not taken
    const Pair zero(s.negative_zero);
    uint32_t m_most = 0, v_most = 0;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const long long i = first + h * 128 + lane * 4;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            if (BITS == 8) {
                m[h][k] = m_values(mq[h], 2 * k, Pair(mu));
                v[h][k] = v_values(vq[h], 2 * k, Pair(vu));
            } else {
                m[h][k] = Pair(mf[h][2 * k], mf[h][2 * k + 1]);
                v[h][k] = Pair(vf[h][2 * k], vf[h][2 * k + 1]);
            }
            const Pair gs = mul(Pair(g[h][2 * k], g[h][2 * k + 1]), Pair(clip));
            m[h][k] = add(product(Pair(s.beta1), m[h][k], zero), product(Pair(s.one_minus_beta1), gs, zero));
            v[h][k] = add(product(Pair(s.beta2), v[h][k], zero), product(Pair(s.one_minus_beta2), mul(gs, gs), zero));
            if (BITS == 8) {
                m_most = larger(m_most, abs(m[h][k]));
                v_most = larger(v_most, v[h][k]);
            }
            // (at least the least normal number: its root is far below any useful eps; a NaN comes through)
            roots[h][k] = Pair(root_of(at_least_normal(v[h][k].lo())), root_of(at_least_normal(v[h][k].hi())));
            const Pair d = fma(roots[h][k], Pair(s.root_scale), Pair(s.eps));
            const Pair step = mul(m[h][k], Pair(reciprocal(d.lo()), reciprocal(d.hi())));
            const Pair q = fma(Pair(-s.rate), step, mul(Pair(p[h][2 * k], p[h][2 * k + 1]), Pair(s.keep)));
            p[h][2 * k] = q.lo(), p[h][2 * k + 1] = q.hi();
            if (BITS == 32) {
                mf[h][2 * k] = m[h][k].lo(), mf[h][2 * k + 1] = m[h][k].hi();
                vf[h][2 * k] = v[h][k].lo(), vf[h][2 * k + 1] = v[h][k].hi();
            }
        }
        store4<VEC>(t.param, i, n, p[h]);
        if (t.copy != nullptr) {
            if (s.copy_dtype == WTCONV_BF16) store4<VEC>(static_cast<__nv_bfloat16 *>(t.copy), i, n, p[h]);
            else store4<VEC>(static_cast<__half *>(t.copy), i, n, p[h]);
        }
        if (BITS == 32) {
            store4<VEC>(static_cast<float *>(t.m), i, n, mf[h]);
            store4<VEC>(static_cast<float *>(t.v), i, n, vf[h]);
        }
    }
    if (BITS == 8) {
        float m_max = block_max(m_most), v_max = block_max(v_most);
        if (m_max < kLeastMax) m_max = 0.f;
        if (v_max < kLeastMax) v_max = 0.f;
        const float mi = inverse_unit(m_max, 127.f * 127.f), vi = inverse_unit(v_max, 4228250625.f);
        const float v_scale = root_of(vi);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const long long i = first + h * 128 + lane * 4;
            const uint32_t w = (uint32_t)i * kIndexStride + s.threshold0;
            FourCodes c;
            if (four_codes<false>(m[h], v[h], roots[h], mi, vi, v_scale, w, zero, c.m, c.v))  // (rare)
                c = exact_codes(m[h][0], m[h][1], v[h][0], v[h][1], mi, vi, w, zero);
            store_codes<VEC>(static_cast<uint8_t *>(t.m), i, n, c.m);
            store_codes<VEC>(static_cast<uint8_t *>(t.v), i, n, c.v);
        }
        if (lane == 0) {
            t.m_max[blk] = m_max;
            t.v_max[blk] = v_max;
        }
    }
}

__device__ __forceinline__ bool vector_ok(const wtconv_optim_tensor &t) {
    const uintptr_t all = reinterpret_cast<uintptr_t>(t.param) | reinterpret_cast<uintptr_t>(t.grad) |
                          reinterpret_cast<uintptr_t>(t.m) | reinterpret_cast<uintptr_t>(t.v) |
                          reinterpret_cast<uintptr_t>(t.copy);
    return (all & 15) == 0;
}

template <typename G, int BITS, int CAP>
__global__ void __launch_bounds__(kThreads) adamw_kernel(const __grid_constant__ TensorTable<CAP> table, StepScalars s,
                                                         const float *clip) {
    begin_kernel();
    const float scale = clip != nullptr ? *clip : 1.f;
    const int which = find_tensor(table, blockIdx.x);
    const wtconv_optim_tensor &t = table.t[which];
    const long long start = (long long)(blockIdx.x - table.first[which]) * kChunk;
    if (vector_ok(t)) update<G, BITS, true>(t, s, scale, start);
    else update<G, BITS, false>(t, s, scale, start);
}

template <bool VEC> __device__ __forceinline__ void write_values(const wtconv_optim_tensor &t, long long start) {
    const int lane = threadIdx.x & 31;
    const long long n = t.n, first = start + (threadIdx.x >> 5) * 256;
    if (first >= n) return;
    float *const m_out = t.param, *const v_out = static_cast<float *>(t.copy);
    const long long blk = first / WTCONV_ADAMW_BLOCK;
    uint32_t mq[2], vq[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const long long i = first + h * 128 + lane * 4;
        mq[h] = load_codes<VEC>(static_cast<const uint8_t *>(t.m), i, n);
        vq[h] = load_codes<VEC>(static_cast<const uint8_t *>(t.v), i, n);
    }
    const float mu = m_unit(t.m_max[blk]), vu = v_unit(t.v_max[blk]);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const long long i = first + h * 128 + lane * 4;
        float m[4], v[4];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const Pair mk = m_values(mq[h] ^ 0x80808080u, 2 * k, Pair(mu)), vk = v_values(vq[h], 2 * k, Pair(vu));
            m[2 * k] = mk.lo(), m[2 * k + 1] = mk.hi();
            v[2 * k] = vk.lo(), v[2 * k + 1] = vk.hi();
        }
        if (m_out != nullptr) store4<VEC>(m_out, i, n, m);
        if (v_out != nullptr) store4<VEC>(v_out, i, n, v);
    }
}

template <int CAP> __global__ void __launch_bounds__(kThreads) state_values_kernel(const __grid_constant__ TensorTable<CAP> table) {
    begin_kernel();
    const int which = find_tensor(table, blockIdx.x);
    const wtconv_optim_tensor &t = table.t[which];
    const long long start = (long long)(blockIdx.x - table.first[which]) * kChunk;
    if (vector_ok(t)) write_values<true>(t, start);
    else write_values<false>(t, start);
}

// ------------------------------------------------------------------------------- the norm

template <typename V> __device__ __forceinline__ V block_sum(V v, V *scratch) {  // 8 warps; result in thread 0
    v = warp_sum(v);
    if ((threadIdx.x & 31) == 0) scratch[threadIdx.x >> 5] = v;
    __syncthreads();
    if (threadIdx.x == 0)
        for (int w = 1; w < kThreads / 32; ++w) v += scratch[w];
    return v;
}

// Sum of squares of g[first..last), by the CTA: sixteen bytes a load, four loads in flight (130 M fp32
// elements 94 us, 5.5 TB/s, bound by HBM; with one load in flight and a search per chunk 114).
template <typename G> __device__ __forceinline__ float squares(const G *g, long long first, long long last) {
    constexpr int per = 16 / sizeof(G);
    float mine[4] = {0.f, 0.f, 0.f, 0.f};
    if ((reinterpret_cast<uintptr_t>(g) & 15) == 0) {  // first is a multiple of kChunk
        long long i = first + threadIdx.x * per;
        for (; i + 3 * kThreads * per + per <= last; i += 4 * kThreads * per) {
            uint4 q[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) q[k] = __ldcs(reinterpret_cast<const uint4 *>(g + i + k * kThreads * per));
#pragma unroll
            for (int k = 0; k < 4; ++k)
#pragma unroll
                for (int j = 0; j < per; ++j) {
                    const float v = to_f32(reinterpret_cast<const G *>(&q[k])[j]);
                    mine[k] = fmaf(v, v, mine[k]);
                }
        }
        for (; i < last; i += kThreads * per)
#pragma unroll
            for (int j = 0; j < per; ++j) {
                const float v = i + j < last ? to_f32(g[i + j]) : 0.f;
                mine[j & 3] = fmaf(v, v, mine[j & 3]);
            }
    } else {
        for (long long i = first + threadIdx.x; i < last; i += 4 * kThreads)
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float v = i + k * kThreads < last ? to_f32(g[i + k * kThreads]) : 0.f;
                mine[k] = fmaf(v, v, mine[k]);
            }
    }
    return (mine[0] + mine[1]) + (mine[2] + mine[3]);
}

// A CTA takes a run of chunks, through one tensor after the other.  A thread's fp32 sum covers at
// most kRun elements' share before it moves to fp64.
template <typename G, int CAP> __device__ __forceinline__ double run_of_squares(const TensorTable<CAP> &table) {
    constexpr int kRun = 64 * kChunk;
    double sum = 0.0;
    const int chunks = table.first[table.count];
    int chunk = (int)((long long)chunks * blockIdx.x / gridDim.x);
    const int end = (int)((long long)chunks * (blockIdx.x + 1) / gridDim.x);
    int which = chunk < end ? find_tensor(table, chunk) : 0;
    while (chunk < end) {
        const wtconv_optim_tensor &t = table.t[which];
        const int upto = min(end, table.first[which + 1]);
        const long long first = (long long)(chunk - table.first[which]) * kChunk;
        const long long last = min((long long)(upto - table.first[which]) * kChunk, t.n);
        for (long long i = first; i < last; i += kRun) sum += squares(static_cast<const G *>(t.grad), i, min(i + kRun, last));
        chunk = upto;
        ++which;
    }
    return sum;
}
template <typename G, int CAP>
__global__ void __launch_bounds__(kThreads) norm_part_kernel(const __grid_constant__ TensorTable<CAP> table, double *part) {
    __shared__ double scratch[kThreads / 32];
    begin_kernel();
    const double sum = block_sum(run_of_squares<G>(table), scratch);
    if (threadIdx.x == 0) part[blockIdx.x] = sum;
}

__device__ __forceinline__ void write_norm(double sum, double max_norm, float *out) {
    const double norm = sqrt(sum);
    out[0] = (float)norm;
    out[1] = norm <= (double)FLT_MAX ? (float)fmin(1.0, max_norm / (norm + 1e-6)) : __int_as_float(0x7fc00000);
}

__global__ void __launch_bounds__(kThreads) norm_final_kernel(const double *part, int count, double max_norm, float *out) {
    __shared__ double scratch[kThreads / 32];
    begin_kernel();
    double sum = 0.0;
    for (int i = threadIdx.x; i < count; i += kThreads) sum += part[i];
    sum = block_sum(sum, scratch);
    if (threadIdx.x == 0) write_norm(sum, max_norm, out);
}

// Sum of squares of g[first..last), at most kChunk elements, by a warp: eight loads a lane in flight.
template <typename G> __device__ __forceinline__ float warp_squares(const G *g, long long first, long long last) {
    constexpr int per = 16 / sizeof(G), kInFlight = 8;
    const int lane = threadIdx.x & 31;
    float mine[4] = {0.f, 0.f, 0.f, 0.f};
    long long i = first;
    if ((reinterpret_cast<uintptr_t>(g) & 15) == 0) {  // first is a multiple of kChunk
        const auto add = [&](const uint4 &q) {
#pragma unroll
            for (int j = 0; j < per; ++j) {
                const float v = to_f32(reinterpret_cast<const G *>(&q)[j]);
                mine[j & 3] = fmaf(v, v, mine[j & 3]);
            }
        };
        for (; i + kInFlight * 32 * per <= last; i += kInFlight * 32 * per) {
            uint4 q[kInFlight];
#pragma unroll
            for (int k = 0; k < kInFlight; ++k) q[k] = __ldcs(reinterpret_cast<const uint4 *>(g + i + (k * 32 + lane) * per));
#pragma unroll
            for (int k = 0; k < kInFlight; ++k) add(q[k]);
        }
#pragma unroll 4
        for (i += lane * per; i + per <= last; i += 32 * per) add(__ldcs(reinterpret_cast<const uint4 *>(g + i)));
        i = first + (last - first) / per * per;  // the elements after the last whole load
    }
    for (; i < last; i += kInFlight * 32) {
        float v[kInFlight];
#pragma unroll
        for (int k = 0; k < kInFlight; ++k) v[k] = i + k * 32 + lane < last ? to_f32(g[i + k * 32 + lane]) : 0.f;
#pragma unroll
        for (int k = 0; k < kInFlight; ++k) mine[k & 3] = fmaf(v[k], v[k], mine[k & 3]);
    }
    return (mine[0] + mine[1]) + (mine[2] + mine[3]);
}

// Few chunks: the warps of one cluster take them, neighbours in different CTAs, and its CTAs leave their
// sums with the first one.  Bound by latency: 100 fp32 tensors of 1500 elements 5.2 us, one of 522,240
// 5.5 us (CTAs that went through their share's tensors one by one: 12.1 and 6.9; 256 threads 6.3 and
// 6.8; 1024 threads 6.0 and 6.4; neighbours in one CTA, with 1024 threads, 7.1 and 6.5).
template <typename G, int CAP>
__global__ void __launch_bounds__(kNormThreads) norm_small_kernel(const __grid_constant__ TensorTable<CAP> table, double max_norm,
                                                                  float *out) {
    constexpr int kWarps = kNormThreads / 32;
    __shared__ double scratch[kWarps], sums[kNormCluster];
    cg::cluster_group cluster = cg::this_cluster();
    auto started = cluster.barrier_arrive();  // the first CTA's shared memory is there
    begin_kernel();
    const int warp = threadIdx.x >> 5, chunks = table.first[table.count];
    double sum = 0.0;
    for (int chunk = warp * kNormCluster + blockIdx.x; chunk < chunks; chunk += kNormCluster * kWarps) {
        const int which = find_tensor(table, chunk);
        const wtconv_optim_tensor &t = table.t[which];
        const long long first = (long long)(chunk - table.first[which]) * kChunk;
        sum += warp_squares(static_cast<const G *>(t.grad), first, min(first + kChunk, t.n));
    }
    sum = warp_sum(sum);
    if ((threadIdx.x & 31) == 0) scratch[warp] = sum;
    __syncthreads();
    cluster.barrier_wait(std::move(started));
    if (warp == 0) {
        sum = warp_sum(threadIdx.x < kWarps ? scratch[threadIdx.x] : 0.0);
        if (threadIdx.x == 0) cluster.map_shared_rank(sums, 0)[blockIdx.x] = sum;
    }
    cluster.sync();
    if (blockIdx.x == 0 && threadIdx.x == 0) {
        double total = 0.0;
        for (int i = 0; i < kNormCluster; ++i) total += sums[i];
        write_norm(total, max_norm, out);
    }
}
template <typename G, int CAP>
cudaError_t launch_adamw_typed(const TensorTable<CAP> &table, const StepScalars &s, const float *clip, cudaStream_t st) {
    const unsigned grid = (unsigned)table.first[table.count];
    return launch_kernel(s.state_bits == 32 ? adamw_kernel<G, 32, CAP> : adamw_kernel<G, 8, CAP>, grid, kThreads, 0, st, 1, table, s,
                         clip);
}

}  // namespace

int norm_blocks(long long chunks) {
    const long long most = (long long)sm_count() * 8;
    return (int)(chunks < most ? chunks : most);
}

template <int CAP> cudaError_t launch_adamw(const TensorTable<CAP> &table, const StepScalars &s, const float *clip, cudaStream_t st) {
    if (s.grad_dtype == WTCONV_F32) return launch_adamw_typed<float>(table, s, clip, st);
    if (s.grad_dtype == WTCONV_BF16) return launch_adamw_typed<__nv_bfloat16>(table, s, clip, st);
    return launch_adamw_typed<__half>(table, s, clip, st);
}

template <int CAP>
cudaError_t launch_norm_part(const TensorTable<CAP> &table, int grad_dtype, double *part, int blocks, cudaStream_t st) {
    const auto kernel = grad_dtype == WTCONV_F32 ? norm_part_kernel<float, CAP>
                        : grad_dtype == WTCONV_BF16 ? norm_part_kernel<__nv_bfloat16, CAP> : norm_part_kernel<__half, CAP>;
    return launch_kernel(kernel, blocks, kThreads, 0, st, 1, table, part);
}

template <int CAP>
cudaError_t launch_norm_small(const TensorTable<CAP> &table, int grad_dtype, double max_norm, float *out, cudaStream_t st) {
    const auto kernel = grad_dtype == WTCONV_F32 ? norm_small_kernel<float, CAP>
                        : grad_dtype == WTCONV_BF16 ? norm_small_kernel<__nv_bfloat16, CAP> : norm_small_kernel<__half, CAP>;
    return launch_kernel(kernel, kNormCluster, kNormThreads, 0, st, kNormCluster, table, max_norm, out);
}

cudaError_t launch_norm_final(const double *part, int count, double max_norm, float *out, cudaStream_t st) {
    return launch_kernel(norm_final_kernel, 1, kThreads, 0, st, 1, part, count, max_norm, out);
}

template <int CAP> cudaError_t launch_state_values(const TensorTable<CAP> &table, cudaStream_t st) {
    return launch_kernel(state_values_kernel<CAP>, (unsigned)table.first[table.count], kThreads, 0, st, 1, table);
}

template cudaError_t launch_adamw<kSmallTable>(const TensorTable<kSmallTable> &, const StepScalars &, const float *, cudaStream_t);
template cudaError_t launch_adamw<kLargeTable>(const TensorTable<kLargeTable> &, const StepScalars &, const float *, cudaStream_t);
template cudaError_t launch_norm_part<kSmallTable>(const TensorTable<kSmallTable> &, int, double *, int, cudaStream_t);
template cudaError_t launch_norm_part<kLargeTable>(const TensorTable<kLargeTable> &, int, double *, int, cudaStream_t);
template cudaError_t launch_norm_small<kSmallTable>(const TensorTable<kSmallTable> &, int, double, float *, cudaStream_t);
template cudaError_t launch_norm_small<kLargeTable>(const TensorTable<kLargeTable> &, int, double, float *, cudaStream_t);
template cudaError_t launch_state_values<kSmallTable>(const TensorTable<kSmallTable> &, cudaStream_t);
template cudaError_t launch_state_values<kLargeTable>(const TensorTable<kLargeTable> &, cudaStream_t);

}  // namespace wtconv
