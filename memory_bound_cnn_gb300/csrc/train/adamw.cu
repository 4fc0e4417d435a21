// AdamW step over a table of tensors (wtconv_optim.h).
//
// One CTA per chunk of 2048 elements of one tensor, one warp per 256 of them (a block of the 8-bit
// states), eight elements per lane in registers between the one read and the one write of each
// array.  Bound by HBM.
#include <float.h>

#include "optim.h"
#include "train_device.cuh"

namespace wtconv {

namespace {

constexpr int kThreads = 256;
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
// Products and sums that decide a code are rounded one by one (no fused multiply-add), so that a
// code is a function of its inputs that any fp32 program can follow.  Conversions between bytes and
// fp32 go through 2^23 + n, whose last bits are n: the conversion instructions run at an eighth of
// the rate of an add, and with them and exact roots the step took 787 us for 130 M elements.

constexpr float kTwo23 = 8388608.f;

// byte j of a word as fp32
__device__ __forceinline__ float byte_of(uint32_t q, int j) {
    return __uint_as_float(__byte_perm(q, 0x4b000000u, 0x7540 | j)) - kTwo23;
}
__device__ __forceinline__ float m_value(float c, float unit) { return __fmul_rn(__fmul_rn(c, fabsf(c)), unit); }  // unit = M / 127^2
__device__ __forceinline__ float v_level(float c) {  // c^4
    const float q = __fmul_rn(c, c);
    return __fmul_rn(q, q);
}
__device__ __forceinline__ float m_unit(float most) { return __fmul_rn(most, (float)(1.0 / (127.0 * 127.0))); }
__device__ __forceinline__ float v_unit(float most) { return __fmul_rn(most, (float)(1.0 / (255.0 * 255.0 * 255.0 * 255.0))); }

// Largest magnitude of a warp's block; magnitudes compare as their bit patterns, NaN above all.
__device__ __forceinline__ float block_max(float mine) {
    return __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(mine)));
}
__device__ __forceinline__ float nan_max(float a, float b) {  // of magnitudes: a NaN stays
    return __uint_as_float(max(__float_as_uint(a), __float_as_uint(b)));
}
// levels per unit of magnitude: top^power / max (0 where the block is held as zeros)
__device__ __forceinline__ float inverse_unit(float most, float top_power) {
    return most > 0.f ? __fmul_rn(__fdiv_rn(1.f, most), top_power) : most;
}
__device__ __forceinline__ float threshold(uint32_t index, uint32_t threshold0) {
    return __fmul_rn((float)((index * kIndexStride + threshold0) >> 8), 5.9604644775390625e-8f);
}
__device__ __forceinline__ float root_of(float v) {
    float r;
    asm("sqrt.approx.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}
__device__ __forceinline__ float reciprocal(float v) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}
// The code of a magnitude at y levels: the one below it (the floor of `root`, the value's place on
// the scale of codes) or the one above, by the share of the way against u.  far: the root was not
// exact enough and y does not lie between the two.
template <bool FOURTH> __device__ __forceinline__ uint32_t code_of(float y, float root, float u, bool &far) {
    constexpr float top = FOURTH ? 255.f : 127.f;
    const float r = __fadd_rd(fminf(root, top - 0.5f), kTwo23);  // last bits: floor(root)
    const float low = r - kTwo23, next = low + 1.f;
    const float below = FOURTH ? v_level(low) : low * low, above = FOURTH ? v_level(next) : next * next;
    far |= y < below || (y > above && next < top);
    const bool up = __fsub_rn(y, below) > __fmul_rn(u, __fsub_rn(above, below));
    return (__float_as_uint(r) & 255u) + up;
}
template <bool FOURTH> __device__ __noinline__ uint32_t exact_code(float y, float u) {
    bool far = false;
    const float root = __fsqrt_rn(y);
    return code_of<FOURTH>(y, FOURTH ? __fsqrt_rn(root) : root, u, far);
}

// ------------------------------------------------------------------------------- the step

template <typename G, int BITS, bool VEC>
__device__ __forceinline__ void update(const wtconv_optim_tensor &t, const StepScalars &s, float clip, long long start) {
    const int lane = threadIdx.x & 31;
    const long long n = t.n;
    const long long first = start + (threadIdx.x >> 5) * 256;
    if (first >= n) return;
    float m[2][4], v[2][4], p[2][4], g[2][4];
    const long long blk = first / WTCONV_ADAMW_BLOCK;
    uint32_t mq[2], vq[2];
    float mu = 0.f, vu = 0.f;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const long long i = first + h * 128 + lane * 4;
        if (BITS == 8) {
            mq[h] = load_codes<VEC>(static_cast<const uint8_t *>(t.m), i, n);
            vq[h] = load_codes<VEC>(static_cast<const uint8_t *>(t.v), i, n);
        } else {
            load4<VEC>(static_cast<const float *>(t.m), i, n, m[h]);
            load4<VEC>(static_cast<const float *>(t.v), i, n, v[h]);
        }
        load4<VEC>(t.param, i, n, p[h]);
        load4<VEC>(static_cast<const G *>(t.grad), i, n, g[h]);
    }
    if (BITS == 8) mu = m_unit(t.m_max[blk]), vu = v_unit(t.v_max[blk]);
    if (!(fabsf(clip) <= FLT_MAX)) return;  // a step over gradients without a norm is not taken
    float m_most = 0.f, v_most = 0.f, root[2][4];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const long long i = first + h * 128 + lane * 4;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (BITS == 8) {
                m[h][j] = m_value(byte_of(mq[h] ^ 0x80808080u, j) - 128.f, mu);
                v[h][j] = __fmul_rn(v_level(byte_of(vq[h], j)), vu);
            }
            const float gs = __fmul_rn(g[h][j], clip);
            m[h][j] = __fadd_rn(__fmul_rn(s.beta1, m[h][j]), __fmul_rn(s.one_minus_beta1, gs));
            v[h][j] = __fadd_rn(__fmul_rn(s.beta2, v[h][j]), __fmul_rn(s.one_minus_beta2, __fmul_rn(gs, gs)));
            if (BITS == 8) {
                m_most = nan_max(m_most, fabsf(m[h][j]));
                v_most = nan_max(v_most, v[h][j]);
            }
            root[h][j] = root_of(v[h][j]);
            const float step = m[h][j] * reciprocal(fmaf(root[h][j], s.root_scale, s.eps));
            p[h][j] = fmaf(-s.rate, step, p[h][j] * s.keep);
        }
        store4<VEC>(t.param, i, n, p[h]);
        if (t.copy != nullptr) {
            if (s.copy_dtype == WTCONV_BF16) store4<VEC>(static_cast<__nv_bfloat16 *>(t.copy), i, n, p[h]);
            else store4<VEC>(static_cast<__half *>(t.copy), i, n, p[h]);
        }
        if (BITS == 32) {
            store4<VEC>(static_cast<float *>(t.m), i, n, m[h]);
            store4<VEC>(static_cast<float *>(t.v), i, n, v[h]);
        }
    }
    if (BITS == 8) {
        m_most = block_max(m_most);
        v_most = block_max(v_most);
        if (m_most < kLeastMax) m_most = 0.f;
        if (v_most < kLeastMax) v_most = 0.f;
        const float mi = inverse_unit(m_most, 127.f * 127.f), vi = inverse_unit(v_most, 4228250625.f);
        const float v_scale = root_of(vi);  // sqrt(y) = sqrt(v) sqrt(vi)
        bool far = false;
        uint32_t mc[2] = {0, 0}, vc[2] = {0, 0};
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float u = threshold((uint32_t)(first + h * 128 + lane * 4 + j), s.threshold0);
                const float my = __fmul_rn(fabsf(m[h][j]), mi), vy = __fmul_rn(v[h][j], vi);
                const uint32_t cm = code_of<false>(my, root_of(my), u, far);
                const uint32_t cv = code_of<true>(vy, root_of(root[h][j] * v_scale), u, far);
                mc[h] |= (m[h][j] < 0.f ? 0u - cm : cm) % 256u << (8 * j);
                vc[h] |= max(cv, vy > 0.f ? 1u : 0u) << (8 * j);
            }
        if (far) {  // about one warp in a hundred
#pragma unroll 1
            for (int k = 0; k < 8; ++k) {
                const int h = k >> 2, j = k & 3;
                float mv = 0.f, vv = 0.f;
#pragma unroll
                for (int q = 0; q < 8; ++q)
                    if (q == k) mv = m[q >> 2][q & 3], vv = v[q >> 2][q & 3];
                const float u = threshold((uint32_t)(first + h * 128 + lane * 4 + j), s.threshold0);
                const float my = __fmul_rn(fabsf(mv), mi), vy = __fmul_rn(vv, vi);
                const uint32_t cm = exact_code<false>(my, u), cv = max(exact_code<true>(vy, u), vy > 0.f ? 1u : 0u);
                const uint32_t mask = 255u << (8 * j);
                const uint32_t mw = (mv < 0.f ? 0u - cm : cm) % 256u << (8 * j), vw = cv << (8 * j);
                if (h == 0) mc[0] = (mc[0] & ~mask) | mw, vc[0] = (vc[0] & ~mask) | vw;
                else mc[1] = (mc[1] & ~mask) | mw, vc[1] = (vc[1] & ~mask) | vw;
            }
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const long long i = first + h * 128 + lane * 4;
            store_codes<VEC>(static_cast<uint8_t *>(t.m), i, n, mc[h]);
            store_codes<VEC>(static_cast<uint8_t *>(t.v), i, n, vc[h]);
        }
        if (lane == 0) {
            t.m_max[blk] = m_most;
            t.v_max[blk] = v_most;
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
        for (int j = 0; j < 4; ++j) {
            m[j] = m_value(byte_of(mq[h] ^ 0x80808080u, j) - 128.f, mu);
            v[j] = __fmul_rn(v_level(byte_of(vq[h], j)), vu);
        }
        if (m_out != nullptr) store4<VEC>(m_out, i, n, m);
        if (v_out != nullptr) store4<VEC>(v_out, i, n, v);
    }
}

template <int CAP> __global__ void __launch_bounds__(kThreads) state_values_kernel(const __grid_constant__ TensorTable<CAP> table) {
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

// Sum of squares of g[first..last), by the CTA: sixteen bytes a load, four loads in flight.
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
template <typename G, int CAP>
__global__ void __launch_bounds__(kThreads) norm_part_kernel(const __grid_constant__ TensorTable<CAP> table, double *part) {
    __shared__ double scratch[kThreads / 32];
    constexpr int kRun = 64 * kChunk;
    double sum = 0.0;
    const int chunks = table.first[table.count];
    int chunk = (int)((long long)chunks * blockIdx.x / gridDim.x);
    const int end = (int)((long long)chunks * (blockIdx.x + 1) / gridDim.x);
    int which = find_tensor(table, chunk);
    while (chunk < end) {
        const wtconv_optim_tensor &t = table.t[which];
        const int upto = min(end, table.first[which + 1]);
        const long long first = (long long)(chunk - table.first[which]) * kChunk;
        const long long last = min((long long)(upto - table.first[which]) * kChunk, t.n);
        for (long long i = first; i < last; i += kRun) sum += squares(static_cast<const G *>(t.grad), i, min(i + kRun, last));
        chunk = upto;
        ++which;
    }
    sum = block_sum(sum, scratch);
    if (threadIdx.x == 0) part[blockIdx.x] = sum;
}

__global__ void __launch_bounds__(kThreads) norm_final_kernel(const double *part, int count, double max_norm, float *out) {
    __shared__ double scratch[kThreads / 32];
    double sum = 0.0;
    for (int i = threadIdx.x; i < count; i += kThreads) sum += part[i];
    sum = block_sum(sum, scratch);
    if (threadIdx.x == 0) {
        const double norm = sqrt(sum);
        out[0] = (float)norm;
        out[1] = norm <= (double)FLT_MAX ? (float)fmin(1.0, max_norm / (norm + 1e-6)) : __int_as_float(0x7fc00000);
    }
}

template <typename G, int CAP>
cudaError_t launch_adamw_typed(const TensorTable<CAP> &table, const StepScalars &s, const float *clip, cudaStream_t st) {
    const unsigned grid = (unsigned)table.first[table.count];
    if (s.state_bits == 32) adamw_kernel<G, 32, CAP><<<grid, kThreads, 0, st>>>(table, s, clip);
    else adamw_kernel<G, 8, CAP><<<grid, kThreads, 0, st>>>(table, s, clip);
    return cudaGetLastError();
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
    if (grad_dtype == WTCONV_F32) norm_part_kernel<float><<<blocks, kThreads, 0, st>>>(table, part);
    else if (grad_dtype == WTCONV_BF16) norm_part_kernel<__nv_bfloat16><<<blocks, kThreads, 0, st>>>(table, part);
    else norm_part_kernel<__half><<<blocks, kThreads, 0, st>>>(table, part);
    return cudaGetLastError();
}

cudaError_t launch_norm_final(const double *part, int count, double max_norm, float *out, cudaStream_t st) {
    norm_final_kernel<<<1, kThreads, 0, st>>>(part, count, max_norm, out);
    return cudaGetLastError();
}

template <int CAP> cudaError_t launch_state_values(const TensorTable<CAP> &table, cudaStream_t st) {
    state_values_kernel<<<(unsigned)table.first[table.count], kThreads, 0, st>>>(table);
    return cudaGetLastError();
}

template cudaError_t launch_adamw<kSmallTable>(const TensorTable<kSmallTable> &, const StepScalars &, const float *, cudaStream_t);
template cudaError_t launch_adamw<kLargeTable>(const TensorTable<kLargeTable> &, const StepScalars &, const float *, cudaStream_t);
template cudaError_t launch_norm_part<kSmallTable>(const TensorTable<kSmallTable> &, int, double *, int, cudaStream_t);
template cudaError_t launch_norm_part<kLargeTable>(const TensorTable<kLargeTable> &, int, double *, int, cudaStream_t);
template cudaError_t launch_state_values<kSmallTable>(const TensorTable<kSmallTable> &, cudaStream_t);
template cudaError_t launch_state_values<kLargeTable>(const TensorTable<kLargeTable> &, cudaStream_t);

}  // namespace wtconv
