// Backward of the selective scan.
#pragma once

#include <algorithm>
#include <type_traits>

#include "column_sums.cuh"
#include "selective_device.cuh"

namespace wtconv {

// A CTA takes 32 channels of a sequence (or of a segment), from the end to the beginning, in blocks of 16
// positions, LANES lanes with four states each to a channel.  A block's states are recomputed from the kept one
// before it and stay in registers (4 x 16 a lane), then the positions are gone through backwards.  Of the
// sums, those over a channel's states meet by exchanges between its lanes for LANES positions at a time; those over
// channels (dB, dC) by exchanges between the warp's channels, then between warps in shared memory, then between
// CTAs in selective_sums_kernel.
// LOCAL: only the gradient that the segment's beginning passes on if nothing enters at its end, and the sum
// of its steps; the CTAs of earlier segments begin with what these compose to.
template <typename T, int LANES, bool PLANES, bool LOCAL>
__global__ void __launch_bounds__(kSelTile *LANES, 16 / LANES) selective_backward_kernel(const __grid_constant__ SelectiveArgs a) {
    constexpr int THREADS = kSelTile * LANES, BLOCK = kSelKeep, SHARE = kSelTile * BLOCK / THREADS, PAD = 4 * LANES, ROW = kSelTile + 1;
    constexpr int GROUP = 32 / LANES;  // channels of a warp
    extern __shared__ float4 shared[];
    float4 *const coef = shared;                          // [BLOCK][ROW]: d, d x, r
    float4 *const bs = coef + BLOCK * ROW, *const cs = bs + BLOCK * LANES;
    float *const sums = reinterpret_cast<float *>(cs + BLOCK * LANES);  // [3][BLOCK][ROW]: over g B, k A, C h
    float *const part = sums + 3 * BLOCK * ROW;           // [warps][BLOCK][2][PAD]: dB and dC of a warp's channels
    begin_kernel();
    const Place at_(a, blockIdx.x);
    if (LOCAL && at_.segment == 0) return;  // nobody is before it
    const int tid = threadIdx.x, b = at_.b, N = a.s.N, stop = min(at_.end, at_.length);
    const int c = tid / LANES, quad = tid % LANES, n0 = 4 * quad, warp = tid / 32, cw = tid % 32 / LANES;
    const bool live = c < at_.channels;
    const long long row = (long long)b * a.s.C + at_.c0 + c;  // of [B][C]
    Quad decay = {Pair(0.f), Pair(0.f)}, carry = decay, dA = decay;
    if (live) {
        decay = load_quad(a.in.A + (long long)(at_.c0 + c) * N, n0, N);
        decay.a = mul(decay.a, Pair(kSelLog2E)), decay.b = mul(decay.b, Pair(kSelLog2E));
    }
    if (!LOCAL && live) {
        if (a.dh_last != nullptr) carry = load_quad(a.dh_last + row * N, n0, N);
        if (at_.first < at_.length)
            for (int k = (at_.length - 1) / a.segment; k > at_.segment; --k) {
                const long long i = ((long long)b * a.segments + k) * a.s.C + at_.c0 + c;
                const Pair d(a.steps[i]);
                const Quad u = quad_of(*reinterpret_cast<const float4 *>(a.ends + i * PAD + n0));
                carry.a = fma(exp2_fast(mul(d, decay.a)), carry.a, u.a), carry.b = fma(exp2_fast(mul(d, decay.b)), carry.b, u.b);
            }
    }
    float step_sum = 0.f;
    constexpr int OWN = PLANES ? SHARE : 1;  // channels of a thread's share
    float dD[OWN], d_bias[OWN];
#pragma unroll
    for (int i = 0; i < OWN; ++i) dD[i] = d_bias[i] = 0.f;

    const int blocks = stop > at_.first ? (stop - at_.first + BLOCK - 1) / BLOCK : 0;
    for (int k = blocks - 1; k >= 0; --k) {
        const int t0 = at_.first + k * BLOCK, count = min(BLOCK, stop - t0);
        float x[SHARE], r[SHARE], slope[SHARE], z_dy[SHARE];  // z_dy: dy silu'(z)
        Quad before = {Pair(0.f), Pair(0.f)};
        if (!LOCAL && live) {
            const long long kept = (long long)b * a.keep + t0 / kSelKeep;
            before = quad_of(*reinterpret_cast<const float4 *>(a.states_in + (kept * a.s.C + at_.c0 + c) * PAD + n0));
        }
#pragma unroll
        for (int i = 0; i < SHARE; ++i) {
            const int e = tid + i * THREADS, pc = PLANES ? e / BLOCK : e % kSelTile, pt = PLANES ? e % BLOCK : e / kSelTile;
            float d = 0.f;
            x[i] = r[i] = slope[i] = z_dy[i] = 0.f;
            if (pc < at_.channels && pt < count) {
                if (!LOCAL) x[i] = to_f32(*at<const T, PLANES>(a.in.x, b, t0 + pt, at_.c0 + pc));
                r[i] = to_f32(*at<const T, PLANES>(a.dy, b, t0 + pt, at_.c0 + pc));
                d = to_f32(*at<const T, PLANES>(a.in.dt, b, t0 + pt, at_.c0 + pc));
                if (a.in.dt_bias != nullptr) d += a.in.dt_bias[at_.c0 + pc];
                slope[i] = 1.f;
                if (a.s.softplus) {
                    const Softplus s = softplus_of(d);
                    d = s.value, slope[i] = s.slope;
                }
                if (a.in.z.p != nullptr) {
                    const float z = to_f32(*at<const T, PLANES>(a.in.z, b, t0 + pt, at_.c0 + pc)), p = sigmoid_of(z);
                    z_dy[i] = r[i] * p * fmaf(z, 1.f - p, 1.f), r[i] *= z * p;
                }
            }
            coef[pt * ROW + pc] = make_float4(d, d * x[i], r[i], 0.f);
        }
#pragma unroll
        for (int i = 0; i < PAD * BLOCK / THREADS; ++i) {
            const int e = tid + i * THREADS, n = PLANES ? e / BLOCK : e % PAD, pt = PLANES ? e % BLOCK : e / PAD;
            const bool ok = n < N && pt < count;
            const int state = at_.group * N + n;
            if (!LOCAL)
                reinterpret_cast<float *>(bs)[pt * PAD + n] = ok ? to_f32(*at<const T, PLANES>(a.in.Bm, b, t0 + pt, state)) : 0.f;
            reinterpret_cast<float *>(cs)[pt * PAD + n] = ok ? to_f32(*at<const T, PLANES>(a.in.Cm, b, t0 + pt, state)) : 0.f;
        }
        __syncthreads();

        if (LOCAL) {
            for (int t = count - 1; t >= 0; --t) {
                const float4 q = coef[t * ROW + c];
                const Quad o = quad_of(cs[t * LANES + quad]);
                const Pair d(q.x), r2(q.z);
                carry.a = mul(exp2_fast(mul(d, decay.a)), fma(o.a, r2, carry.a));
                carry.b = mul(exp2_fast(mul(d, decay.b)), fma(o.b, r2, carry.b));
                step_sum += q.x;
            }
            __syncthreads();
            continue;
        }

        const auto scan = [&](auto full) {
            constexpr bool FULL = decltype(full)::value;
            Quad h[BLOCK];
#pragma unroll
            for (int t = 0; t < BLOCK; ++t) {
                if (!FULL && t >= count) break;
                const float4 q = coef[t * ROW + c];
                const Quad u = quad_of(bs[t * LANES + quad]), last = t == 0 ? before : h[t == 0 ? 0 : t - 1];
                const Pair d(q.x), dx(q.y);
                h[t].a = fma(exp2_fast(mul(d, decay.a)), last.a, mul(dx, u.a));
                h[t].b = fma(exp2_fast(mul(d, decay.b)), last.b, mul(dx, u.b));
            }
            Quad dA_block = {Pair(0.f), Pair(0.f)};
#pragma unroll
            for (int batch = BLOCK / LANES - 1; batch >= 0; --batch) {
                if (!FULL && batch * LANES >= count) continue;
                float s1[LANES], s2[LANES], s3[LANES];
#pragma unroll
                for (int j = LANES - 1; j >= 0; --j) {
                    const int t = batch * LANES + j;
                    s1[j] = s2[j] = s3[j] = 0.f;
                    float v[8] = {};
                    if (FULL || t < count) {
                        const float4 q = coef[t * ROW + c];
                        const Quad u = quad_of(bs[t * LANES + quad]), o = quad_of(cs[t * LANES + quad]);
                        const Quad last = t == 0 ? before : h[t == 0 ? 0 : t - 1];
                        const Pair d(q.x), dx(q.y), r2(q.z);
                        const Quad g = {fma(o.a, r2, carry.a), fma(o.b, r2, carry.b)};
                        carry.a = mul(exp2_again(mul(d, decay.a)), g.a), carry.b = mul(exp2_again(mul(d, decay.b)), g.b);
                        const Quad kk = {mul(carry.a, last.a), mul(carry.b, last.b)};
                        dA_block.a = fma(kk.a, d, dA_block.a), dA_block.b = fma(kk.b, d, dA_block.b);
                        const Pair p1 = fma(g.a, u.a, mul(g.b, u.b)), p2 = fma(kk.a, decay.a, mul(kk.b, decay.b));
                        const Pair p3 = fma(o.a, h[t].a, mul(o.b, h[t].b));
                        s1[j] = p1.lo() + p1.hi(), s2[j] = p2.lo() + p2.hi(), s3[j] = p3.lo() + p3.hi();
                        const Pair b0 = mul(g.a, dx), b1 = mul(g.b, dx), c0 = mul(h[t].a, r2), c1 = mul(h[t].b, r2);
                        v[0] = b0.lo(), v[1] = b0.hi(), v[2] = b1.lo(), v[3] = b1.hi();
                        v[4] = c0.lo(), v[5] = c0.hi(), v[6] = c1.lo(), v[7] = c1.hi();
                    }
                    // over the warp's channels: GROUP of them, of which 8 at most can share the 8 values
                    float *const to = part + (((warp * BLOCK + t) * 2) * PAD);
                    if constexpr (GROUP >= 8) {
                        sum_exchange<8, LANES>(v, cw % 8);
                        if (GROUP == 16) v[0] += __shfl_xor_sync(0xffffffffu, v[0], 8 * LANES);
                        if (cw < 8) to[cw / 4 * PAD + n0 + cw % 4] = v[0];
                    } else {
                        constexpr int LEFT = 8 / GROUP;  // values that stay with a lane
#pragma unroll
                        for (int w = GROUP / 2; w >= 1; w /= 2) {
                            const bool upper = cw & w;
#pragma unroll
                            for (int i = 0; i < w * LEFT; ++i) {
                                const float send = upper ? v[i] : v[i + w * LEFT], keep = upper ? v[i + w * LEFT] : v[i];
                                v[i] = keep + __shfl_xor_sync(0xffffffffu, send, w * LANES);
                            }
                        }
#pragma unroll
                        for (int i = 0; i < LEFT; ++i) to[(cw * LEFT + i) / 4 * PAD + n0 + (cw * LEFT + i) % 4] = v[i];
                    }
                }
                sum_exchange<LANES, 1>(s1, quad), sum_exchange<LANES, 1>(s2, quad), sum_exchange<LANES, 1>(s3, quad);
                float *const to = sums + (batch * LANES + quad) * ROW + c;
                to[0] = s1[0], to[BLOCK * ROW] = s2[0], to[2 * BLOCK * ROW] = s3[0];
            }
            dA.a = add(dA.a, dA_block.a), dA.b = add(dA.b, dA_block.b);
        };
        if (count == BLOCK) scan(std::true_type{});
        else scan(std::false_type{});
        __syncthreads();

#pragma unroll
        for (int i = 0; i < SHARE; ++i) {
            const int e = tid + i * THREADS, pc = PLANES ? e / BLOCK : e % kSelTile, pt = PLANES ? e % BLOCK : e / kSelTile;
            if (pc >= at_.channels || pt >= count) continue;
            const float into = sums[pt * ROW + pc], through = sums[(BLOCK + pt) * ROW + pc] * kSelLn2, ch = sums[(2 * BLOCK + pt) * ROW + pc];
            const float D = a.in.D == nullptr ? 0.f : a.in.D[at_.c0 + pc];
            const float d = coef[pt * ROW + pc].x;
            const float dd = fmaf(x[i], into, through) * slope[i];
            dD[PLANES ? i : 0] = fmaf(r[i], x[i], dD[PLANES ? i : 0]), d_bias[PLANES ? i : 0] += dd;
            *at<T, PLANES>(a.g.dx, b, t0 + pt, at_.c0 + pc) = from_f32<T>(fmaf(D, r[i], d * into));
            *at<T, PLANES>(a.g.d_dt, b, t0 + pt, at_.c0 + pc) = from_f32<T>(dd);
            if (a.in.z.p != nullptr) *at<T, PLANES>(a.g.dz, b, t0 + pt, at_.c0 + pc) = from_f32<T>(z_dy[i] * fmaf(D, x[i], ch));
        }
        float *const to = a.part_bc + (((long long)at_.tile * a.s.B + b) * a.s.T + t0) * 2 * PAD;
        for (int e = tid; e < count * 2 * PAD; e += THREADS) {
            float v = 0.f;
#pragma unroll
            for (int w = 0; w < LANES; ++w) v += part[w * BLOCK * 2 * PAD + e];
            to[e] = v;
        }
        __syncthreads();
    }

    if (LOCAL) {
        if (live && at_.first < at_.length) {
            const long long i = ((long long)b * a.segments + at_.segment) * a.s.C + at_.c0 + c;
            *reinterpret_cast<float4 *>(a.ends + i * PAD + n0) = float4_of(carry);
            if (quad == 0) a.steps[i] = step_sum;
        }
        return;
    }
    if (at_.segment == 0 && live && a.g.d_h0 != nullptr) store_quad(a.g.d_h0 + row * N, n0, N, carry);
    const long long i = ((long long)b * a.segments + at_.segment) * a.s.C + at_.c0;
    if (live) store_quad(a.part_a + (i + c) * N, n0, N, dA);
    // dD and d_dt_bias: the threads that share a channel
    const long long half = (long long)a.s.B * a.segments * a.s.C;
    if (PLANES) {  // 16 neighbouring lanes
#pragma unroll
        for (int j = 0; j < OWN; ++j) {
            float v = dD[j], w = d_bias[j];
#pragma unroll
            for (int m = 8; m >= 1; m /= 2) v += __shfl_xor_sync(0xffffffffu, v, m), w += __shfl_xor_sync(0xffffffffu, w, m);
            const int pc = (tid + j * THREADS) / BLOCK;
            if (tid % BLOCK == 0 && pc < at_.channels) a.part_c[i + pc] = v, a.part_c[half + i + pc] = w;
        }
    } else {  // one of each warp
        sums[tid] = dD[0], sums[THREADS + tid] = d_bias[0];  // (at most 1024 of the 3 x 16 x 33; all have passed the last barrier)
        __syncthreads();
        if (tid < at_.channels) {
            float v = 0.f, w = 0.f;
            for (int j = 0; j < LANES; ++j) v += sums[tid + j * kSelTile], w += sums[THREADS + tid + j * kSelTile];
            a.part_c[i + tid] = v, a.part_c[half + i + tid] = w;
        }
    }
    // positions past the sequence's end
    for (int t0 = max(at_.first, at_.length); t0 < at_.end; t0 += BLOCK) {
#pragma unroll
        for (int j = 0; j < SHARE; ++j) {
            const int e = tid + j * THREADS, pc = PLANES ? e / BLOCK : e % kSelTile, pt = PLANES ? e % BLOCK : e / kSelTile;
            if (pc >= at_.channels || pt >= at_.end - t0) continue;
            *at<T, PLANES>(a.g.dx, b, t0 + pt, at_.c0 + pc) = from_f32<T>(0.f);
            *at<T, PLANES>(a.g.d_dt, b, t0 + pt, at_.c0 + pc) = from_f32<T>(0.f);
            if (a.in.z.p != nullptr) *at<T, PLANES>(a.g.dz, b, t0 + pt, at_.c0 + pc) = from_f32<T>(0.f);
        }
    }
}

// dB and dC: the sums over a group's tiles, in their order; 0 past a sequence's end.
template <typename T, bool PLANES> __global__ void __launch_bounds__(256) selective_sums_kernel(const __grid_constant__ SelectiveArgs a) {
    begin_kernel();
    const int N = a.s.N, width = 2 * a.padded;
    const long long per = (long long)a.s.B * a.s.T * width, all = (long long)a.s.B * a.s.T * a.s.G * 2 * N;
    for (long long e = (long long)blockIdx.x * 256 + threadIdx.x; e < all; e += (long long)gridDim.x * 256) {
        // in the order of the outputs' memory
        long long rest = e;
        int n, g, t, b, which;
        if (PLANES) {
            t = rest % a.s.T, rest /= a.s.T, n = rest % N, rest /= N, which = rest % 2, rest /= 2;
            g = rest % a.s.G, b = rest / a.s.G;
        } else {
            n = rest % N, rest /= N, which = rest % 2, rest /= 2, g = rest % a.s.G, rest /= a.s.G;
            t = rest % a.s.T, b = rest / a.s.T;
        }
        const int length = a.in.lengths == nullptr ? a.s.T : a.in.lengths[b];
        float v = 0.f;
        if (t < length) {
            const float *p = a.part_bc + (long long)g * a.tiles * per + ((long long)b * a.s.T + t) * width + which * a.padded + n;
            for (int i = 0; i < a.tiles; ++i) v += p[i * per];
        }
        *at<T, PLANES>(which ? a.g.dC : a.g.dB, b, t, g * N + n) = from_f32<T>(v);
    }
}

inline size_t selective_backward_shared(int lanes) {
    return sizeof(float) * ((size_t)kSelKeep * (kSelTile + 1) * 4 + 2 * kSelKeep * lanes * 4 + 3 * kSelKeep * (kSelTile + 1) +
                            (size_t)lanes * kSelKeep * 2 * 4 * lanes);
}

template <typename T, int LANES, bool PLANES> cudaError_t launch_selective_backward_as(const SelectiveArgs &a, cudaStream_t st) {
    const unsigned threads = kSelTile * LANES, grid = (unsigned)a.ctas() * a.segments;
    const size_t shared = selective_backward_shared(LANES);
    cudaError_t e = cudaSuccess;
    if (a.segments > 1) {
        if ((e = allow_shared(selective_backward_kernel<T, LANES, PLANES, true>, shared)) != cudaSuccess) return e;
        if ((e = launch_kernel(selective_backward_kernel<T, LANES, PLANES, true>, grid, threads, shared, st, 1, a)) != cudaSuccess) return e;
    }
    if ((e = allow_shared(selective_backward_kernel<T, LANES, PLANES, false>, shared)) != cudaSuccess) return e;
    if ((e = launch_kernel(selective_backward_kernel<T, LANES, PLANES, false>, grid, threads, shared, st, 1, a)) != cudaSuccess) return e;
    const long long outputs = (long long)a.s.B * a.s.T * a.s.G * 2 * a.s.N;
    const unsigned blocks = (unsigned)std::min<long long>((outputs + 255) / 256, 1 << 16);
    if ((e = launch_kernel(selective_sums_kernel<T, PLANES>, blocks, 256, 0, st, 1, a)) != cudaSuccess) return e;
    ColumnSums s = {};
    s.parts = a.s.B * a.segments;
    const size_t half = (size_t)s.parts * a.s.C;
    s.part[0] = a.part_a, s.part[1] = a.part_c, s.part[2] = a.part_c + half;
    s.out[0] = a.g.dA, s.out[1] = a.g.dD, s.out[2] = a.g.d_dt_bias;
    s.width[0] = a.s.C * a.s.N, s.width[1] = s.width[2] = a.s.C;
    return launch_column_sums(s, st);
}

template <typename T> cudaError_t launch_selective_backward(const SelectiveArgs &a, cudaStream_t st) {
    const bool planes = a.s.layout == WTCONV_SCAN_PLANES;
    switch (a.lanes) {
        case 2: return planes ? launch_selective_backward_as<T, 2, true>(a, st) : launch_selective_backward_as<T, 2, false>(a, st);
        case 4: return planes ? launch_selective_backward_as<T, 4, true>(a, st) : launch_selective_backward_as<T, 4, false>(a, st);
        case 8: return planes ? launch_selective_backward_as<T, 8, true>(a, st) : launch_selective_backward_as<T, 8, false>(a, st);
        default: return planes ? launch_selective_backward_as<T, 16, true>(a, st) : launch_selective_backward_as<T, 16, false>(a, st);
    }
}

}  // namespace wtconv
