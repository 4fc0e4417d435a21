// Forward of the selective scan and its one-token step.
#pragma once

#include "selective_device.cuh"

namespace wtconv {

// A CTA scans 32 channels of one sequence (or of a segment of it), LANES lanes with four states each to a
// channel.  It works in rounds of 32 positions: every thread computes d and d x of its share of the round's
// 32 x 32 positions and channels once, all lanes then scan the round out of shared memory, sums over the states
// meet by exchanges between lanes, and the epilogue (D, gate, store) goes by the share again.
// LOCAL: only the state that the segment ends with if it begins with 0, and the sum of its steps; the CTAs of
// later segments begin with what these compose to.
template <typename T, int LANES, bool PLANES, bool LOCAL>
__global__ void __launch_bounds__(kSelTile *LANES) selective_forward_kernel(const __grid_constant__ SelectiveArgs a) {
    constexpr int THREADS = kSelTile * LANES, SHARE = kSelTile * kSelRound / THREADS, PAD = 4 * LANES, ROW = kSelTile + 1;
    __shared__ float2 coef[kSelRound * ROW];  // d, d x
    __shared__ float4 bs[kSelRound * LANES], cs[LOCAL ? 1 : kSelRound * LANES];
    __shared__ float sums[LOCAL ? 1 : kSelRound * ROW];
    begin_kernel();
    const Place at_(a, blockIdx.x);
    if (LOCAL && at_.segment == a.segments - 1) return;  // its end is nobody's beginning
    const int tid = threadIdx.x, b = at_.b, N = a.s.N, stop = min(at_.end, at_.length);
    const int c = tid / LANES, quad = tid % LANES, n0 = 4 * quad;  // the lane's channel and states
    const bool live = c < at_.channels;
    Quad decay = {Pair(0.f), Pair(0.f)}, h = {Pair(0.f), Pair(0.f)};
    if (live) {
        decay = load_quad(a.in.A + (long long)(at_.c0 + c) * N, n0, N);
        decay.a = mul(decay.a, Pair(kSelLog2E)), decay.b = mul(decay.b, Pair(kSelLog2E));
    }
    if (!LOCAL && live) {
        if (a.in.h0 != nullptr) h = load_quad(a.in.h0 + ((long long)b * a.s.C + at_.c0 + c) * N, n0, N);
        if (at_.first < at_.length)
            for (int k = 0; k < at_.segment; ++k) {
                const long long i = ((long long)b * a.segments + k) * a.s.C + at_.c0 + c;
                const Pair d(a.steps[i]);
                const Quad u = quad_of(*reinterpret_cast<const float4 *>(a.ends + i * PAD + n0));
                h.a = fma(exp2_fast(mul(d, decay.a)), h.a, u.a), h.b = fma(exp2_fast(mul(d, decay.b)), h.b, u.b);
            }
    }
    float step_sum = 0.f;

    for (int t0 = at_.first; t0 < stop; t0 += kSelRound) {
        const int count = min(kSelRound, stop - t0);
        float x[SHARE], z[SHARE];
#pragma unroll
        for (int i = 0; i < SHARE; ++i) {
            const int e = tid + i * THREADS, pc = PLANES ? e / kSelRound : e % kSelTile, pt = PLANES ? e % kSelRound : e / kSelTile;
            float d = 0.f;
            x[i] = z[i] = 0.f;
            if (pc < at_.channels && pt < count) {
                x[i] = to_f32(*at<const T, PLANES>(a.in.x, b, t0 + pt, at_.c0 + pc));
                if (!LOCAL && a.in.z.p != nullptr) z[i] = to_f32(*at<const T, PLANES>(a.in.z, b, t0 + pt, at_.c0 + pc));
                d = to_f32(*at<const T, PLANES>(a.in.dt, b, t0 + pt, at_.c0 + pc));
                if (a.in.dt_bias != nullptr) d += a.in.dt_bias[at_.c0 + pc];
                if (a.s.softplus) d = softplus_of(d).value;
            }
            coef[pt * ROW + pc] = make_float2(d, d * x[i]);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int e = tid + i * THREADS, n = PLANES ? e / kSelRound : e % PAD, pt = PLANES ? e % kSelRound : e / PAD;
            const bool ok = n < N && pt < count;
            const int state = at_.group * N + n;
            reinterpret_cast<float *>(bs)[pt * PAD + n] = ok ? to_f32(*at<const T, PLANES>(a.in.Bm, b, t0 + pt, state)) : 0.f;
            if (!LOCAL)
                reinterpret_cast<float *>(cs)[pt * PAD + n] = ok ? to_f32(*at<const T, PLANES>(a.in.Cm, b, t0 + pt, state)) : 0.f;
        }
        __syncthreads();

        const auto step = [&](int t) {  // one position; its sum over the lane's states
            const float2 q = coef[t * ROW + c];
            const Quad u = quad_of(bs[t * LANES + quad]);
            const Pair d(q.x), dx(q.y);
            h.a = fma(exp2_fast(mul(d, decay.a)), h.a, mul(dx, u.a));
            h.b = fma(exp2_fast(mul(d, decay.b)), h.b, mul(dx, u.b));
            if (LOCAL) {
                step_sum += q.x;
                return 0.f;
            }
            const Quad o = quad_of(cs[t * LANES + quad]);
            const Pair s = fma(o.a, h.a, mul(o.b, h.b));
            return s.lo() + s.hi();
        };
        const auto keep = [&](int t) {
            if (!LOCAL && t % kSelKeep == 0 && a.states_out != nullptr && live) {
                const long long k = (long long)b * a.keep + (t0 + t) / kSelKeep;
                *reinterpret_cast<float4 *>(a.states_out + (k * a.s.C + at_.c0 + c) * PAD + n0) = float4_of(h);
            }
        };
        for (int t = 0; t < count; t += LANES) {
            keep(t);
            float s[LANES];
            if (t + LANES <= count) {
#pragma unroll
                for (int j = 0; j < LANES; ++j) s[j] = step(t + j);
            } else {
#pragma unroll
                for (int j = 0; j < LANES; ++j) s[j] = t + j < count ? step(t + j) : 0.f;
            }
            if (!LOCAL) {
                sum_exchange<LANES, 1>(s, quad);
                sums[(t + quad) * ROW + c] = s[0];
            }
        }
        __syncthreads();
        if (!LOCAL) {
#pragma unroll
            for (int i = 0; i < SHARE; ++i) {
                const int e = tid + i * THREADS, pc = PLANES ? e / kSelRound : e % kSelTile, pt = PLANES ? e % kSelRound : e / kSelTile;
                if (pc >= at_.channels || pt >= count) continue;
                float v = sums[pt * ROW + pc];
                if (a.in.D != nullptr) v = fmaf(a.in.D[at_.c0 + pc], x[i], v);
                if (a.in.z.p != nullptr) v *= z[i] * sigmoid_of(z[i]);
                *at<T, PLANES>(a.y, b, t0 + pt, at_.c0 + pc) = from_f32<T>(v);
            }
        }
    }

    if (LOCAL) {
        if (live && at_.first < at_.length) {
            const long long i = ((long long)b * a.segments + at_.segment) * a.s.C + at_.c0 + c;
            *reinterpret_cast<float4 *>(a.ends + i * PAD + n0) = float4_of(h);
            if (quad == 0) a.steps[i] = step_sum;
        }
        return;
    }
    // the sequence ends in this segment
    if (a.h_last != nullptr && live && (at_.segment == 0 ? at_.length <= at_.end : at_.first < at_.length && at_.length <= at_.end))
        store_quad(a.h_last + ((long long)b * a.s.C + at_.c0 + c) * N, n0, N, h);
    // positions past its end
    for (int t0 = max(at_.first, at_.length); t0 < at_.end; t0 += kSelRound) {
#pragma unroll
        for (int i = 0; i < SHARE; ++i) {
            const int e = tid + i * THREADS, pc = PLANES ? e / kSelRound : e % kSelTile, pt = PLANES ? e % kSelRound : e / kSelTile;
            if (pc < at_.channels && pt < at_.end - t0) *at<T, PLANES>(a.y, b, t0 + pt, at_.c0 + pc) = from_f32<T>(0.f);
        }
    }
}

template <typename T, int LANES, bool PLANES> cudaError_t launch_selective_forward_as(const SelectiveArgs &a, cudaStream_t st) {
    const unsigned threads = kSelTile * LANES, grid = (unsigned)a.ctas() * a.segments;
    if (a.segments > 1) {
        const cudaError_t e = launch_kernel(selective_forward_kernel<T, LANES, PLANES, true>, grid, threads, 0, st, 1, a);
        if (e != cudaSuccess) return e;
    }
    return launch_kernel(selective_forward_kernel<T, LANES, PLANES, false>, grid, threads, 0, st, 1, a);
}

template <typename T> cudaError_t launch_selective_forward(const SelectiveArgs &a, cudaStream_t st) {
    const bool planes = a.s.layout == WTCONV_SCAN_PLANES;
    switch (a.lanes) {
        case 2: return planes ? launch_selective_forward_as<T, 2, true>(a, st) : launch_selective_forward_as<T, 2, false>(a, st);
        case 4: return planes ? launch_selective_forward_as<T, 4, true>(a, st) : launch_selective_forward_as<T, 4, false>(a, st);
        case 8: return planes ? launch_selective_forward_as<T, 8, true>(a, st) : launch_selective_forward_as<T, 8, false>(a, st);
        default: return planes ? launch_selective_forward_as<T, 16, true>(a, st) : launch_selective_forward_as<T, 16, false>(a, st);
    }
}

// One position of every sequence: LANES lanes to a channel, each with four of its states.
template <typename T, int LANES, bool WIDE>
__global__ void __launch_bounds__(128) selective_step_kernel(const __grid_constant__ SelectiveArgs a, float *pool, int n_states,
                                                             const int *slots) {
    constexpr int CHANNELS = 128 / LANES;
    begin_kernel();
    const int tiles = (a.s.C + CHANNELS - 1) / CHANNELS, b = blockIdx.x / tiles, N = a.s.N;
    const int c = blockIdx.x % tiles * CHANNELS + threadIdx.x / LANES, quad = threadIdx.x % LANES, n0 = 4 * quad;
    const int slot = slots == nullptr ? b : slots[b];
    const bool live = c < a.s.C, busy = live && slot >= 0 && slot < n_states;
    float v = 0.f, x = 0.f;
    if (busy) {
        float *row = pool + ((long long)slot * a.s.C + c) * N;
        const int state = c / a.channels * N;
        Quad h = {Pair(0.f), Pair(0.f)}, A = h, in = h, out = h;
        if (WIDE && n0 < N) {
            h = quad_of(*reinterpret_cast<const float4 *>(row + n0));
            A = quad_of(*reinterpret_cast<const float4 *>(a.in.A + (long long)c * N + n0));
        } else if (!WIDE) {
            h = load_quad(row, n0, N), A = load_quad(a.in.A + (long long)c * N, n0, N);
        }
        const T *bp = static_cast<const T *>(a.in.Bm.p) + b * a.in.Bm.row + state;
        const T *cp = static_cast<const T *>(a.in.Cm.p) + b * a.in.Cm.row + state;
        float bn[4], cn[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) bn[i] = n0 + i < N ? to_f32(bp[n0 + i]) : 0.f, cn[i] = n0 + i < N ? to_f32(cp[n0 + i]) : 0.f;
        in = {Pair(bn[0], bn[1]), Pair(bn[2], bn[3])}, out = {Pair(cn[0], cn[1]), Pair(cn[2], cn[3])};
        x = to_f32(static_cast<const T *>(a.in.x.p)[b * a.in.x.row + c]);
        float d = to_f32(static_cast<const T *>(a.in.dt.p)[b * a.in.dt.row + c]);
        if (a.in.dt_bias != nullptr) d += a.in.dt_bias[c];
        if (a.s.softplus) d = softplus_of(d).value;
        const Pair rate(d * kSelLog2E), dx(d * x);
        h.a = fma(exp2_fast(mul(rate, A.a)), h.a, mul(dx, in.a)), h.b = fma(exp2_fast(mul(rate, A.b)), h.b, mul(dx, in.b));
        if (WIDE && n0 < N) *reinterpret_cast<float4 *>(row + n0) = float4_of(h);
        if (!WIDE) store_quad(row, n0, N, h);
        const Pair s = fma(out.a, h.a, mul(out.b, h.b));
        v = s.lo() + s.hi();
    }
#pragma unroll
    for (int w = LANES / 2; w >= 1; w /= 2) v += __shfl_xor_sync(0xffffffffu, v, w);
    if (!live || quad != 0) return;
    if (busy) {
        if (a.in.D != nullptr) v = fmaf(a.in.D[c], x, v);
        if (a.in.z.p != nullptr) {
            const float z = to_f32(static_cast<const T *>(a.in.z.p)[b * a.in.z.row + c]);
            v *= z * sigmoid_of(z);
        }
    }
    static_cast<T *>(a.y.p)[b * a.y.row + c] = from_f32<T>(v);
}

template <typename T, int LANES>
cudaError_t launch_selective_step_as(const SelectiveArgs &a, float *pool, int n_states, const int *slots, cudaStream_t st) {
    const unsigned grid = (unsigned)a.s.B * ceil_div(a.s.C, 128 / LANES);
    const bool wide = a.s.N % 4 == 0 && aligned_to(pool, 16) && aligned_to(a.in.A, 16);
    return wide ? launch_kernel(selective_step_kernel<T, LANES, true>, grid, 128, 0, st, 1, a, pool, n_states, slots)
                : launch_kernel(selective_step_kernel<T, LANES, false>, grid, 128, 0, st, 1, a, pool, n_states, slots);
}

template <typename T>
cudaError_t launch_selective_step(const SelectiveArgs &a, float *pool, int n_states, const int *slots, cudaStream_t st) {
    switch (a.lanes) {
        case 2: return launch_selective_step_as<T, 2>(a, pool, n_states, slots, st);
        case 4: return launch_selective_step_as<T, 4>(a, pool, n_states, slots, st);
        case 8: return launch_selective_step_as<T, 8>(a, pool, n_states, slots, st);
        default: return launch_selective_step_as<T, 16>(a, pool, n_states, slots, st);
    }
}

}  // namespace wtconv
