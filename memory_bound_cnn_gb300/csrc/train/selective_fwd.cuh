// Forward of the selective scan and its one-token step.
#pragma once

#include "selective_device.cuh"

namespace wtconv {

// A CTA takes 32 channels of one sequence (or of a segment of it) in rounds of 32 positions.  LANES lanes with four states
// each scan a channel; the CTA's other warps, the helpers, compute d and d x of the next round's 32 x 32
// positions and channels once for all lanes, and finish the round before (sum the lanes' parts, D, gate, store).
// LOCAL: only the state that the segment ends with if it begins with 0, and the sum of its steps; the CTAs of
// later segments begin with what these compose to.
template <int LANES, bool PLANES> struct ForwardShared {
    using L = Layout<LANES, PLANES, kSelRound>;
    alignas(16) float2 coef[L::COEFS];  // d, d x
    alignas(16) float maps[2][kSelRound * L::MAP];
    alignas(16) float sums[L::PARTS * L::APART];  // over a channel's states
};

template <typename T, int LANES, bool PLANES, bool WIDE, bool LOCAL>
__global__ void __launch_bounds__(Roles<LANES>::THREADS, LANES == 2 ? 3 : LANES == 4 ? 2 : 1) selective_forward_kernel(const __grid_constant__ SelectiveArgs a) {
    using L = Layout<LANES, PLANES, kSelRound>;
    using R = Roles<LANES>;
    extern __shared__ float4 shared_memory[];
    ForwardShared<LANES, PLANES> *const rounds = reinterpret_cast<ForwardShared<LANES, PLANES> *>(shared_memory);  // two
    begin_kernel();
    const Place at_(a, blockIdx.x);
    if (LOCAL && at_.segment == a.segments - 1) return;  // its end is nobody's beginning
    const int b = at_.b, N = a.s.N, stop = min(at_.end, at_.length);
    const int count_rounds = stop > at_.first ? (stop - at_.first + kSelRound - 1) / kSelRound : 0;

    if (!R::scans()) {
        using Part = Share<PLANES, kSelTile, kSelRound, R::HELPERS, WIDE>;
        using Maps = Share<PLANES, L::PAD, kSelRound, R::HELPERS, WIDE>;
        using Two = typename Raw<T>::Two;
        const Part part(R::helper());
        const Maps maps(R::helper());
        const bool gated = !LOCAL && a.in.z.p != nullptr;
        Pair bias[Part::OWN], D[Part::OWN];
        part.parameters(a.in.dt_bias == nullptr ? nullptr : a.in.dt_bias + at_.c0, at_.channels, bias);
        part.parameters(a.in.D == nullptr ? nullptr : a.in.D + at_.c0, at_.channels, D);
        // two rounds ahead, in turns (moved from one place to another, a value would have to arrive first)
        struct Fetched {
            Two d[Part::COUNT], x[Part::COUNT], z[Part::COUNT], b[Maps::COUNT], c[Maps::COUNT];
        } even, odd;
        Two x[Part::COUNT], z[Part::COUNT], x_old[Part::COUNT] = {}, z_old[Part::COUNT] = {};  // of the scanned round, the one before
        using In = Cursor<const T, PLANES>;
        In d_at(part, a.in.dt, b, at_.first, at_.c0), x_at(part, a.in.x, b, at_.first, at_.c0), z_at(part, a.in.z, b, at_.first, at_.c0);
        In b_at(maps, a.in.Bm, b, at_.first, at_.group * N), c_at(maps, a.in.Cm, b, at_.first, at_.group * N);
        const auto fetch = [&](int r, Fetched &f) {
            if (r >= count_rounds) return;
            const int count = stop - at_.first - r * kSelRound;
            part.load(d_at.p, d_at.row, at_.channels, count, f.d), d_at.step(kSelRound);
            part.load(x_at.p, x_at.row, at_.channels, count, f.x), x_at.step(kSelRound);
            maps.load(b_at.p, b_at.row, N, count, f.b), b_at.step(kSelRound);
            if (!LOCAL) maps.load(c_at.p, c_at.row, N, count, f.c), c_at.step(kSelRound);
            if (gated) part.load(z_at.p, z_at.row, at_.channels, count, f.z), z_at.step(kSelRound);
        };
        const auto prepare = [&](int r, Fetched &f) {
            if (r >= count_rounds) return;
            ForwardShared<LANES, PLANES> &to = rounds[r & 1];
            arrived(f.d), arrived(f.x), arrived(f.b);
            if (!LOCAL) arrived(f.c);
            if (gated) arrived(f.z);
            const auto put = [&](int i, Pair d) {
                const Pair dx = mul(d, pair_of<T>(f.x[i]));
                // (past the end d x is what it may be: those positions are not scanned)
                if (part.busy())
                    *reinterpret_cast<float4 *>(to.coef + L::coef(part.position(i), part.channel(i))) = make_float4(d.lo(), dx.lo(), d.hi(), dx.hi());
            };
            if (a.s.softplus) {
#pragma unroll
                for (int i = 0; i < Part::COUNT; ++i) put(i, softplus_of(add(pair_of<T>(f.d[i]), bias[PLANES ? i : 0])));
            } else {
#pragma unroll
                for (int i = 0; i < Part::COUNT; ++i) put(i, add(pair_of<T>(f.d[i]), bias[PLANES ? i : 0]));
            }
            L::template put_map<T>(maps, f.b, to.maps[0]);
            if (!LOCAL) L::template put_map<T>(maps, f.c, to.maps[1]);
#pragma unroll
            for (int i = 0; i < Part::COUNT; ++i) x[i] = f.x[i], z[i] = f.z[i];
        };
        Cursor<T, PLANES> y_at(part, a.y, b, at_.first, at_.c0);
        const auto finish = [&](int r) {
            const int count = stop - at_.first - r * kSelRound;
            const float *const sums = rounds[r & 1].sums;
            const auto value = [&](int i) {
                const Pair s = L::get_sums(sums, L::value(part.position(i), part.channel(i)));
                return fma(D[PLANES ? i : 0], pair_of<T>(x_old[i]), s);
            };
            if (gated)
                part.store(y_at.p, y_at.row, at_.channels, count, [&](int i) {
                    const Pair g = pair_of<T>(z_old[i]);
                    return mul(value(i), mul(g, sigmoid_of(g)));
                });
            else
                part.store(y_at.p, y_at.row, at_.channels, count, value);
            y_at.step(kSelRound);
        };
        const auto during = [&](int r, Fetched &next, Fetched &after) {  // round r is scanned
            fetch(r + 2, after);
            if (!LOCAL && r > 0) finish(r - 1);
#pragma unroll
            for (int i = 0; i < Part::COUNT; ++i) x_old[i] = x[i], z_old[i] = z[i];
            prepare(r + 1, next);
            R::meet();
        };
        fetch(0, even), fetch(1, odd), prepare(0, even);
        R::meet();
        for (int r = 0; r < count_rounds; r += 2) {
            during(r, odd, even);
            if (r + 1 < count_rounds) during(r + 1, even, odd);
        }
        if (!LOCAL && count_rounds > 0) finish(count_rounds - 1);
        if (!LOCAL)  // positions past the sequence's end
            for (int t0 = max(at_.first, at_.length); t0 < at_.end; t0 += kSelRound)
                part.clear(part.mine(at<T, PLANES>(a.y, b, t0, at_.c0), a.y.row), a.y.row, at_.channels, at_.end - t0);
        return;
    }

    const LanePlace<LANES> lane;
    const int c = lane.c, quad = lane.quad, n0 = lane.n0;
    const bool live = c < at_.channels;
    Quad decay = {Pair(0.f), Pair(0.f)}, h = {Pair(0.f), Pair(0.f)};
    if (live) {
        decay = load_rates(a.in.A + (long long)(at_.c0 + c) * N, n0, N);
        decay.a = mul(decay.a, Pair(kSelLog2E)), decay.b = mul(decay.b, Pair(kSelLog2E));
    }
    if (!LOCAL && live) {
        if (a.in.h0 != nullptr) h = load_quad(a.in.h0 + ((long long)b * a.s.C + at_.c0 + c) * N, n0, N);
        if (count_rounds > 0)
#pragma unroll 4
            for (int k = 0; k < at_.segment; ++k) {
                const long long i = ((long long)b * a.segments + k) * a.s.C + at_.c0 + c;
                const Pair d(0.25f * a.steps[i]);
                const Quad u = quad_of(*reinterpret_cast<const float4 *>(a.ends + i * L::PAD + n0));
                h.a = through_part(mul(d, decay.a), h.a, u.a), h.b = through_part(mul(d, decay.b), h.b, u.b);
            }
    }
    float step_sum = 0.f;
    float *states = nullptr;  // the lane's of the next kept position
    if (!LOCAL && live && a.states_out != nullptr)
        states = a.states_out + (((long long)b * a.keep + at_.first / kSelKeep) * a.s.C + at_.c0 + c) * L::PAD + n0;
    R::meet();
    for (int r = 0; r < count_rounds; ++r) {
        ForwardShared<LANES, PLANES> &s = rounds[r & 1];
        const int count = min(kSelRound, stop - at_.first - r * kSelRound);
        // Four positions at a time, what the next four need is loaded before their sums are stored: a load of shared
        // memory is not moved above a store, and would wait for all that the store waits for.
        constexpr int TOGETHER = L::TOGETHER, BATCH = 4;
        struct Operands {
            float2 q;
            float4 u, o;
        };
        const auto operands = [&](int t) {
            Operands p;
            p.q = s.coef[L::coef(t, c)], p.u = *reinterpret_cast<const float4 *>(s.maps[0] + t * L::MAP + n0);
            if (!LOCAL) p.o = *reinterpret_cast<const float4 *>(s.maps[1] + t * L::MAP + n0);
            return p;
        };
        const auto step = [&](const Operands &p) {  // one position; its sum over the lane's states
            const Quad u = quad_of(p.u);
            const Pair d(p.q.x), dx(p.q.y);
            h.a = fma(decays_of(d, decay.a), h.a, mul(dx, u.a));
            h.b = fma(decays_of(d, decay.b), h.b, mul(dx, u.b));
            if (LOCAL) {
                step_sum += p.q.x;
                return 0.f;
            }
            const Quad o = quad_of(p.o);
            const Pair v = fma(o.a, h.a, mul(o.b, h.b));
            return v.lo() + v.hi();
        };
        const auto keep = [&](int t) {
            if (!LOCAL && t % kSelKeep == 0 && states != nullptr) {
                *reinterpret_cast<float4 *>(states) = float4_of(h);
                states += (long long)a.s.C * L::PAD;
            }
        };
        if (count == kSelRound) {
            Operands now[BATCH], next[BATCH];
#pragma unroll
            for (int j = 0; j < BATCH; ++j) now[j] = operands(j);
#pragma unroll(kSelKeep / BATCH)
            for (int t = 0; t < kSelRound; t += BATCH) {
                keep(t);
                const int ahead = min(t + BATCH, kSelRound - BATCH);
#pragma unroll
                for (int j = 0; j < BATCH; ++j) next[j] = operands(ahead + j);
                float v[BATCH / TOGETHER][TOGETHER];
#pragma unroll
                for (int j = 0; j < BATCH; ++j) v[j / TOGETHER][j % TOGETHER] = step(now[j]);
                if (!LOCAL) {
#pragma unroll
                    for (int j = 0; j < BATCH / TOGETHER; ++j) L::put_sums(s.sums, t + j * TOGETHER, c, quad, v[j]);
                }
#pragma unroll
                for (int j = 0; j < BATCH; ++j) now[j] = next[j];
            }
        } else {
            for (int t = 0; t < count; t += TOGETHER) {
                keep(t);
                float v[TOGETHER];
#pragma unroll
                for (int j = 0; j < TOGETHER; ++j) v[j] = t + j < count ? step(operands(t + j)) : 0.f;
                if (!LOCAL) L::put_sums(s.sums, t, c, quad, v);
            }
        }
        R::meet();
    }

    if (LOCAL) {
        if (live && count_rounds > 0) {
            const long long i = ((long long)b * a.segments + at_.segment) * a.s.C + at_.c0 + c;
            *reinterpret_cast<float4 *>(a.ends + i * L::PAD + n0) = float4_of(h);
            if (quad == 0) a.steps[i] = step_sum;
        }
        return;
    }
    // the sequence ends in this segment
    if (a.h_last != nullptr && live && (at_.segment == 0 ? at_.length <= at_.end : at_.first < at_.length && at_.length <= at_.end))
        store_quad(a.h_last + ((long long)b * a.s.C + at_.c0 + c) * N, n0, N, h);
}

template <typename T, int LANES, bool PLANES, bool WIDE> cudaError_t launch_selective_forward_as(const SelectiveArgs &a, cudaStream_t st) {
    const unsigned threads = Roles<LANES>::THREADS, grid = (unsigned)a.ctas() * a.segments;
    const size_t shared = 2 * sizeof(ForwardShared<LANES, PLANES>);
    const auto local = selective_forward_kernel<T, LANES, PLANES, WIDE, true>, whole = selective_forward_kernel<T, LANES, PLANES, WIDE, false>;
    cudaError_t e = cudaSuccess;
    if (a.segments > 1) {
        if ((e = allow_shared(local, shared)) != cudaSuccess) return e;
        if ((e = launch_kernel(local, grid, threads, shared, st, 1, a)) != cudaSuccess) return e;
    }
    if ((e = allow_shared(whole, shared)) != cudaSuccess) return e;
    return launch_kernel(whole, grid, threads, shared, st, 1, a);
}

template <typename T> cudaError_t launch_selective_forward(const SelectiveArgs &a, cudaStream_t st) {
    return with_selective_shape(a, [&](auto lanes, auto planes, auto wide) {
        return launch_selective_forward_as<T, decltype(lanes)::value, decltype(planes)::value, decltype(wide)::value>(a, st);
    });
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
            h = load_quad(row, n0, N), A = load_rates(a.in.A + (long long)c * N, n0, N);
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
        if (a.s.softplus) d = softplus_of(Pair(d)).lo();
        const Pair rate(d * kSelLog2E), dx(d * x);
        h.a = fma(decays_of(rate, A.a), h.a, mul(dx, in.a)), h.b = fma(decays_of(rate, A.b), h.b, mul(dx, in.b));
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
            v *= z * sigmoid_of(Pair(z)).lo();
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
