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
// sums, those over a channel's states are put down by its lanes and meet in the epilogue; those over channels (dB, dC)
// meet by exchanges between the warp's channels, then between warps in shared memory, then between CTAs in
// selective_sums_kernel.  Lanes of neighbouring channels hold their four states in different orders (state n0 +
// (i ^ order) in place i), so that what a lane sends in such an exchange and what it keeps are the same places in
// all lanes; B and C lie in shared memory in each of the orders.
// LOCAL: only the gradient that the segment's beginning passes on if nothing enters at its end, and the sum
// of its steps; the CTAs of earlier segments begin with what these compose to.
template <int LANES, bool PLANES> struct BackwardShared {
    using Part = Share<PLANES, LANES, kSelKeep, false>;
    static constexpr int PAD = 4 * LANES, COPIES = LANES == 16 ? 2 : 4;
    float2 coef[Part::COEFS];                       // d, d x
    float r[Part::VALUES];                          // dy silu(z)
    float sums[3][Part::PARTS * Part::APART];       // over a channel's states: g B, k A, C h
    static constexpr int APART = kSelKeep * PAD + (LANES == 16 ? 16 : 8);  // of two copies: their lanes meet on no bank
    alignas(16) float maps[2][COPIES][APART];                   // B, C
    float2 stash[2][Part::COUNT][Part::THREADS];    // of a thread's pairs, for the epilogue: slope of d, dy silu'(z)
    float part[LANES][kSelKeep][2][PAD];            // dB and dC of a warp's channels
};

template <typename T, int LANES, bool PLANES, bool WIDE, bool LOCAL>
__global__ void __launch_bounds__(kSelTile *LANES, LANES == 16 ? 1 : 12 / LANES) selective_backward_kernel(const __grid_constant__ SelectiveArgs a) {
    constexpr int THREADS = kSelTile * LANES, BLOCK = kSelKeep, PAD = 4 * LANES, CHANNELS = 32 / LANES;
    using Part = Share<PLANES, LANES, BLOCK, WIDE>;
    using Maps = MapShare<PLANES, LANES, BLOCK>;
    using Shared = BackwardShared<LANES, PLANES>;
    constexpr int COUNT = Part::COUNT, OWN = Part::OWN, TOGETHER = Part::TOGETHER;
    extern __shared__ float4 shared_memory[];
    Shared &s = *reinterpret_cast<Shared *>(shared_memory);
    begin_kernel();
    const Place at_(a, blockIdx.x);
    if (LOCAL && at_.segment == 0) return;  // nobody is before it
    const int tid = threadIdx.x, b = at_.b, N = a.s.N, stop = min(at_.end, at_.length);
    const LanePlace<LANES> lane;
    const int c = lane.c, quad = lane.quad, n0 = lane.n0;
    // (two lanes that read the same order are neighbours, as those that read the same states: see LanePlace)
    const int order = CHANNELS >= 8 ? lane.cl >> 1 & 3 : CHANNELS == 4 ? lane.cl : 2 * lane.cl;
    const bool live = c < at_.channels, gated = a.in.z.p != nullptr;
    const long long row = (long long)b * a.s.C + at_.c0 + c;  // of [B][C]
    const Part mine;
    const Maps maps;
    const int blocks = stop > at_.first ? (stop - at_.first + BLOCK - 1) / BLOCK : 0;
    typename Raw<T>::Two x_next[COUNT], d_next[COUNT], z_next[COUNT], dy_next[COUNT];
    uint32_t b_next[Maps::COUNT], c_next[Maps::COUNT];
    float4 kept_next = make_float4(0.f, 0.f, 0.f, 0.f);
    const auto fetch = [&](int k) {
        const int t0 = at_.first + k * BLOCK, count = stop - t0;
        mine.load(at<const T, PLANES>(a.in.dt, b, t0, at_.c0), a.in.dt.row, at_.channels, count, d_next);
        mine.load(at<const T, PLANES>(a.dy, b, t0, at_.c0), a.dy.row, at_.channels, count, dy_next);
        if (gated) mine.load(at<const T, PLANES>(a.in.z, b, t0, at_.c0), a.in.z.row, at_.channels, count, z_next);
        maps.load(at<const T, PLANES>(a.in.Cm, b, t0, at_.group * N), a.in.Cm.row, N, count, c_next);
        if (LOCAL) return;
        mine.load(at<const T, PLANES>(a.in.x, b, t0, at_.c0), a.in.x.row, at_.channels, count, x_next);
        maps.load(at<const T, PLANES>(a.in.Bm, b, t0, at_.group * N), a.in.Bm.row, N, count, b_next);
        if (live)
            kept_next = *reinterpret_cast<const float4 *>(
                a.states_in + (((long long)b * a.keep + t0 / kSelKeep) * a.s.C + at_.c0 + c) * PAD + n0);
    };
    if (blocks > 0) fetch(blocks - 1);
    Pair bias[OWN], D[OWN];
    mine.parameters(a.in.dt_bias == nullptr ? nullptr : a.in.dt_bias + at_.c0, at_.channels, bias);
    mine.parameters(a.in.D == nullptr ? nullptr : a.in.D + at_.c0, at_.channels, D);
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
    decay = reordered(decay, order), carry = reordered(carry, order);
    float step_sum = 0.f;
    Pair dD[OWN], d_bias[OWN];
#pragma unroll
    for (int i = 0; i < OWN; ++i) dD[i] = d_bias[i] = Pair(0.f);
    const float4 *const bs = reinterpret_cast<const float4 *>(s.maps[0][order / (4 / Shared::COPIES)]) + quad;
    const float4 *const cs = reinterpret_cast<const float4 *>(s.maps[1][order / (4 / Shared::COPIES)]) + quad;

    for (int k = blocks - 1; k >= 0; --k) {
        const int t0 = at_.first + k * BLOCK, count = min(BLOCK, stop - t0);
        if (!LOCAL) asm volatile("" : "+f"(kept_next.x), "+f"(kept_next.y), "+f"(kept_next.z), "+f"(kept_next.w));  // (see arrived)
        const Quad before = reordered(quad_of(kept_next), order);
        typename Raw<T>::Two x[COUNT];
        arrived(d_next), arrived(dy_next), arrived(c_next);
        if (!LOCAL) arrived(x_next), arrived(b_next);
        if (gated) arrived(z_next);
#pragma unroll
        for (int i = 0; i < COUNT; ++i) {
            x[i] = x_next[i];
            if (!mine.busy()) continue;
            const int t = mine.position(i), at_c = mine.channel(i);
            Pair d = add(pair_of<T>(d_next[i]), bias[PLANES ? i : 0]), r = pair_of<T>(dy_next[i]);
            if (a.s.softplus) {
                const Pair e = exp_of_minus_abs(d);
                if (!LOCAL) *reinterpret_cast<unsigned long long *>(&s.stash[0][i][tid]) = softplus_slope(d, e).q;
                d = softplus_of(d, e);
            }
            if (gated) {
                const Pair z = pair_of<T>(z_next[i]), p = sigmoid_of(z), zp = mul(z, p);
                // silu'(z) = p + z p (1 - p)
                if (!LOCAL) *reinterpret_cast<unsigned long long *>(&s.stash[1][i][tid]) = mul(r, fma(zp, sub(Pair(1.f), p), p)).q;
                r = mul(r, zp);
            }
            const Pair dx = LOCAL ? Pair(0.f) : mul(d, pair_of<T>(x[i]));
            *reinterpret_cast<float4 *>(s.coef + mine.coef(t, at_c)) = make_float4(d.lo(), dx.lo(), d.hi(), dx.hi());
            *reinterpret_cast<unsigned long long *>(s.r + mine.value(t, at_c)) = r.q;
        }
        if (!LOCAL) maps.template put<T, Shared::COPIES, Shared::APART>(b_next, s.maps[0][0]);
        maps.template put<T, Shared::COPIES, Shared::APART>(c_next, s.maps[1][0]);
        __syncthreads();
        if (k > 0) fetch(k - 1);  // while this block is gone through

        if (LOCAL) {
            const auto pass = [&](int t) {
                const float2 q = s.coef[mine.coef(t, c)];
                const Quad o = quad_of(cs[t * LANES]);
                const Pair d(q.x), r(s.r[mine.value(t, c)]);
                carry.a = mul(exp2_fast(mul(d, decay.a)), fma(o.a, r, carry.a));
                carry.b = mul(exp2_fast(mul(d, decay.b)), fma(o.b, r, carry.b));
                step_sum += q.x;
            };
            if (count == BLOCK) {
#pragma unroll
                for (int t = BLOCK - 1; t >= 0; --t) pass(t);
            } else {
                for (int t = count - 1; t >= 0; --t) pass(t);
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
                const float2 q = s.coef[mine.coef(t, c)];
                const Quad u = quad_of(bs[t * LANES]), last = t == 0 ? before : h[t == 0 ? 0 : t - 1];
                const Pair d(q.x), dx(q.y);
                h[t].a = fma(exp2_fast(mul(d, decay.a)), last.a, mul(dx, u.a));
                h[t].b = fma(exp2_fast(mul(d, decay.b)), last.b, mul(dx, u.b));
            }
            Quad dA_block = {Pair(0.f), Pair(0.f)};
            // (what a position needs is loaded before the one after it is stored, as in the forward)
            struct Operands {
                float2 q;
                float4 u, o;
                float r;
            };
            const auto operands = [&](int t) { return Operands{s.coef[mine.coef(t, c)], bs[t * LANES], cs[t * LANES], s.r[mine.value(t, c)]}; };
            Operands next = operands(FULL ? BLOCK - 1 : count - 1);
#pragma unroll
            for (int batch = BLOCK / TOGETHER - 1; batch >= 0; --batch) {
                if (!FULL && batch * TOGETHER >= count) continue;
                float s1[TOGETHER], s2[TOGETHER], s3[TOGETHER];
#pragma unroll
                for (int j = TOGETHER - 1; j >= 0; --j) {
                    const int t = batch * TOGETHER + j;
                    s1[j] = s2[j] = s3[j] = 0.f;
                    if (!FULL && t >= count) continue;
                    const Operands now = next;
                    if (t > 0) next = operands(t - 1);
                    const Quad u = quad_of(now.u), o = quad_of(now.o), last = t == 0 ? before : h[t == 0 ? 0 : t - 1];
                    const Pair d(now.q.x), dx(now.q.y), r(now.r);
                    const Quad g = {fma(o.a, r, carry.a), fma(o.b, r, carry.b)};
                    carry.a = mul(exp2_again(mul(d, decay.a)), g.a), carry.b = mul(exp2_again(mul(d, decay.b)), g.b);
                    const Quad kk = {mul(carry.a, last.a), mul(carry.b, last.b)};
                    dA_block.a = fma(kk.a, d, dA_block.a), dA_block.b = fma(kk.b, d, dA_block.b);
                    const Pair p1 = fma(g.a, u.a, mul(g.b, u.b)), p2 = fma(kk.a, decay.a, mul(kk.b, decay.b));
                    const Pair p3 = fma(o.a, h[t].a, mul(o.b, h[t].b));
                    s1[j] = p1.lo() + p1.hi(), s2[j] = p2.lo() + p2.hi(), s3[j] = p3.lo() + p3.hi();
                    // over the warp's channels: first lanes whose orders differ in 2 (a lane keeps its places 0 and 1), then
                    // in 1 (it keeps place 0)
                    constexpr int FIRST = CHANNELS >= 8 ? 4 : CHANNELS / 2;
                    const auto swap = [](float v, int m) { return __shfl_xor_sync(0xffffffffu, v, m); };
                    const Pair b1 = mul(g.b, dx), c1 = mul(h[t].b, r);
                    const Pair db = fma(g.a, dx, Pair(swap(b1.lo(), FIRST), swap(b1.hi(), FIRST)));
                    const Pair dc = fma(h[t].a, r, Pair(swap(c1.lo(), FIRST), swap(c1.hi(), FIRST)));
                    float(&to)[2][PAD] = s.part[lane.warp][t];
                    if constexpr (CHANNELS == 2) {
                        float(&mine_of)[PAD] = to[0], (&other)[PAD] = to[1];
                        mine_of[n0 + order] = db.lo(), mine_of[n0 + (order ^ 1)] = db.hi();
                        other[n0 + order] = dc.lo(), other[n0 + (order ^ 1)] = dc.hi();
                    } else {
                        const float vb = db.lo() + swap(db.hi(), FIRST / 2), vc = dc.lo() + swap(dc.hi(), FIRST / 2);
                        if constexpr (CHANNELS == 4) {
                            to[0][n0 + order] = vb, to[1][n0 + order] = vc;
                        } else {
                            const bool odd = lane.cl & 1;
                            float v = (odd ? vc : vb) + swap(odd ? vb : vc, 1);
                            if (CHANNELS == 16) v += swap(v, 8);
                            if (CHANNELS == 8 || lane.cl < 8) to[odd][n0 + order] = v;
                        }
                    }
                }
                Part::put_sums(s.sums[0], batch * TOGETHER, c, quad, s1);
                Part::put_sums(s.sums[1], batch * TOGETHER, c, quad, s2);
                Part::put_sums(s.sums[2], batch * TOGETHER, c, quad, s3);
            }
            dA.a = add(dA.a, dA_block.a), dA.b = add(dA.b, dA_block.b);
        };
        if (count == BLOCK) scan(std::true_type{});
        else scan(std::false_type{});
        __syncthreads();

        Pair dx[COUNT], dd[COUNT], dz[COUNT];
        const auto sum = [&](int which, int place) { return Part::get_sums(s.sums[which], place); };
#pragma unroll
        for (int i = 0; i < COUNT; ++i) {
            if (!mine.busy()) continue;
            const int t = mine.position(i), at_c = mine.channel(i), place = mine.value(t, at_c);
            // (an element past the end or beside the tile has whatever an earlier block left: it is neither stored nor summed)
            const float4 q = *reinterpret_cast<const float4 *>(s.coef + mine.coef(t, at_c));
            const Pair into = sum(0, place), xi = pair_of<T>(x[i]), r(*reinterpret_cast<const unsigned long long *>(s.r + place)), Di = D[PLANES ? i : 0];
            dd[i] = fma(xi, into, mul(sum(1, place), Pair(kSelLn2)));
            if (a.s.softplus) dd[i] = mul(dd[i], Pair(*reinterpret_cast<const unsigned long long *>(&s.stash[0][i][tid])));
            dx[i] = fma(Di, r, mul(Pair(q.x, q.z), into));
            if (gated) dz[i] = mul(Pair(*reinterpret_cast<const unsigned long long *>(&s.stash[1][i][tid])), fma(Di, xi, sum(2, place)));
            Pair rx = mul(r, xi), di = dd[i];
            if (count < BLOCK || at_.channels < kSelTile) {
                const bool first = mine.in(i, 0, at_.channels, count), second = mine.in(i, 1, at_.channels, count);
                rx = {first ? rx.lo() : 0.f, second ? rx.hi() : 0.f}, di = {first ? di.lo() : 0.f, second ? di.hi() : 0.f};
            }
            dD[PLANES ? i : 0] = add(dD[PLANES ? i : 0], rx), d_bias[PLANES ? i : 0] = add(d_bias[PLANES ? i : 0], di);
        }
        mine.store(at<T, PLANES>(a.g.dx, b, t0, at_.c0), a.g.dx.row, at_.channels, count, [&](int i) { return dx[i]; });
        mine.store(at<T, PLANES>(a.g.d_dt, b, t0, at_.c0), a.g.d_dt.row, at_.channels, count, [&](int i) { return dd[i]; });
        if (gated) mine.store(at<T, PLANES>(a.g.dz, b, t0, at_.c0), a.g.dz.row, at_.channels, count, [&](int i) { return dz[i]; });
        float *const to = a.part_bc + (((long long)at_.tile * a.s.B + b) * a.s.T + t0) * 2 * PAD;
        for (int e = tid; e < count * 2 * PAD; e += THREADS) {
            const float *const from = &s.part[0][0][0][0] + e;
            float v = 0.f;
#pragma unroll
            for (int w = 0; w < LANES; ++w) v += from[w * BLOCK * 2 * PAD];
            to[e] = v;
        }
        // (the next block's coefficients are read by the thread that writes them here, the rest after its first barrier)
    }

    if (LOCAL) {
        if (live && at_.first < at_.length) {
            const long long i = ((long long)b * a.segments + at_.segment) * a.s.C + at_.c0 + c;
            *reinterpret_cast<float4 *>(a.ends + i * PAD + n0) = float4_of(reordered(carry, order));
            if (quad == 0) a.steps[i] = step_sum;
        }
        return;
    }
    if (at_.segment == 0 && live && a.g.d_h0 != nullptr) store_quad(a.g.d_h0 + row * N, n0, N, reordered(carry, order));
    const long long i = ((long long)b * a.segments + at_.segment) * a.s.C + at_.c0;
    if (live) store_quad(a.part_a + (i + c) * N, n0, N, reordered(dA, order));
    // dD and d_dt_bias: the threads that share a channel
    const long long half = (long long)a.s.B * a.segments * a.s.C;
    if (PLANES) {  // neighbouring lanes
#pragma unroll
        for (int j = 0; j < OWN; ++j) {
            float v = dD[j].lo() + dD[j].hi(), w = d_bias[j].lo() + d_bias[j].hi();
#pragma unroll
            for (int m = Part::INNER / 2; m >= 1; m /= 2) v += __shfl_xor_sync(0xffffffffu, v, m), w += __shfl_xor_sync(0xffffffffu, w, m);
            const int pc = mine.channel(j);
            if (mine.busy() && mine.inner == 0 && pc < at_.channels) a.part_c[i + pc] = v, a.part_c[half + i + pc] = w;
        }
    } else {
        __syncthreads();
        float2 *const meet = reinterpret_cast<float2 *>(s.part);  // [2][THREADS]
        *reinterpret_cast<unsigned long long *>(meet + tid) = dD[0].q, *reinterpret_cast<unsigned long long *>(meet + THREADS + tid) = d_bias[0].q;
        __syncthreads();
        if (tid < at_.channels) {
            float v = 0.f, w = 0.f;
            for (int j = 0; j < THREADS / Part::INNER; ++j) {
                const float *const p = reinterpret_cast<const float *>(meet + j * Part::INNER) + tid;
                v += p[0], w += p[2 * THREADS];
            }
            a.part_c[i + tid] = v, a.part_c[half + i + tid] = w;
        }
    }
    // positions past the sequence's end
    for (int t0 = max(at_.first, at_.length); t0 < at_.end; t0 += BLOCK) {
        mine.clear(at<T, PLANES>(a.g.dx, b, t0, at_.c0), a.g.dx.row, at_.channels, at_.end - t0);
        mine.clear(at<T, PLANES>(a.g.d_dt, b, t0, at_.c0), a.g.d_dt.row, at_.channels, at_.end - t0);
        if (gated) mine.clear(at<T, PLANES>(a.g.dz, b, t0, at_.c0), a.g.dz.row, at_.channels, at_.end - t0);
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

template <typename T, int LANES, bool PLANES, bool WIDE> cudaError_t launch_selective_backward_as(const SelectiveArgs &a, cudaStream_t st) {
    const unsigned threads = kSelTile * LANES, grid = (unsigned)a.ctas() * a.segments;
    const size_t shared = sizeof(BackwardShared<LANES, PLANES>);
    const auto local = selective_backward_kernel<T, LANES, PLANES, WIDE, true>, whole = selective_backward_kernel<T, LANES, PLANES, WIDE, false>;
    cudaError_t e = cudaSuccess;
    if (a.segments > 1) {
        if ((e = allow_shared(local, shared)) != cudaSuccess) return e;
        if ((e = launch_kernel(local, grid, threads, shared, st, 1, a)) != cudaSuccess) return e;
    }
    if ((e = allow_shared(whole, shared)) != cudaSuccess) return e;
    if ((e = launch_kernel(whole, grid, threads, shared, st, 1, a)) != cudaSuccess) return e;
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
    return with_selective_shape(a, [&](auto lanes, auto planes, auto wide) {
        return launch_selective_backward_as<T, decltype(lanes)::value, decltype(planes)::value, decltype(wide)::value>(a, st);
    });
}

}  // namespace wtconv
