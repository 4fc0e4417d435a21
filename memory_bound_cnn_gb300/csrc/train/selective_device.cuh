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

// A position's decays of two states: exp2 of d times A log2 e.  The approximate exp2 of a value between -0.7 and 0 is low
// by 1.4e-8 of itself on average (measured over 2^20 of them); a state multiplies it up for as many positions as it
// remembers, a thousand and more, so the argument is raised by as much.  That is the average of steps that differ: a channel
// whose step is always the same has one argument, whose own error, up to two units, stays.
constexpr float kSelRaise = 2.0e-8f;  // log2(1 + 1.4e-8)
__device__ __forceinline__ Pair decays_of(Pair d, Pair rate) { return exp2_fast(fma(d, rate, Pair(kSelRaise))); }
__device__ __forceinline__ Pair decays_again(Pair d, Pair rate) { return exp2_again(fma(d, rate, Pair(kSelRaise))); }

// What a part of a sequence makes of the states h that enter it: exp2 of 4 q times h, and u.  The decay over a part may leave
// the range of fp32 where the product does not (and is 0 where h is), so it is multiplied up in four steps.  Bounded at
// 2^127, each of them is finite; four such take all but a 0 past the range, as the decay would.
__device__ __forceinline__ Pair through_part(Pair q, Pair h, Pair u) {
    const Pair f = exp2_fast(Pair(fminf(q.lo(), 127.f), fminf(q.hi(), 127.f)));
    return fma(mul(mul(mul(h, f), f), f), f, u);
}

// softplus(v) = max(v, 0) + log(1 + e) with e = exp(-|v|) in (0, 1]: nothing cancels.  With s = e / (2 + e)
// <= 1/3, log(1 + e) = 2 artanh s = 2 (s + s^3/3 + ... + s^13/13); the next term is 1.4e-8 of the value.
__device__ __forceinline__ Pair exp_of_minus_abs(Pair v) {
    return {exp2_fast(-kSelLog2E * fabsf(v.lo())), exp2_fast(-kSelLog2E * fabsf(v.hi()))};
}
__device__ __forceinline__ Pair reciprocal(Pair v) { return {reciprocal(v.lo()), reciprocal(v.hi())}; }
__device__ __forceinline__ Pair softplus_of(Pair v, Pair e) {
    const Pair s = mul(e, reciprocal(add(e, Pair(2.f)))), q = mul(s, s);
    Pair p = fma(Pair(1.f / 13), q, Pair(1.f / 11));
    p = fma(p, q, Pair(1.f / 9)), p = fma(p, q, Pair(1.f / 7)), p = fma(p, q, Pair(1.f / 5)), p = fma(p, q, Pair(1.f / 3));
    p = fma(p, q, Pair(1.f));
    return fma(add(s, s), p, Pair(fmaxf(v.lo(), 0.f), fmaxf(v.hi(), 0.f)));
}
__device__ __forceinline__ Pair softplus_of(Pair v) { return softplus_of(v, exp_of_minus_abs(v)); }
// Its slope sigmoid(v), from the same e.
__device__ __forceinline__ Pair softplus_slope(Pair v, Pair e) {
    const Pair r = reciprocal(add(e, Pair(1.f))), s = mul(e, r);
    return {v.lo() >= 0.f ? r.lo() : s.lo(), v.hi() >= 0.f ? r.hi() : s.hi()};
}
__device__ __forceinline__ Pair sigmoid_of(Pair v) {
    const Pair w = mul(v, Pair(-kSelLog2E));
    return reciprocal(add(exp2_fast(w), Pair(1.f)));
}

// Element (position, channel) of an activation.
template <typename T, bool PLANES>
__device__ __forceinline__ T *at(const wtconv_ssm_tensor &t, int b, int position, int channel) {
    const long long outer = PLANES ? channel : position, inner = PLANES ? position : channel;
    return static_cast<T *>(t.p) + b * t.batch + outer * t.row + inner;
}

// Sums v[0..COUNT) over COUNT lanes whose numbers differ by multiples of FIRST below COUNT * FIRST: they exchange
// halves, so that COUNT sums take COUNT - 1 exchanges.  A lane ends with the sum of v[i] in v[0], i its index
// among the COUNT lanes.
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

// A scanning lane's place in a CTA: of a warp's lanes `CHANNELS` neighbours have neighbouring channels, and WITHIN lanes
// with four states each share a channel (with 16 lanes to a channel, two warps have half of its states each).  Lanes
// that read the same 16 bytes of B or C are then neighbours: such a load takes two cycles of the shared memory,
// and four where they lie apart.
template <int LANES> struct LanePlace {
    static constexpr int WITHIN = LANES < 8 ? LANES : 8, HALVES = LANES / WITHIN, CHANNELS = 32 / WITHIN;
    int lane, warp, row, c, quad, n0;  // row: of the warps that have the same states
    __device__ __forceinline__ LanePlace() {
        lane = threadIdx.x % 32, warp = threadIdx.x / 32, row = warp / HALVES;
        c = row * CHANNELS + lane % CHANNELS, quad = warp % HALVES * WITHIN + lane / CHANNELS, n0 = 4 * quad;
    }
};

// Of a CTA's threads, the first 32 LANES scan; the others prepare the round after the scanned one and finish
// the one before.  All meet once a round.
template <int LANES> struct Roles {
    static constexpr int SCANNERS = kSelTile * LANES, HELPERS = 128, THREADS = SCANNERS + HELPERS;
    static __device__ __forceinline__ bool scans() { return threadIdx.x < SCANNERS; }
    static __device__ __forceinline__ int helper() { return threadIdx.x - SCANNERS; }
    // Registers of a thread, from what the CTA was launched with: scanners take what helpers give.  Whole groups of four
    // warps do so together; the sum over the CTA stays.  (8 x 4096 x 1024 with 16 states in bf16: 184 and 72 take 1143 us where
    // 176 and 80 take 1087 and 168 and 88 1100; in fp32, whose helpers hold wider words, 160 and 96 take 1227, 144 and 112 1136.)
    static constexpr bool TRADE = LANES >= 4;
    static constexpr int LAUNCHED = LANES == 4 ? 128 : LANES == 8 ? 168 : 96, GROUPS = SCANNERS / 128;
    template <typename T> static constexpr int GIVEN = LANES == 4 ? (sizeof(T) == 4 ? 16 : 48) : LANES == 8 ? 64 : 32;  // by a helper
    template <typename T> static __device__ __forceinline__ void take() {
        static_assert(!TRADE || (SCANNERS % 128 == 0 && GIVEN<T> % (8 * (TRADE ? GROUPS : 1)) == 0), "");
        if constexpr (TRADE) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(LAUNCHED + GIVEN<T> / GROUPS));
    }
    template <typename T> static __device__ __forceinline__ void give() {
        if constexpr (TRADE) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(LAUNCHED - GIVEN<T>));
    }
    static __device__ __forceinline__ void meet() { asm volatile("bar.sync 1, %0;" ::"n"(THREADS) : "memory"); }
    static __device__ __forceinline__ void helpers_meet() { asm volatile("bar.sync 2, %0;" ::"n"(HELPERS) : "memory"); }
};

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

// A helper's part of ROUND positions of WIDTH channels (or states): pairs of neighbours along the axis that is
// contiguous.  All of a round's loads are issued before the first is used (a load that waits behind a branch on
// another's value makes a round as long as all their latencies together).  WIDE: pairs lie at multiples of their size.
template <bool PLANES, int WIDTH, int ROUND, int THREADS, bool WIDE> struct Share {
    static constexpr int INNER = (PLANES ? ROUND : WIDTH) / 2, PAIRS = WIDTH * ROUND / 2;
    static constexpr int COUNT = PAIRS < THREADS ? 1 : PAIRS / THREADS, STEP = THREADS / INNER, OWN = PLANES ? COUNT : 1;
    static constexpr bool ALL = PAIRS >= THREADS;  // every thread has pairs
    static_assert(THREADS % INNER == 0 && (ALL ? PAIRS % THREADS == 0 : true), "");
    int inner, outer;  // of the first pair
    __device__ __forceinline__ explicit Share(int thread) : inner(thread % INNER * 2), outer(thread / INNER) {}
    __device__ __forceinline__ bool busy() const { return ALL || outer < (PLANES ? WIDTH : ROUND); }
    __device__ __forceinline__ int channel(int i) const { return PLANES ? outer + i * STEP : inner; }
    __device__ __forceinline__ int position(int i) const { return PLANES ? inner : outer + i * STEP; }
    // whether the pair's k-th element is one of `width` and `count`
    __device__ __forceinline__ bool in(int i, int k, int width, int count) const {
        return busy() && channel(i) + (PLANES ? 0 : k) < width && position(i) + (PLANES ? k : 0) < count;
    }
    // The thread's first pair of a round, from the round's first position and the first channel.  (A pointer that moves
    // along, kept from round to round: made anew, it is 20 instructions.)
    template <typename T> __device__ __forceinline__ T *mine(T *base, long long row) const { return base + outer * row + inner; }
    template <typename T>
    __device__ __forceinline__ void load(const T *p, long long row, int width, int count, typename Raw<T>::Two (&v)[COUNT]) const {
        const long long step = STEP * row;
        if (WIDE && ALL && width == WIDTH && count >= ROUND) {
#pragma unroll
            for (int i = 0; i < COUNT; ++i) v[i] = *reinterpret_cast<const typename Raw<T>::Two *>(p + i * step);
            return;
        }
#pragma unroll
        for (int i = 0; i < COUNT; ++i) {
            uint32_t first = 0, second = 0;
            if (in(i, 0, width, count)) first = load_one(p + i * step);
            if (in(i, 1, width, count)) second = load_one(p + i * step + 1);
            v[i] = two_of<T>(first, second);
        }
    }
    // value(i), a Pair, to its place
    template <typename T, typename F> __device__ __forceinline__ void store(T *p, long long row, int width, int count, F value) const {
        const long long step = STEP * row;
        if (WIDE && ALL && width == WIDTH && count >= ROUND) {
#pragma unroll
            for (int i = 0; i < COUNT; ++i) {
                const Pair v = value(i);
                Vec<T, 2> q;
                q.v[0] = from_f32<T>(v.lo()), q.v[1] = from_f32<T>(v.hi());
                *reinterpret_cast<Vec<T, 2> *>(p + i * step) = q;
            }
            return;
        }
#pragma unroll
        for (int i = 0; i < COUNT; ++i) {
            if (!in(i, 0, width, count)) continue;
            const Pair v = value(i);
            p[i * step] = from_f32<T>(v.lo());
            if (in(i, 1, width, count)) p[i * step + 1] = from_f32<T>(v.hi());
        }
    }
    // 0 to a round that may begin at an odd position: an element at a time
    template <typename T> __device__ __forceinline__ void clear(T *p, long long row, int width, int count) const {
#pragma unroll
        for (int i = 0; i < COUNT; ++i) {
            if (in(i, 0, width, count)) p[i * STEP * row] = from_f32<T>(0.f);
            if (in(i, 1, width, count)) p[i * STEP * row + 1] = from_f32<T>(0.f);
        }
    }
    // one fp32 parameter for each channel of the thread's pairs
    __device__ __forceinline__ void parameters(const float *of_tile, int width, Pair (&v)[OWN]) const {
#pragma unroll
        for (int i = 0; i < OWN; ++i) {
            const int c = channel(i);
            const float a = of_tile != nullptr && c < width ? of_tile[c] : 0.f;
            v[i] = Pair(a, PLANES ? a : of_tile != nullptr && c + 1 < width ? of_tile[c + 1] : 0.f);
        }
    }
};

// A tensor's place of a thread, round after round: `by` positions on with every step.
template <typename T, bool PLANES> struct Cursor {
    T *p;
    long long row;
    template <typename S> __device__ __forceinline__ Cursor(const S &share, const wtconv_ssm_tensor &t, int b, int position, int first) : row(t.row) {
        p = t.p == nullptr ? nullptr : share.mine(at<T, PLANES>(t, b, position, first), row);
    }
    __device__ __forceinline__ void step(int by) { p += PLANES ? by : by * row; }
};

// A round of the tile in shared memory has 32 channels to a position (tokens) or ROUND positions to a channel (planes),
// rows apart such that neither the helpers' pairs nor a warp's lanes, one channel apart, meet on a bank.
template <int LANES, bool PLANES, int ROUND> struct Layout {
    static constexpr int COEF = PLANES ? ROUND + 2 : kSelTile, COEFS = COEF * (PLANES ? kSelTile : ROUND);    // of two floats
    static constexpr int VALUE = PLANES ? ROUND + 4 : kSelTile, VALUES = VALUE * (PLANES ? kSelTile : ROUND);  // of one
    // Of a channel's lanes PARTS write their part of a sum (with 8 or 16 lanes, 2 or 4 of them meet by exchanges first).
    static constexpr int PARTS = LANES < 4 ? LANES : 4, TOGETHER = LANES / PARTS, APART = VALUES + (PLANES ? 2 : kSelTile / PARTS);
    // B and C: a row of the states to a position (planes: rows apart for the helpers, who write one state at a time)
    static constexpr int PAD = 4 * LANES, MAP = PLANES && LANES < 16 ? PAD + 4 : PAD;
    static __device__ __forceinline__ int coef(int t, int c) { return PLANES ? c * COEF + t : t * COEF + c; }
    static __device__ __forceinline__ int value(int t, int c) { return PLANES ? c * VALUE + t : t * VALUE + c; }
    // the lane's part of TOGETHER positions' sums from t on
    static __device__ __forceinline__ void put_sums(float *sums, int t, int c, int quad, float (&v)[TOGETHER]) {
        if (TOGETHER > 1) sum_exchange<TOGETHER, LanePlace<LANES>::CHANNELS>(v, quad % TOGETHER);
        sums[quad / TOGETHER * APART + value(t + quad % TOGETHER, c)] = v[0];
    }
    static __device__ __forceinline__ Pair get_sums(const float *sums, int place) {
        Pair s(*reinterpret_cast<const unsigned long long *>(sums + place));
#pragma unroll
        for (int i = 1; i < PARTS; ++i) s = add(s, Pair(*reinterpret_cast<const unsigned long long *>(sums + i * APART + place)));
        return s;
    }
    template <typename T, typename M> static __device__ __forceinline__ void put_map(const M &maps, typename Raw<T>::Two (&v)[M::COUNT], float *to) {
#pragma unroll
        for (int i = 0; i < M::COUNT; ++i) {
            if (!maps.busy()) continue;
            const Pair p = pair_of<T>(v[i]);
            float *const q = to + maps.position(i) * MAP + maps.channel(i);
            if (PLANES) q[0] = p.lo(), q[MAP] = p.hi();
            else *reinterpret_cast<unsigned long long *>(q) = p.q;
        }
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
// Rates of the lane's states; those past N have the last one's.  They hold 0 and pass on 0 whatever the step is: with a rate of
// 0 an infinite step, whose decay is 0, would be a NaN there, and flow back to all positions before it.
__device__ __forceinline__ Quad load_rates(const float *row, int n0, int N) {
    const int last = N - 1;
    return {Pair(row[min(n0, last)], row[min(n0 + 1, last)]), Pair(row[min(n0 + 2, last)], row[min(n0 + 3, last)])};
}
__device__ __forceinline__ void store_quad(float *row, int n0, int N, const Quad &q) {
    if (n0 < N) row[n0] = q.a.lo();
    if (n0 + 1 < N) row[n0 + 1] = q.a.hi();
    if (n0 + 2 < N) row[n0 + 2] = q.b.lo();
    if (n0 + 3 < N) row[n0 + 3] = q.b.hi();
}
__device__ __forceinline__ Quad quad_of(const float4 &v) { return {Pair(v.x, v.y), Pair(v.z, v.w)}; }
__device__ __forceinline__ float4 float4_of(const Quad &q) { return make_float4(q.a.lo(), q.a.hi(), q.b.lo(), q.b.hi()); }
}  // namespace wtconv
