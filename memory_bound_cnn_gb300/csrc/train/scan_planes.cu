// Gated scan of planes [B][C][T] (time contiguous).
//
// A lane owns 32 consecutive bytes of a row (16 or 8 positions), a warp 1024 (a span).  A stretch of the
// recurrence is the map h -> a h + u, and such maps compose (Span).  A lane takes its two halves as the
// two lanes of packed fp32 arithmetic (one instruction for both), joins their maps, and the warp scans
// the lanes' maps by shuffles; every lane then runs its positions again from the state that reaches it.
// The backward finds h again by the same scan over the few lanes between two kept states.  x, gate and
// (backward) dy are read once, through a ring of asynchronous copies that each warp keeps for itself
// (Cell): a queue in registers left the backward of 16-bit planes 72 registers too many.
//
// Rows of one span or less: several rows share a warp (scan_short_*).  Longer rows: the warps of a CTA
// take neighbouring spans of one row in rounds, exchange their maps through shared memory (one barrier
// a round) and carry the state in a register (scan_planes_*).  Few, long rows do not fill the GPU that
// way: they are cut into segments, a first kernel reduces each segment to its map, and the scan of a
// segment starts from the maps before it (after it, backward).  That reads two of the inputs twice, the
// second time mostly from L2.
//
// Bound by HBM, closely followed by the issue of instructions (25 an element forward, 35 backward, at
// 67 % and 53 % of the issue slots).  Alone, with cold caches: 16x64x65536 bf16 forward 75 us (5.3 TB/s,
// 80 % of a copy), backward 129 us (5.2 TB/s, 78 %); 64x96x3136 fp32 49 us (70 %) and 74 us (78 %).
// With eight positions a lane the shuffles and the exchange weighed twice as much (83 and 146 us).
#include "scan_device.cuh"

namespace wtconv {

namespace {

constexpr int kMaxWarps = 4;
template <typename T> constexpr int kLane = 32 / (int)sizeof(T);                // positions of a lane,
template <typename T> constexpr int kHalf = kLane<T> / 2;                       // of its halves,
template <typename T> constexpr int kWarpSpan = 32 * kLane<T>;                  // of a warp's round
template <typename T> constexpr int kKeepLanes = WTCONV_SCAN_KEEP / kLane<T>;   // lanes between two kept states

enum Mode { kReduce, kApply };

// A lane's positions as raw words; pair j holds positions j and kHalf<T> + j.
template <typename T> struct Strip {
    static constexpr int words = kLane<T> * (int)sizeof(T) / 4;
    uint32_t w[words];
    __device__ __forceinline__ Pair get(int j) const {
        if constexpr (sizeof(T) == 4) return {__uint_as_float(w[j]), __uint_as_float(w[kHalf<T> + j])};
        else {
            const Pair a = widen<T>(w[j >> 1]), b = widen<T>(w[(kHalf<T> + j) >> 1]);
            return j & 1 ? Pair(a.hi(), b.hi()) : Pair(a.lo(), b.lo());
        }
    }
    __device__ __forceinline__ void set(const Pair (&v)[kHalf<T>]) {
#pragma unroll
        for (int j = 0; j < kHalf<T>; j += 2) {
            if constexpr (sizeof(T) == 4) {
                w[j] = __float_as_uint(v[j].lo()), w[j + 1] = __float_as_uint(v[j + 1].lo());
                w[kHalf<T> + j] = __float_as_uint(v[j].hi()), w[kHalf<T> + j + 1] = __float_as_uint(v[j + 1].hi());
            } else {
                w[j >> 1] = narrow<T>(Pair(v[j].lo(), v[j + 1].lo()));
                w[(kHalf<T> + j) >> 1] = narrow<T>(Pair(v[j].hi(), v[j + 1].hi()));
            }
        }
    }
    // Straight from and to memory (short rows): positions 0 .. valid-1, as vectors where CP is 16.
    template <int CP> __device__ __forceinline__ void load(const T *p, int valid) {
        if (CP == 16 && valid >= kLane<T>) {
#pragma unroll
            for (int k = 0; k < words; k += 4) {
                const uint4 v = __ldg(reinterpret_cast<const uint4 *>(p) + k / 4);
                w[k] = v.x, w[k + 1] = v.y, w[k + 2] = v.z, w[k + 3] = v.w;
            }
            return;
        }
#pragma unroll
        for (int k = 0; k < words; ++k) w[k] = 0;
#pragma unroll
        for (int j = 0; j < kLane<T>; ++j) {
            if (j >= valid) continue;
            if constexpr (sizeof(T) == 4) w[j] = __float_as_uint(p[j]);
            else w[j >> 1] |= (uint32_t)*reinterpret_cast<const uint16_t *>(p + j) << (16 * (j & 1));
        }
    }
    template <int CP> __device__ __forceinline__ void store(T *p, int valid) const {
        if (CP == 16 && valid >= kLane<T>) {
#pragma unroll
            for (int k = 0; k < words; k += 4)
                reinterpret_cast<uint4 *>(p)[k / 4] = make_uint4(w[k], w[k + 1], w[k + 2], w[k + 3]);
            return;
        }
#pragma unroll
        for (int j = 0; j < kLane<T>; ++j) {
            if (j >= valid) continue;
            if constexpr (sizeof(T) == 4) p[j] = __uint_as_float(w[j]);
            else *reinterpret_cast<uint16_t *>(p + j) = (uint16_t)(w[j >> 1] >> (16 * (j & 1)));
        }
    }
    // zeros from position `valid` on
    __device__ __forceinline__ void cut(int valid) {
#pragma unroll
        for (int j = 0; j < kLane<T>; ++j) {
            if (j < valid) continue;
            if constexpr (sizeof(T) == 4) w[j] = 0;
            else w[j >> 1] &= j & 1 ? 0x0000ffffu : 0xffff0000u;
        }
    }
};

// A warp's span of one tensor in shared memory, which the warp itself brings in and reads: a queue that
// takes no registers and no barrier of the CTA.  It moves in order, CP bytes a lane at a time, so that a
// warp's copies lie side by side; a lane then reads its own positions.  CP 2: rows that start at any
// 16-bit element are copied by whole words, from the one that holds the span's first position on, and
// lie one element further (`shift`) where that is not a multiple of 4.
template <typename T> struct Cell {
    static constexpr int bytes = kWarpSpan<T> * (int)sizeof(T);
    uint4 q[bytes / 16 + 1];
    __device__ __forceinline__ char *at(int offset) { return reinterpret_cast<char *>(q) + offset; }
    // The span from p (the warp's first position) on.  Positions from `valid` on are not read and come
    // as zeros; base is the tensor's first element, an address that stands in where nothing is read.
    template <int CP> __device__ __forceinline__ void fetch(const T *p, int valid, int lane, const void *base) {
        if constexpr (CP == 2) {
            const int shift = (int)(reinterpret_cast<uintptr_t>(p) >> 1 & 1);
            const void *anchor = reinterpret_cast<const void *>(reinterpret_cast<uintptr_t>(base) + 2 & ~(uintptr_t)3);
#pragma unroll
            for (int k = 0; k <= bytes / 128; ++k) {
                if (k == bytes / 128 && lane > 0) continue;  // one word more
                const int t = (k * 32 + lane) * 2 - shift;   // the word's first position
                const T *from = p + t;
                const int left = min(max(valid - t, 0), 2) * 2;
                if (t < 0 && from < base) {  // before the tensor: its first element alone
                    const uint16_t v = valid > 0 ? *reinterpret_cast<const uint16_t *>(from + 1) : (uint16_t)0;
                    *reinterpret_cast<uint32_t *>(at(0)) = (uint32_t)v << 16;
                } else {
                    copy_async<4>(at((k * 32 + lane) * 4), left > 0 ? static_cast<const void *>(from) : anchor, left);
                }
            }
            return;
        } else {
            const char *from = reinterpret_cast<const char *>(p) + lane * CP;
            if (valid >= kWarpSpan<T>) {
#pragma unroll
                for (int k = 0; k < bytes / (32 * CP); ++k) copy_async<CP>(at((k * 32 + lane) * CP), from + k * 32 * CP, CP);
            } else {
                const int have = max(valid, 0) * (int)sizeof(T);  // (valid may be as low as -2^30)
#pragma unroll
                for (int k = 0; k < bytes / (32 * CP); ++k) {
                    const int left = min(max(have - (k * 32 + lane) * CP, 0), CP);
                    copy_async<CP>(at((k * 32 + lane) * CP), left > 0 ? from + k * 32 * CP : base, left);
                }
            }
        }
    }
    // shift: of the span that was fetched (0 unless CP is 2)
    template <int CP> __device__ __forceinline__ Strip<T> read(int lane, int shift) const {
        Strip<T> s;
#pragma unroll
        for (int k = 0; k < Strip<T>::words / 4; ++k) {
            const uint4 v = q[lane * (Strip<T>::words / 4) + k];
            s.w[4 * k] = v.x, s.w[4 * k + 1] = v.y, s.w[4 * k + 2] = v.z, s.w[4 * k + 3] = v.w;
        }
        if constexpr (CP == 2) {
            const uint32_t last = q[(lane + 1) * (Strip<T>::words / 4)].x;
#pragma unroll
            for (int k = 0; k < Strip<T>::words; ++k)
                s.w[k] = __funnelshift_r(s.w[k], k + 1 < Strip<T>::words ? s.w[k + 1] : last, 16 * shift);
        }
        return s;
    }
    // The lanes' positions to p (the warp's first position), those before `valid`: straight from the
    // registers, or through this cell where single elements or words would lie far apart.
    template <int CP> __device__ __forceinline__ void store(T *p, const Strip<T> &s, int valid, int lane) {
        if (CP == 16 && valid >= kWarpSpan<T>) {
#pragma unroll
            for (int k = 0; k < Strip<T>::words; k += 4)
                reinterpret_cast<uint4 *>(p + lane * kLane<T>)[k / 4] = make_uint4(s.w[k], s.w[k + 1], s.w[k + 2], s.w[k + 3]);
            return;
        }
        __syncwarp();
#pragma unroll
        for (int k = 0; k < Strip<T>::words / 4; ++k)
            q[lane * (Strip<T>::words / 4) + k] = make_uint4(s.w[4 * k], s.w[4 * k + 1], s.w[4 * k + 2], s.w[4 * k + 3]);
        __syncwarp();
        char *to = reinterpret_cast<char *>(p);
        if (CP >= 4 && valid >= kWarpSpan<T>) {
#pragma unroll
            for (int k = 0; k < bytes / 128; ++k)
                *reinterpret_cast<uint32_t *>(to + (k * 32 + lane) * 4) = *reinterpret_cast<const uint32_t *>(at((k * 32 + lane) * 4));
        } else {
            constexpr int e = (int)sizeof(T);
#pragma unroll
            for (int k = 0; k < kLane<T>; ++k)
                if (k * 32 + lane < valid) *reinterpret_cast<T *>(to + (k * 32 + lane) * e) = *reinterpret_cast<const T *>(at((k * 32 + lane) * e));
        }
        __syncwarp();
    }
};
constexpr int kStages = 2;

// A lane's two halves as maps (Span of positions in time order: lo then hi).
struct Halves {
    Pair a, u;
    __device__ __forceinline__ Span lo() const { return {a.lo(), u.lo()}; }
    __device__ __forceinline__ Span hi() const { return {a.hi(), u.hi()}; }
};

// Gates of a lane's positions; those at or past `live` hold the state (a = 1, b = 0).
template <typename T>
__device__ __forceinline__ void lane_gates(const Strip<T> &g, Pair bias, int live, Pair (&av)[kHalf<T>], Pair (&bv)[kHalf<T>]) {
#pragma unroll
    for (int j = 0; j < kHalf<T>; ++j) {
        const Gates q = gates_of(g.get(j), bias);
        av[j] = q.a, bv[j] = q.b;
    }
    if (live < kLane<T>) {
#pragma unroll
        for (int j = 0; j < kHalf<T>; ++j) {
            if (j >= live) av[j] = Pair(1.f, av[j].hi()), bv[j] = Pair(0.f, bv[j].hi());
            if (kHalf<T> + j >= live) av[j] = Pair(av[j].lo(), 1.f), bv[j] = Pair(bv[j].lo(), 0.f);
        }
    }
}

// The forward of a lane: its map, then its outputs from the state before it.
template <typename T> struct LaneForward {
    Pair av[kHalf<T>], uv[kHalf<T>];
    Halves halves;
    __device__ __forceinline__ Span reduce(const Strip<T> &x, const Strip<T> &g, Pair bias, int live) {
        lane_gates(g, bias, live, av, uv);
        halves = {Pair(1.f), Pair(0.f)};
#pragma unroll
        for (int j = 0; j < kHalf<T>; ++j) {
            uv[j] = mul(uv[j], x.get(j));  // (x is 0 beyond the length)
            halves.u = fma(av[j], halves.u, uv[j]);
            halves.a = mul(halves.a, av[j]);
        }
        return halves.lo().then(halves.hi());
    }
    __device__ __forceinline__ Strip<T> outputs(float before, int live) {
        Pair h(before, halves.lo().of(before)), out[kHalf<T>];
#pragma unroll
        for (int j = 0; j < kHalf<T>; ++j) out[j] = h = fma(av[j], h, uv[j]);
        Strip<T> y;
        y.set(out);
        if (live < kLane<T>) y.cut(live);  // past the length the state stands still, and y is 0
        return y;
    }
};

// The backward of a lane: the maps of dh (backward) and of h (forward), then its gradients.  x and dy
// are taken from their cells again rather than kept.
template <typename T> struct LaneBackward {
    Pair av[kHalf<T>], bv[kHalf<T>];
    Halves back, fwd;
    __device__ __forceinline__ Span reduce(const Strip<T> &g, const Strip<T> &dy, Pair bias, int live) {
        lane_gates(g, bias, live, av, bv);
        back = {Pair(1.f), Pair(0.f)};
#pragma unroll
        for (int j = kHalf<T> - 1; j >= 0; --j) {
            back.u = mul(av[j], add(dy.get(j), back.u));
            back.a = mul(back.a, av[j]);
        }
        return back.hi().then(back.lo());
    }
    __device__ __forceinline__ Span reduce_h(const Strip<T> &x) {
        fwd = {back.a, Pair(0.f)};
#pragma unroll
        for (int j = 0; j < kHalf<T>; ++j) fwd.u = fma(av[j], fwd.u, mul(bv[j], x.get(j)));
        return fwd.lo().then(fwd.hi());
    }
    // h: the state before the lane; flow: a dh of the position after it
    __device__ __forceinline__ void gradients(float h_before, float flow_after, const Strip<T> &x, const Strip<T> &dy, int live,
                                              Strip<T> &dx, Strip<T> &dg, Pair &sum) {
        Pair h(h_before, fwd.lo().of(h_before)), diff[kHalf<T>];
#pragma unroll
        for (int j = 0; j < kHalf<T>; ++j) {
            const Pair xv = x.get(j);
            diff[j] = sub(h, xv);  // h_{t-1} - x_t
            h = fma(av[j], h, mul(bv[j], xv));
        }
        Pair flow(back.hi().of(flow_after), flow_after);
        const Pair before = sum;
#pragma unroll
        for (int j = kHalf<T> - 1; j >= 0; --j) {
            const Pair dh = add(dy.get(j), flow);
            diff[j] = mul(mul(dh, diff[j]), mul(av[j], bv[j]));
            sum = add(sum, diff[j]);
            bv[j] = mul(bv[j], dh);
            flow = mul(av[j], dh);
        }
        dx.set(bv);
        dg.set(diff);
        if (live < kLane<T>) {
            // Nothing past the length: 1 - a is 0 there, but a state or dh that is not finite makes its
            // products NaN.  (Apart from the loop, and the sum formed again: with every lane's sum after the
            // loop 16x64x65536 bf16 forward + backward took 209 us, with selections in it 200, so 193.)
            dx.cut(live), dg.cut(live);
            sum = before;
#pragma unroll
            for (int j = kHalf<T> - 1; j >= 0; --j)
                sum = add(sum, Pair(j < live ? diff[j].lo() : 0.f, kHalf<T> + j < live ? diff[j].hi() : 0.f));
        }
    }
};

// ------------------------------------------------------------------------- rows of several spans

// Map of the segments [first, last) of a row in the scan's order, by all lanes of a warp alike.
__device__ __forceinline__ Span fold_segments(const float2 *maps, int first, int last, bool backward, int lane) {
    const int count = last - first, per = (count + 31) / 32;
    Span s = {1.f, 0.f};
    for (int k = 0; k < per; ++k) {
        const int i = lane * per + k;
        if (i < count) {
            const float2 m = maps[backward ? last - 1 - i : first + i];
            s = s.then({m.x, m.y});
        }
    }
    s = warp_scan<false>(s, 32);
    s.a = __shfl_sync(0xffffffffu, s.a, 31);
    s.u = __shfl_sync(0xffffffffu, s.u, 31);
    return s;
}

// One round's exchange between the CTA's warps.  mine: the warp's whole map in lane `from`.  Returns
// the state before this warp's span and moves carry past the round.
template <bool BACKWARD>
__device__ __forceinline__ float exchange(Span mine, float2 *slots, int warp, int warps, int lane, float &carry) {
    constexpr int from = BACKWARD ? 0 : 31;
    if (warps == 1) {
        const float before = carry;
        const Span whole = {__shfl_sync(0xffffffffu, mine.a, from), __shfl_sync(0xffffffffu, mine.u, from)};
        carry = whole.of(carry);
        return before;
    }
    if (lane == from) slots[warp] = make_float2(mine.a, mine.u);
    __syncthreads();
    float before = 0.f;
    for (int i = 0; i < warps; ++i) {
        const int w = BACKWARD ? warps - 1 - i : i;
        if (w == warp) before = carry;
        const float2 m = slots[w];
        carry = fmaf(m.x, carry, m.y);
    }
    return before;
}

struct Segment {
    int b, c, seg, n;    // n: length of the sequence
    long long row;       // b * C + c
    int round0, round1;  // rounds of this segment
};
__device__ __forceinline__ Segment segment_of(const ScanArgs &a, int segments, int rounds_per, int round_span) {
    Segment s;
    s.row = blockIdx.x / segments;
    s.seg = (int)(blockIdx.x - s.row * segments);
    s.b = (int)(s.row / a.C);
    s.c = (int)(s.row - (long long)s.b * a.C);
    s.n = scan_length(a.lengths, s.b, a.T);
    const int rounds = (a.T + round_span - 1) / round_span;
    s.round0 = s.seg * rounds_per;
    s.round1 = min(s.round0 + rounds_per, rounds);
    return s;
}
// Elements that a span from p on lies further in its cell (CP 2).
template <int CP, typename T> __device__ __forceinline__ int shift_of(const T *p) {
    return CP == 2 ? (int)(reinterpret_cast<uintptr_t>(p) >> 1 & 1) : 0;
}
template <typename T> __device__ __forceinline__ T *row_of(const ScanTensor &t, int b, int c) {
    return static_cast<T *>(t.p) + b * t.batch + c * t.row;
}

// Shared memory of a kernel: kStages cells of each of TENSORS per warp.
template <typename T, int TENSORS> using Ring = Cell<T>[kStages][TENSORS];
template <typename T, int TENSORS> __device__ __forceinline__ Ring<T, TENSORS> &ring_of(unsigned char *raw, int warp) {
    return reinterpret_cast<Ring<T, TENSORS> *>(raw)[warp];
}
static_assert(kMaxWarps * sizeof(Ring<float, 3>) <= 40 * 1024 && kMaxWarps * sizeof(Ring<__half, 3>) <= 40 * 1024,
              "with its static part a CTA stays within the 48 KB that need no permission");
__device__ __forceinline__ int next_stage(int s) { return s + 1 == kStages ? 0 : s + 1; }

// 72 registers leave room for 28 warps an SM (forward_warps).  Forward, cold caches: 16x64x65536 bf16 74 us,
// 64x96x3136 fp32 48, 4x300x40000 fp16 68, 2x400x100000 fp32 167.  Capped at 64, for 32 warps: 76, 50, 59 and
// 167; at 80, for 24: 93, 52, 68 and 165.
template <typename T, int CP, Mode MODE>
__global__ void __maxnreg__(72) scan_planes_forward_kernel(const ScanArgs a, int segments, int rounds_per, float2 *maps) {
    extern __shared__ __align__(16) unsigned char raw[];
    __shared__ float2 slots[2][kMaxWarps];
    begin_kernel();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const int round_span = warps * kWarpSpan<T>;
    const Segment s = segment_of(a, segments, rounds_per, round_span);
    auto &ring = ring_of<T, 2>(raw, warp);
    int t0 = s.round0 * round_span + warp * kWarpSpan<T>;  // the warp's first position
    const T *x = row_of<T>(a.x, s.b, s.c) + t0, *g = row_of<T>(a.gate, s.b, s.c) + t0;
    T *y = row_of<T>(a.y, s.b, s.c) + t0;
    const int shift_x = shift_of<CP>(x), shift_g = shift_of<CP>(g);  // (a span is an even number of positions)
    int ahead = s.n - t0;  // valid positions of the next cells
    const auto fetch = [&](int stage) {
        ring[stage][0].template fetch<CP>(x, ahead, lane, a.x.p);
        ring[stage][1].template fetch<CP>(g, ahead, lane, a.gate.p);
        commit_copies();
        x += round_span, g += round_span, ahead -= round_span;
    };
    int left = s.round1 - s.round0;  // rounds that are not fetched yet
#pragma unroll
    for (int k = 0; k < kStages - 1; ++k) {
        if (left > 0) fetch(k), --left;
        else commit_copies();
    }
    const Pair bias(a.gate_bias[s.c]);

    float carry = 0.f;
    Span whole = {1.f, 0.f};  // kReduce: the segment so far
    if (MODE == kApply) {
        carry = a.h0 != nullptr ? a.h0[s.row] : 0.f;
        if (s.seg > 0) carry = fold_segments(maps + s.row * segments, 0, s.seg, false, lane).of(carry);
    }
    int stage = 0, free_stage = kStages - 1;
    for (int round = s.round0; round < s.round1; ++round, t0 += round_span) {
        wait_copies<kStages - 2>();
        __syncwarp();
        LaneForward<T> f;
        const int t = t0 + lane * kLane<T>, live = s.n - t;
        Span span = {1.f, 0.f};
        if (t0 < a.T) span = f.reduce(ring[stage][0].template read<CP>(lane, shift_x), ring[stage][1].template read<CP>(lane, shift_g), bias, live);
        if (left > 0) fetch(free_stage), --left;
        else commit_copies();
        Cell<T> &out = ring[stage][0];  // read already
        stage = next_stage(stage), free_stage = next_stage(free_stage);
        if (t0 < a.T) span = warp_scan<false>(span, 32);
        float2 *slot = slots[round & 1];
        if (MODE == kReduce) {
            // every warp folds the whole round, so that all end with the segment's map
            if (lane == 31) slot[warp] = make_float2(span.a, span.u);
            __syncthreads();
            for (int w = 0; w < warps; ++w) whole = whole.then({slot[w].x, slot[w].y});
            continue;
        }
        const Span before = lane_before<false>(span, 32);
        const float h = before.of(exchange<false>(span, slot, warp, warps, lane, carry));
        if (t0 >= a.T) break;  // the row's last round, and nothing of it for this warp
        if (a.states_out != nullptr && (lane & (kKeepLanes<T> - 1)) == 0 && t < a.T)
            a.states_out[s.row * a.keep + t / WTCONV_SCAN_KEEP] = h;
        out.template store<CP>(y, f.outputs(h, live), a.T - t0, lane);
        y += round_span;
    }
    if (MODE == kReduce) {
        if (threadIdx.x == 0) maps[blockIdx.x] = make_float2(whole.a, whole.u);
    } else if (a.h_last != nullptr && s.seg == segments - 1 && threadIdx.x == 0) {
        a.h_last[s.row] = carry;
    }
}

template <typename T, int CP, Mode MODE>
__global__ void __launch_bounds__(kMaxWarps * 32, sizeof(T) == 4 ? 6 : 4)
    scan_planes_backward_kernel(const ScanArgs a, int segments, int rounds_per, float2 *maps, float *bias_part) {
    extern __shared__ __align__(16) unsigned char raw[];
    __shared__ float2 slots[2][kMaxWarps];
    __shared__ float sums[kMaxWarps];
    begin_kernel();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const int round_span = warps * kWarpSpan<T>;
    const Segment s = segment_of(a, segments, rounds_per, round_span);
    auto &ring = ring_of<T, 3>(raw, warp);
    int t0 = (s.round1 - 1) * round_span + warp * kWarpSpan<T>;  // the warp's first position
    const T *x = row_of<T>(a.x, s.b, s.c) + t0, *g = row_of<T>(a.gate, s.b, s.c) + t0, *dy = row_of<T>(a.dy, s.b, s.c) + t0;
    T *dx = row_of<T>(a.dx, s.b, s.c) + t0, *dg = row_of<T>(a.d_gate, s.b, s.c) + t0;
    const int shift_x = shift_of<CP>(x), shift_g = shift_of<CP>(g), shift_dy = shift_of<CP>(dy);
    int ahead = s.n - t0;  // valid positions of the next cells
    const auto fetch = [&](int stage) {
        ring[stage][0].template fetch<CP>(g, ahead, lane, a.gate.p);
        ring[stage][1].template fetch<CP>(dy, ahead, lane, a.dy.p);
        if (MODE == kApply) ring[stage][2].template fetch<CP>(x, ahead, lane, a.x.p);
        commit_copies();
        x -= round_span, g -= round_span, dy -= round_span, ahead += round_span;
    };
    int left = s.round1 - s.round0;  // rounds that are not fetched yet
#pragma unroll
    for (int k = 0; k < kStages - 1; ++k) {
        if (left > 0) fetch(k), --left;
        else commit_copies();
    }
    const auto kept_at = [&](int at) {
        return MODE == kApply && at < a.T ? a.states_in[s.row * a.keep + at / WTCONV_SCAN_KEEP] : 0.f;
    };
    float next_kept = kept_at(t0 + lane * kLane<T>);
    const Pair bias(a.gate_bias[s.c]);

    float carry = 0.f;  // a dh of the position after the round
    Pair sum(0.f);
    Span whole = {1.f, 0.f};
    if (MODE == kApply) {
        carry = a.dh_last != nullptr ? a.dh_last[s.row] : 0.f;
        if (s.seg < segments - 1)
            carry = fold_segments(maps + s.row * segments, s.seg + 1, segments, true, lane).of(carry);
    }
    int stage = 0, free_stage = kStages - 1;
    for (int round = s.round1 - 1; round >= s.round0; --round, t0 -= round_span) {
        wait_copies<kStages - 2>();
        __syncwarp();
        LaneBackward<T> f;
        const float kept = next_kept;
        const int t = t0 + lane * kLane<T>, live = s.n - t;
        Span span = {1.f, 0.f};
        if (t0 < a.T) span = f.reduce(ring[stage][0].template read<CP>(lane, shift_g), ring[stage][1].template read<CP>(lane, shift_dy), bias, live);
        if (left > 0) fetch(free_stage), --left;
        else commit_copies();
        if (round > s.round0) next_kept = kept_at(t - round_span);
        if (t0 < a.T) span = warp_scan<true>(span, 32);
        float2 *slot = slots[round & 1];
        if (MODE == kReduce) {
            stage = next_stage(stage), free_stage = next_stage(free_stage);
            if (lane == 0) slot[warp] = make_float2(span.a, span.u);
            __syncthreads();
            for (int w = warps - 1; w >= 0; --w) whole = whole.then({slot[w].x, slot[w].y});
            continue;
        }
        if (t0 >= a.T) {  // the row's last round, and nothing of it for this warp
            exchange<true>(span, slot, warp, warps, lane, carry);
            stage = next_stage(stage), free_stage = next_stage(free_stage);
            dx -= round_span, dg -= round_span;
            continue;
        }
        const Span fwd = warp_scan<false>(f.reduce_h(ring[stage][2].template read<CP>(lane, shift_x)), kKeepLanes<T>);
        const float h = lane_before<false>(fwd, kKeepLanes<T>).of(kept);
        const Span after = lane_before<true>(span, 32);
        const float flow = after.of(exchange<true>(span, slot, warp, warps, lane, carry));
        Strip<T> odx, odg;
        f.gradients(h, flow, ring[stage][2].template read<CP>(lane, shift_x), ring[stage][1].template read<CP>(lane, shift_dy), live, odx, odg,
                    sum);
        ring[stage][0].template store<CP>(dx, odx, a.T - t0, lane);
        ring[stage][0].template store<CP>(dg, odg, a.T - t0, lane);
        stage = next_stage(stage), free_stage = next_stage(free_stage);
        dx -= round_span, dg -= round_span;
    }
    if (MODE == kReduce) {
        if (threadIdx.x == 0) maps[blockIdx.x] = make_float2(whole.a, whole.u);
        return;
    }
    float total = warp_sum(sum.lo() + sum.hi());
    if (lane == 0) sums[warp] = total;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int w = 1; w < warps; ++w) total += sums[w];
        bias_part[blockIdx.x] = total;
        if (a.d_h0 != nullptr && s.seg == 0) a.d_h0[s.row] = carry;
    }
}

// --------------------------------------------------------------------- rows of one span or less

constexpr int kShortThreads = 128;

struct ShortRow {
    int b, c, n, t, group;  // t: the lane's first position; group: its place among the row's lanes
    long long row;          // past the last row: no position is live or stored
    bool any;
};
template <typename T> __device__ __forceinline__ ShortRow short_row(const ScanArgs &a, int lanes) {
    ShortRow s;
    const unsigned per_cta = kShortThreads / lanes;
    s.group = threadIdx.x & (lanes - 1);
    s.row = (long long)blockIdx.x * per_cta + threadIdx.x / lanes;
    s.any = s.row < (long long)a.B * a.C;
    if (!s.any) s.row = 0;
    s.b = (int)(s.row / a.C);
    s.c = (int)(s.row - (long long)s.b * a.C);
    s.n = s.any ? scan_length(a.lengths, s.b, a.T) : 0;
    s.t = s.group * kLane<T>;
    return s;
}

template <typename T, int CP> __global__ void __launch_bounds__(kShortThreads) scan_short_forward_kernel(const ScanArgs a, int lanes) {
    begin_kernel();
    const ShortRow s = short_row<T>(a, lanes);
    Strip<T> x, g;
    x.template load<CP>(row_of<T>(a.x, s.b, s.c) + s.t, s.n - s.t);
    g.template load<CP>(row_of<T>(a.gate, s.b, s.c) + s.t, s.n - s.t);
    const Pair bias(a.gate_bias[s.c]);
    const float h0 = a.h0 != nullptr ? a.h0[s.row] : 0.f;
    LaneForward<T> f;
    const Span span = warp_scan<false>(f.reduce(x, g, bias, s.n - s.t), lanes);
    const float h = lane_before<false>(span, lanes).of(h0);
    if (!s.any) return;
    if (a.states_out != nullptr && s.t % WTCONV_SCAN_KEEP == 0 && s.t < a.T)
        a.states_out[s.row * a.keep + s.t / WTCONV_SCAN_KEEP] = h;
    f.outputs(h, s.n - s.t).template store<CP>(row_of<T>(a.y, s.b, s.c) + s.t, a.T - s.t);
    if (a.h_last != nullptr && s.group == lanes - 1) a.h_last[s.row] = span.of(h0);
}

template <typename T, int CP>
__global__ void __launch_bounds__(kShortThreads) scan_short_backward_kernel(const ScanArgs a, int lanes, float *bias_part) {
    begin_kernel();
    const ShortRow s = short_row<T>(a, lanes);
    Strip<T> x, g, dy;
    x.template load<CP>(row_of<T>(a.x, s.b, s.c) + s.t, s.n - s.t);
    g.template load<CP>(row_of<T>(a.gate, s.b, s.c) + s.t, s.n - s.t);
    dy.template load<CP>(row_of<T>(a.dy, s.b, s.c) + s.t, s.n - s.t);
    const Pair bias(a.gate_bias[s.c]);
    const float dh_last = a.dh_last != nullptr ? a.dh_last[s.row] : 0.f;
    const float kept = a.states_in[s.row * a.keep];  // the state before the row
    LaneBackward<T> f;
    const Span back = warp_scan<true>(f.reduce(g, dy, bias, s.n - s.t), lanes);
    const Span fwd = warp_scan<false>(f.reduce_h(x), lanes);
    const float h = lane_before<false>(fwd, lanes).of(kept);
    const float flow = lane_before<true>(back, lanes).of(dh_last);
    Strip<T> dx, dg;
    Pair sum(0.f);
    f.gradients(h, flow, x, dy, s.n - s.t, dx, dg, sum);
    float total = sum.lo() + sum.hi();
    for (int d = lanes >> 1; d > 0; d >>= 1) total += __shfl_xor_sync(0xffffffffu, total, d);
    if (!s.any) return;
    dx.template store<CP>(row_of<T>(a.dx, s.b, s.c) + s.t, a.T - s.t);
    dg.template store<CP>(row_of<T>(a.d_gate, s.b, s.c) + s.t, a.T - s.t);
    if (s.group == 0) {
        bias_part[s.row] = total;
        if (a.d_h0 != nullptr) a.d_h0[s.row] = back.of(dh_last);
    }
}

// d_gate_bias_c = sum over sequences and segments of the parts, in a fixed order: one warp per channel.
__global__ void __launch_bounds__(128) scan_planes_bias_kernel(const float *part, float *out, int B, int C, int segments) {
    begin_kernel();
    const int c = blockIdx.x * 4 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    if (c >= C) return;
    float sum = 0.f;
    const int count = B * segments;
    for (int i = lane; i < count; i += 32) {
        const int b = i / segments;
        sum += part[((long long)b * C + c) * segments + (i - b * segments)];
    }
    sum = warp_sum(sum);
    if (lane == 0) out[c] = sum;
}

// ------------------------------------------------------------------------------------------- host

// How rows are cut.  lanes > 0: one span or less, that many lanes a row.  Else CTAs of `warps` warps,
// as many as a row has spans for and as leave every row resident at once (`per_sm` warps fit an SM, a
// multiple of kMaxWarps); where rows exceed that anyway, four.  segments > 1 only where rows leave half
// the GPU idle.
struct Plan {
    int lanes, warps, segments, rounds_per;
};
Plan plan_of(const ScanArgs &a, int per_sm) {
    Plan p = {0, 1, 1, 1};
    const long long rows = (long long)a.B * a.C;
    const int lane = 32 / elem_bytes_of(a.dtype), span = 32 * lane, sms = sm_count();
    if (a.T <= span) {
        for (p.lanes = 1; p.lanes * lane < a.T;) p.lanes *= 2;
        return p;
    }
    const int spans = (a.T + span - 1) / span;
    const long long fit = (long long)per_sm * sms;
    p.warps = rows > fit ? 4 : 1;
    while (p.warps < kMaxWarps && rows * p.warps * 2 <= fit) p.warps *= 2;
    while (p.warps > 1 && p.warps / 2 >= spans) p.warps /= 2;
    // (fewer warps where that wastes less of the last round)
    for (int w = p.warps / 2; w > 1; w /= 2)
        if ((spans + w - 1) / w * w < (spans + p.warps - 1) / p.warps * p.warps) p.warps = w;
    const int rounds = (spans + p.warps - 1) / p.warps;
    if (rows * p.warps * 2 < fit) p.segments = (int)(fit / (rows * p.warps));
    if (p.segments > rounds) p.segments = rounds;
    p.rounds_per = (rounds + p.segments - 1) / p.segments;
    p.segments = (rounds + p.rounds_per - 1) / p.rounds_per;
    return p;
}
// warps that fit an SM: by registers, and in fp32 by the rings
int forward_warps(const ScanArgs &) { return 28; }
int backward_warps(const ScanArgs &a) { return a.dtype == WTCONV_F32 ? 24 : 16; }

bool rows_at(const ScanTensor &s, const ScanArgs &a, int bytes) {
    const int per = bytes / elem_bytes_of(a.dtype);
    return aligned_to(s.p, bytes) && (a.B == 1 || s.batch % per == 0) && (a.C == 1 || s.row % per == 0);
}

size_t map_bytes(const ScanArgs &a, const Plan &p) {
    return p.segments > 1 ? ((size_t)a.B * a.C * p.segments * sizeof(float2) + 255) / 256 * 256 : 0;
}
unsigned short_grid(const ScanArgs &a, const Plan &p) {
    const long long per_cta = kShortThreads / p.lanes;
    return (unsigned)(((long long)a.B * a.C + per_cta - 1) / per_cta);
}

template <typename... P, typename... A>
cudaError_t launch(void (*kernel)(P...), unsigned grid, const Plan &p, size_t per_warp, cudaStream_t st, A... args) {
    return launch_kernel(kernel, grid, p.warps * 32, p.warps * per_warp, st, 1, args...);
}

template <typename T, int CP> cudaError_t forward_typed(const ScanArgs &a, cudaStream_t st) {
    const Plan p = plan_of(a, forward_warps(a));
    if (p.lanes > 0) {
        return launch_kernel(scan_short_forward_kernel<T, CP>, short_grid(a, p), kShortThreads, 0, st, 1, a, p.lanes);
    }
    const unsigned grid = (unsigned)((long long)a.B * a.C * p.segments);
    const size_t ring = sizeof(Ring<T, 2>);
    float2 *maps = static_cast<float2 *>(a.workspace);
    if (p.segments > 1) {
        const cudaError_t e = launch(scan_planes_forward_kernel<T, CP, kReduce>, grid, p, ring, st, a, p.segments, p.rounds_per, maps);
        if (e != cudaSuccess) return e;
    }
    return launch(scan_planes_forward_kernel<T, CP, kApply>, grid, p, ring, st, a, p.segments, p.rounds_per, maps);
}

template <typename T, int CP> cudaError_t backward_typed(const ScanArgs &a, cudaStream_t st) {
    const Plan p = plan_of(a, backward_warps(a));
    const unsigned grid = (unsigned)((long long)a.B * a.C * p.segments);
    const size_t ring = sizeof(Ring<T, 3>);
    float2 *maps = static_cast<float2 *>(a.workspace);
    float *part = reinterpret_cast<float *>(static_cast<char *>(a.workspace) + map_bytes(a, p));
    cudaError_t e = cudaSuccess;
    if (p.lanes > 0) {
        e = launch_kernel(scan_short_backward_kernel<T, CP>, short_grid(a, p), kShortThreads, 0, st, 1, a, p.lanes, part);
    } else {
        if (p.segments > 1) e = launch(scan_planes_backward_kernel<T, CP, kReduce>, grid, p, ring, st, a, p.segments, p.rounds_per, maps, part);
        if (e == cudaSuccess) e = launch(scan_planes_backward_kernel<T, CP, kApply>, grid, p, ring, st, a, p.segments, p.rounds_per, maps, part);
    }
    if (e != cudaSuccess) return e;
    return launch_kernel(scan_planes_bias_kernel, ceil_div(a.C, 4), 128, 0, st, 1, part, a.d_gate_bias, a.B, a.C, p.segments);
}

}  // namespace

size_t scan_planes_workspace(int op, const ScanArgs &a) {
    const bool back = op == WTCONV_SCAN_OP_BACKWARD;
    const Plan p = plan_of(a, back ? backward_warps(a) : forward_warps(a));
    const size_t part = back ? (size_t)a.B * a.C * p.segments * sizeof(float) : 0;
    return map_bytes(a, p) + (part + 255) / 256 * 256;
}

namespace {

// by the widest copies that every row's address allows
template <typename T> cudaError_t forward_any(const ScanArgs &a, cudaStream_t st) {
    const auto all = [&](int bytes) { return rows_at(a.x, a, bytes) && rows_at(a.gate, a, bytes) && rows_at(a.y, a, bytes); };
    if (all(16)) return forward_typed<T, 16>(a, st);
    if constexpr (sizeof(T) == 4) return forward_typed<T, 4>(a, st);
    else return all(4) ? forward_typed<T, 4>(a, st) : forward_typed<T, 2>(a, st);
}
template <typename T> cudaError_t backward_any(const ScanArgs &a, cudaStream_t st) {
    const auto all = [&](int bytes) {
        return rows_at(a.x, a, bytes) && rows_at(a.gate, a, bytes) && rows_at(a.dy, a, bytes) && rows_at(a.dx, a, bytes) &&
               rows_at(a.d_gate, a, bytes);
    };
    if (all(16)) return backward_typed<T, 16>(a, st);
    if constexpr (sizeof(T) == 4) return backward_typed<T, 4>(a, st);
    else return all(4) ? backward_typed<T, 4>(a, st) : backward_typed<T, 2>(a, st);
}

}  // namespace

cudaError_t launch_scan_planes_forward(const ScanArgs &a, cudaStream_t st) {
    if (a.dtype == WTCONV_F32) return forward_any<float>(a, st);
    return a.dtype == WTCONV_BF16 ? forward_any<__nv_bfloat16>(a, st) : forward_any<__half>(a, st);
}

cudaError_t launch_scan_planes_backward(const ScanArgs &a, cudaStream_t st) {
    if (a.dtype == WTCONV_F32) return backward_any<float>(a, st);
    return a.dtype == WTCONV_BF16 ? backward_any<__nv_bfloat16>(a, st) : backward_any<__half>(a, st);
}

}  // namespace wtconv
