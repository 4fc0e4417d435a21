// Gated scan of planes [B][C][T] (time contiguous): one CTA per row, or per segment of a long one.
//
// A warp takes 256 consecutive positions at a time, eight per lane.  A stretch of the recurrence is
// the map h -> a h + u, and such maps compose (Span), so each lane reduces its eight positions, the
// warp scans the lanes' maps by shuffles, the CTA's warps exchange theirs through shared memory (one
// barrier per round of 256 positions a warp), and every lane then runs its eight positions again from
// the state that reaches it: x, gate and (backward) dy are read once and everything stays in
// registers.  The next round's loads are issued before the barrier.  The state that a round leaves is
// carried to the next in a register of every thread.
//
// Few, long rows do not fill the GPU that way: they are cut into segments, a first kernel reduces
// each segment to its map, and the scan of a segment starts from the maps before it (after it,
// backward).  That reads two of the inputs twice, the second time mostly from L2.
#include "scan_device.cuh"

namespace wtconv {

namespace {

constexpr int kWarpSpan = 256;  // positions of a warp's round
constexpr int kMaxWarps = 8;
constexpr int kKeepLanes = WTCONV_SCAN_KEEP / 8;  // lanes between two kept states

enum Mode { kReduce, kApply };

// Map of the segments [first, last) of a row in time order, by all lanes of a warp alike.
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
    s = warp_scan<32, false>(s, lane);
    s.a = __shfl_sync(0xffffffffu, s.a, 31);
    s.u = __shfl_sync(0xffffffffu, s.u, 31);
    return s;
}

// One round's exchange between the CTA's warps.  mine: the warp's whole map (any lane: lane `from`
// holds it).  Returns the state before this warp's stretch and moves carry past the round.
__device__ __forceinline__ float exchange(Span mine, int from, float2 *slots, int warp, int warps, int lane, bool backward,
                                          float &carry) {
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
        const int w = backward ? warps - 1 - i : i;
        if (w == warp) before = carry;
        const float2 m = slots[w];
        carry = fmaf(m.x, carry, m.y);
    }
    return before;
}

struct Segment {
    int b, c, seg, n;              // n: length of the sequence
    long long row;                 // b * C + c
    int round0, round1;            // rounds of this segment
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

// ---------------------------------------------------------------------------------------- forward

template <typename T, bool VEC, Mode MODE>
__global__ void __launch_bounds__(kMaxWarps * 32) scan_planes_forward_kernel(const ScanArgs a, int segments, int rounds_per,
                                                                             float2 *maps) {
    __shared__ float2 slots[2][kMaxWarps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const int round_span = warps * kWarpSpan;
    const Segment s = segment_of(a, segments, rounds_per, round_span);
    const T *x = static_cast<const T *>(a.x.p) + s.b * a.x.batch + s.c * a.x.row;
    const T *g = static_cast<const T *>(a.gate.p) + s.b * a.gate.batch + s.c * a.gate.row;
    T *y = static_cast<T *>(a.y.p) + s.b * a.y.batch + s.c * a.y.row;
    const Pair bias(-kLog2E * a.gate_bias[s.c]);

    float carry = 0.f;
    Span whole = {1.f, 0.f};  // kReduce: the segment so far
    if (MODE == kApply) {
        carry = a.h0 != nullptr ? a.h0[s.row] : 0.f;
        if (s.seg > 0) carry = fold_segments(maps + s.row * segments, 0, s.seg, false, lane).of(carry);
    }
    int t = s.round0 * round_span + warp * kWarpSpan + lane * 8;
    Eight<T> nx, ng;
    nx.template load<VEC>(x + t, s.n - t);
    ng.template load<VEC>(g + t, s.n - t);
    for (int round = s.round0; round < s.round1; ++round, t += round_span) {
        const Eight<T> ex = nx, eg = ng;
        float av[8], uv[8];
        Span span = {1.f, 0.f};
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
            const Gates q = gates_of(Pair(eg.get(j), eg.get(j + 1)), bias);
            const Pair u = mul(q.b, Pair(ex.get(j), ex.get(j + 1)));
            av[j] = q.a.lo(), av[j + 1] = q.a.hi();
            uv[j] = u.lo(), uv[j + 1] = u.hi();
        }
        if (t + 8 > s.n) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (t + j >= s.n) av[j] = 1.f, uv[j] = 0.f;
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) span = span.then({av[j], uv[j]});
        if (round + 1 < s.round1) {
            nx.template load<VEC>(x + t + round_span, s.n - t - round_span);
            ng.template load<VEC>(g + t + round_span, s.n - t - round_span);
        }
        span = warp_scan<32, false>(span, lane);
        const Span before = lane_before<32, false>(span, lane);
        if (MODE == kReduce) {
            // every warp folds the whole round, so that all end with the segment's map
            float2 *slot = slots[round & 1];
            if (lane == 31) slot[warp] = make_float2(span.a, span.u);
            __syncthreads();
            for (int w = 0; w < warps; ++w) whole = whole.then({slot[w].x, slot[w].y});
            continue;
        }
        float h = before.of(exchange(span, 31, slots[round & 1], warp, warps, lane, false, carry));
        if (a.states_out != nullptr && (lane & (kKeepLanes - 1)) == 0 && t < a.T) a.states_out[s.row * a.keep + t / WTCONV_SCAN_KEEP] = h;
        Eight<T> out;
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
            const float h0 = fmaf(av[j], h, uv[j]);
            h = fmaf(av[j + 1], h0, uv[j + 1]);
            out.set(j, h0, h);
        }
        if (t + 8 > s.n) {  // past the length the state stands still, and y is 0
#pragma unroll
            for (int j = 0; j < 8; j += 2)
                out.set(j, t + j < s.n ? out.get(j) : 0.f, t + j + 1 < s.n ? out.get(j + 1) : 0.f);
        }
        out.template store<VEC>(y + t, a.T - t);
    }
    if (MODE == kReduce) {
        if (threadIdx.x == 0) maps[blockIdx.x] = make_float2(whole.a, whole.u);
    } else if (a.h_last != nullptr && s.seg == segments - 1 && threadIdx.x == 0) {
        a.h_last[s.row] = carry;
    }
}

// --------------------------------------------------------------------------------------- backward

template <typename T, bool VEC, Mode MODE>
__global__ void __launch_bounds__(kMaxWarps * 32) scan_planes_backward_kernel(const ScanArgs a, int segments, int rounds_per,
                                                                              float2 *maps, float *bias_part) {
    __shared__ float2 slots[2][kMaxWarps];
    __shared__ float sums[kMaxWarps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const int round_span = warps * kWarpSpan;
    const Segment s = segment_of(a, segments, rounds_per, round_span);
    const T *x = static_cast<const T *>(a.x.p) + s.b * a.x.batch + s.c * a.x.row;
    const T *g = static_cast<const T *>(a.gate.p) + s.b * a.gate.batch + s.c * a.gate.row;
    const T *dy = static_cast<const T *>(a.dy.p) + s.b * a.dy.batch + s.c * a.dy.row;
    T *dx = static_cast<T *>(a.dx.p) + s.b * a.dx.batch + s.c * a.dx.row;
    T *dg = static_cast<T *>(a.d_gate.p) + s.b * a.d_gate.batch + s.c * a.d_gate.row;
    const Pair bias(-kLog2E * a.gate_bias[s.c]);

    float carry = 0.f, sum = 0.f;  // carry: a_{t+1} dh_{t+1} of the position after this round
    Span whole = {1.f, 0.f};
    if (MODE == kApply) {
        carry = a.dh_last != nullptr ? a.dh_last[s.row] : 0.f;
        if (s.seg < segments - 1)
            carry = fold_segments(maps + s.row * segments, s.seg + 1, segments, true, lane).of(carry);
    }
    int t = (s.round1 - 1) * round_span + warp * kWarpSpan + lane * 8;
    Eight<T> nx, ng, ndy;
    float nh = 0.f;
    const auto fetch = [&](int at) {
        ng.template load<VEC>(g + at, s.n - at);
        ndy.template load<VEC>(dy + at, s.n - at);
        if (MODE == kApply) {
            nx.template load<VEC>(x + at, s.n - at);
            nh = at < a.T ? a.states_in[s.row * a.keep + at / WTCONV_SCAN_KEEP] : 0.f;
        }
    };
    fetch(t);
    for (int round = s.round1 - 1; round >= s.round0; --round, t -= round_span) {
        const Eight<T> ex = nx, eg = ng, edy = ndy;
        const float kept = nh;
        float av[8], bv[8];
        Span span = {1.f, 0.f};
        float flow = 0.f;
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
            const Gates q = gates_of(Pair(eg.get(j), eg.get(j + 1)), bias);
            av[j] = q.a.lo(), av[j + 1] = q.a.hi();
            bv[j] = q.b.lo(), bv[j + 1] = q.b.hi();
        }
        if (t + 8 > s.n) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (t + j >= s.n) av[j] = 1.f, bv[j] = 0.f;
        }
#pragma unroll
        for (int j = 7; j >= 0; --j) {
            flow = av[j] * (edy.get(j) + flow);
            span.a *= av[j];
        }
        span.u = flow;
        if (round > s.round0) fetch(t - round_span);
        float diff[8];  // h_{t-1} - x_t
        if (MODE == kApply) {
            // h again, by groups of lanes: a kept state stands before each
            Span fwd = {span.a, 0.f};
#pragma unroll
            for (int j = 0; j < 8; ++j) fwd.u = fmaf(av[j], fwd.u, bv[j] * ex.get(j));
            float h = lane_before<kKeepLanes, false>(warp_scan<kKeepLanes, false>(fwd, lane), lane).of(kept);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float xv = ex.get(j);
                diff[j] = h - xv;
                h = fmaf(av[j], h, bv[j] * xv);
            }
        }
        span = warp_scan<32, true>(span, lane);
        const Span after = lane_before<32, true>(span, lane);
        if (MODE == kReduce) {
            float2 *slot = slots[round & 1];
            if (lane == 0) slot[warp] = make_float2(span.a, span.u);
            __syncthreads();
            for (int w = warps - 1; w >= 0; --w) whole = whole.then({slot[w].x, slot[w].y});
            continue;
        }
        flow = after.of(exchange(span, 0, slots[round & 1], warp, warps, lane, true, carry));
        Eight<T> odx, odg;
#pragma unroll
        for (int j = 7; j > 0; j -= 2) {
            float dxv[2], dgv[2];
#pragma unroll
            for (int k = 1; k >= 0; --k) {
                const int i = j - 1 + k;
                const float dh = edy.get(i) + flow;
                dxv[k] = bv[i] * dh;
                dgv[k] = dh * diff[i] * (av[i] * bv[i]);
                sum += dgv[k];
                flow = av[i] * dh;
            }
            odx.set(j - 1, dxv[0], dxv[1]);
            odg.set(j - 1, dgv[0], dgv[1]);
        }
        odx.template store<VEC>(dx + t, a.T - t);
        odg.template store<VEC>(dg + t, a.T - t);
    }
    if (MODE == kReduce) {
        if (threadIdx.x == 0) maps[blockIdx.x] = make_float2(whole.a, whole.u);
        return;
    }
    sum = warp_sum(sum);
    if (lane == 0) sums[warp] = sum;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int w = 1; w < warps; ++w) sum += sums[w];
        bias_part[blockIdx.x] = sum;
        if (a.d_h0 != nullptr && s.seg == 0) a.d_h0[s.row] = carry;
    }
}

// d_gate_bias_c = sum over sequences and segments of the parts, in a fixed order: one warp per channel.
__global__ void __launch_bounds__(128) scan_planes_bias_kernel(const float *part, float *out, int B, int C, int segments) {
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

// How rows are cut.  warps: 256 positions each; as many as a row has work for, at most eight (four
// where rows alone fill the GPU).  segments > 1 only where the rows leave most of the GPU idle.
struct Plan {
    int warps, segments, rounds_per;
};
Plan plan_of(const ScanArgs &a) {
    Plan p;
    const long long rows = (long long)a.B * a.C;
    const int spans = (a.T + kWarpSpan - 1) / kWarpSpan, sms = sm_count();
    p.warps = rows >= 4ll * sms ? 4 : kMaxWarps;
    while (p.warps > 1 && p.warps / 2 >= spans) p.warps /= 2;
    const int rounds = (spans + p.warps - 1) / p.warps;
    const long long want = 4ll * sms;
    p.segments = 1;
    if (rows * 2 < want) p.segments = (int)((want + rows - 1) / rows);
    if (p.segments > rounds) p.segments = rounds;
    p.rounds_per = (rounds + p.segments - 1) / p.segments;
    p.segments = (rounds + p.rounds_per - 1) / p.rounds_per;
    return p;
}

bool rows_aligned(const ScanTensor &s, const ScanArgs &a) {
    const int per = 16 / elem_bytes_of(a.dtype);
    return aligned_to(s.p, 16) && (a.B == 1 || s.batch % per == 0) && (a.C == 1 || s.row % per == 0);
}

size_t map_bytes(const ScanArgs &a, const Plan &p) {
    return p.segments > 1 ? ((size_t)a.B * a.C * p.segments * sizeof(float2) + 255) / 256 * 256 : 0;
}

template <typename T, bool VEC> cudaError_t forward_typed(const ScanArgs &a, const Plan &p, cudaStream_t st) {
    const unsigned grid = (unsigned)((long long)a.B * a.C * p.segments);
    float2 *maps = static_cast<float2 *>(a.workspace);
    if (p.segments > 1)
        scan_planes_forward_kernel<T, VEC, kReduce><<<grid, p.warps * 32, 0, st>>>(a, p.segments, p.rounds_per, maps);
    scan_planes_forward_kernel<T, VEC, kApply><<<grid, p.warps * 32, 0, st>>>(a, p.segments, p.rounds_per, maps);
    return cudaGetLastError();
}

template <typename T, bool VEC> cudaError_t backward_typed(const ScanArgs &a, const Plan &p, cudaStream_t st) {
    const unsigned grid = (unsigned)((long long)a.B * a.C * p.segments);
    float2 *maps = static_cast<float2 *>(a.workspace);
    float *part = reinterpret_cast<float *>(static_cast<char *>(a.workspace) + map_bytes(a, p));
    if (p.segments > 1)
        scan_planes_backward_kernel<T, VEC, kReduce><<<grid, p.warps * 32, 0, st>>>(a, p.segments, p.rounds_per, maps, part);
    scan_planes_backward_kernel<T, VEC, kApply><<<grid, p.warps * 32, 0, st>>>(a, p.segments, p.rounds_per, maps, part);
    scan_planes_bias_kernel<<<(a.C + 3) / 4, 128, 0, st>>>(part, a.d_gate_bias, a.B, a.C, p.segments);
    return cudaGetLastError();
}

}  // namespace

size_t scan_planes_workspace(int op, const ScanArgs &a) {
    const Plan p = plan_of(a);
    const size_t part = op == WTCONV_SCAN_OP_BACKWARD ? (size_t)a.B * a.C * p.segments * sizeof(float) : 0;
    return map_bytes(a, p) + (part + 255) / 256 * 256;
}

cudaError_t launch_scan_planes_forward(const ScanArgs &a, cudaStream_t st) {
    const Plan p = plan_of(a);
    const bool vec = rows_aligned(a.x, a) && rows_aligned(a.gate, a) && rows_aligned(a.y, a);
    if (a.dtype == WTCONV_F32) return vec ? forward_typed<float, true>(a, p, st) : forward_typed<float, false>(a, p, st);
    if (a.dtype == WTCONV_BF16)
        return vec ? forward_typed<__nv_bfloat16, true>(a, p, st) : forward_typed<__nv_bfloat16, false>(a, p, st);
    return vec ? forward_typed<__half, true>(a, p, st) : forward_typed<__half, false>(a, p, st);
}

cudaError_t launch_scan_planes_backward(const ScanArgs &a, cudaStream_t st) {
    const Plan p = plan_of(a);
    const bool vec = rows_aligned(a.x, a) && rows_aligned(a.gate, a) && rows_aligned(a.dy, a) && rows_aligned(a.dx, a) &&
                     rows_aligned(a.d_gate, a);
    if (a.dtype == WTCONV_F32) return vec ? backward_typed<float, true>(a, p, st) : backward_typed<float, false>(a, p, st);
    if (a.dtype == WTCONV_BF16)
        return vec ? backward_typed<__nv_bfloat16, true>(a, p, st) : backward_typed<__nv_bfloat16, false>(a, p, st);
    return vec ? backward_typed<__half, true>(a, p, st) : backward_typed<__half, false>(a, p, st);
}

}  // namespace wtconv
