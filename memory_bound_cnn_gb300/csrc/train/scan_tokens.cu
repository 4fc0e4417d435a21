// Gated scan of tokens [B][T][C] (channels contiguous): one CTA per strip of channels of a sequence,
// or a cluster of CTAs along its time.
//
// A round is 64 positions of a strip: 128 bytes of every row, brought into shared memory by
// asynchronous copies two rounds ahead.  A lane owns V neighbouring channels (4 bytes) and a warp
// eight consecutive positions of them, which each lane reduces to the map h -> a h + u of the state
// before them (Span, scan_device.cuh).  The eight warps exchange their maps through shared memory, and
// every lane runs its eight positions again from the state that reaches it, out of registers: x, gate
// and (backward) dy are read once.
//
// A strip of a sequence is a chain along time.  Where there are too few of them to fill the GPU, R
// CTAs of a cluster share one: in a round CTA r takes the r-th 64 positions, pushes its map into the
// shared memory of the others, and after the cluster's barrier each folds the maps before its own.
// Where even that leaves most SMs idle, the sequence is cut into segments whose maps a first kernel
// reduces (reading two inputs twice, the second time mostly from L2).
#include <cooperative_groups.h>

#include <initializer_list>

#include "scan_device.cuh"

namespace wtconv {

namespace {

namespace cg = cooperative_groups;

constexpr int kWarps = 8, kThreads = kWarps * 32, kSteps = 8;
constexpr int kSpan = kWarps * kSteps;  // positions of a CTA's round
static_assert(kSpan == WTCONV_SCAN_KEEP, "a round starts at a kept state");
constexpr int kMaxCluster = 8;
constexpr int kRowBytes = 128;  // of a strip

enum Mode { kReduce, kApply };

// 32 * V channels of kSpan positions of one tensor.
template <typename T, int V> struct Tile {
    static_assert(32 * V * sizeof(T) == kRowBytes, "");
    T v[kSpan][32 * V];
};

// Copies of CP bytes: 16 or 4 asynchronously (what is past the length or the last channel reads as
// zeros and is not touched), 2 through registers.
template <int CP> __device__ __forceinline__ void copy_async(void *to, const void *from, int bytes) {
    const unsigned dst = (unsigned)__cvta_generic_to_shared(to);
    if constexpr (CP == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(from), "r"(bytes) : "memory");
    else asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(from), "r"(bytes) : "memory");
}
__device__ __forceinline__ void commit_copies() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int PENDING> __device__ __forceinline__ void wait_copies() {
    asm volatile("cp.async.wait_group %0;" ::"n"(PENDING) : "memory");
}
// rows: valid positions from `from` on; width: valid channels of the strip
template <typename T, int V, int CP>
__device__ __forceinline__ void fetch_tile(Tile<T, V> &tile, const T *from, long long row, int rows, int width) {
    constexpr int per_row = kRowBytes / CP, elems = CP / (int)sizeof(T);
#pragma unroll
    for (int k = 0; k < kSpan * per_row / kThreads; ++k) {
        const int i = k * kThreads + threadIdx.x, r = i / per_row, c = (i - r * per_row) * elems;
        const int left = r < rows ? width - c : 0;
        T *to = &tile.v[r][c];
        if constexpr (CP == 2) *to = left > 0 ? from[r * row + c] : from_f32<T>(0.f);
        else copy_async<CP>(to, left > 0 ? from + (r * row + c) : from, left <= 0 ? 0 : left >= elems ? CP : left * (int)sizeof(T));
    }
}

template <typename T, int V> __device__ __forceinline__ void read_few(const Tile<T, V> &tile, int r, int lane, float (&v)[V]) {
    if constexpr (V == 1) v[0] = to_f32(tile.v[r][lane]);
    else {
        const uint32_t q = *reinterpret_cast<const uint32_t *>(&tile.v[r][lane * 2]);
        const uint16_t lo = (uint16_t)q, hi = (uint16_t)(q >> 16);
        v[0] = to_f32(*reinterpret_cast<const T *>(&lo)), v[1] = to_f32(*reinterpret_cast<const T *>(&hi));
    }
}
// V values of one row; `both`: the address is a multiple of 4 bytes and all V are there
template <typename T, int V> __device__ __forceinline__ void store_few(T *p, const float (&v)[V], bool both, int width) {
    if constexpr (V == 1) {
        if (width > 0) *p = from_f32<T>(v[0]);
    } else {
        const T lo = from_f32<T>(v[0]), hi = from_f32<T>(v[1]);
        if (both) {
            *reinterpret_cast<uint32_t *>(p) = (uint32_t)*reinterpret_cast<const uint16_t *>(&lo) |
                                               (uint32_t)*reinterpret_cast<const uint16_t *>(&hi) << 16;
        } else {
            if (width > 0) p[0] = lo;
            if (width > 1) p[1] = hi;
        }
    }
}

struct TokenPlan {
    int strips, cluster, segments, rounds_per;  // rounds_per: rounds of the cluster in a segment
};

template <int V> struct Shared {
    float2 warp_maps[2][kWarps][32 * V];
    float2 cta_maps[2][kMaxCluster][32 * V];
};

// Exchange of one round.  mine[v]: the warp's maps.  before[v]: the state before this warp's
// positions; carry[v] moves past the round.  BACKWARD: the last warp and CTA come first.
template <int V, bool BACKWARD>
__device__ __forceinline__ void exchange(const Span (&mine)[V], Shared<V> &sh, int parity, int warp, int lane, int cluster,
                                         int rank, float (&carry)[V], float (&before)[V]) {
#pragma unroll
    for (int v = 0; v < V; ++v) sh.warp_maps[parity][warp][lane * V + v] = make_float2(mine[v].a, mine[v].u);
    __syncthreads();
    if (cluster == 1) {
#pragma unroll
        for (int i = 0; i < kWarps; ++i) {
            const int w = BACKWARD ? kWarps - 1 - i : i;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                if (w == warp) before[v] = carry[v];
                const float2 m = sh.warp_maps[parity][w][lane * V + v];
                carry[v] = fmaf(m.x, carry[v], m.y);
            }
        }
        return;
    }
    Span pre[V], all[V];
#pragma unroll
    for (int v = 0; v < V; ++v) all[v] = {1.f, 0.f};
#pragma unroll
    for (int i = 0; i < kWarps; ++i) {
        const int w = BACKWARD ? kWarps - 1 - i : i;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            if (w == warp) pre[v] = all[v];
            const float2 m = sh.warp_maps[parity][w][lane * V + v];
            all[v] = all[v].then({m.x, m.y});
        }
    }
    cg::cluster_group group = cg::this_cluster();
    if (warp < cluster) {  // warp r brings the CTA's map to CTA r
        Shared<V> *there = group.map_shared_rank(&sh, warp);
#pragma unroll
        for (int v = 0; v < V; ++v) there->cta_maps[parity][rank][lane * V + v] = make_float2(all[v].a, all[v].u);
    }
    group.sync();
    float start[V];
    for (int i = 0; i < cluster; ++i) {
        const int r = BACKWARD ? cluster - 1 - i : i;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            if (r == rank) start[v] = carry[v];
            const float2 m = sh.cta_maps[parity][r][lane * V + v];
            carry[v] = fmaf(m.x, carry[v], m.y);
        }
    }
#pragma unroll
    for (int v = 0; v < V; ++v) before[v] = pre[v].of(start[v]);
}

// A round of a segment's reduction: every warp appends all warps' maps to whole.
template <int V, bool BACKWARD>
__device__ __forceinline__ void reduce_round(const Span (&mine)[V], Shared<V> &sh, int parity, int warp, int lane,
                                             Span (&whole)[V]) {
#pragma unroll
    for (int v = 0; v < V; ++v) sh.warp_maps[parity][warp][lane * V + v] = make_float2(mine[v].a, mine[v].u);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kWarps; ++i)
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const float2 m = sh.warp_maps[parity][BACKWARD ? kWarps - 1 - i : i][lane * V + v];
            whole[v] = whole[v].then({m.x, m.y});
        }
}

// State that the segments before (after, if BACKWARD) this one leave, from carry: their maps are
// folded by the warps in parallel, then as in a round.
template <int V, bool BACKWARD>
__device__ __forceinline__ void fold_segments(const float2 *maps, int first, int last, Shared<V> &sh, int warp, int lane,
                                              float (&carry)[V]) {
    const int count = last - first, per = (count + kWarps - 1) / kWarps;
    Span mine[V];
#pragma unroll
    for (int v = 0; v < V; ++v) mine[v] = {1.f, 0.f};
    const int place = BACKWARD ? kWarps - 1 - warp : warp;
    for (int k = 0; k < per; ++k) {
        const int i = place * per + k;
        if (i >= count) break;
        const float2 *m = maps + (long long)(BACKWARD ? last - 1 - i : first + i) * (32 * V) + lane * V;
#pragma unroll
        for (int v = 0; v < V; ++v) mine[v] = mine[v].then({m[v].x, m[v].y});
    }
    float before[V];
    exchange<V, BACKWARD>(mine, sh, 0, warp, lane, 1, 0, carry, before);
    __syncthreads();
}

struct Place {
    int b, seg, rank, n, c0, c;  // first channel of the strip and of the lane
    int width;                   // channels that the lane has (V, fewer at the end, or <= 0)
    long long unit;              // (b * strips + strip) * segments
};
template <int V> __device__ __forceinline__ Place place_of(const ScanArgs &a, const TokenPlan &p, int lane) {
    Place s;
    s.rank = blockIdx.x % p.cluster;
    unsigned i = blockIdx.x / p.cluster;
    s.seg = i % p.segments;
    i /= p.segments;
    s.unit = (long long)i * p.segments;
    const int strip = i % p.strips;
    s.b = i / p.strips;
    s.c0 = strip * 32 * V;
    s.c = s.c0 + lane * V;
    s.width = a.C - s.c;
    s.n = scan_length(a.lengths, s.b, a.T);
    return s;
}

// ---------------------------------------------------------------------------------------- forward

template <typename T, int V> struct ForwardShared {
    Tile<T, V> x[2], g[2];
    Shared<V> maps;
};

// CP: bytes of a copy; PAIRED: the outputs' rows allow 4-byte stores
template <typename T, int V, int CP, bool PAIRED, Mode MODE>
__global__ void __launch_bounds__(kThreads, 4) scan_tokens_forward_kernel(const ScanArgs a, const TokenPlan p, float2 *maps) {
    extern __shared__ __align__(16) unsigned char raw[];
    ForwardShared<T, V> &sh = *reinterpret_cast<ForwardShared<T, V> *>(raw);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const Place s = place_of<V>(a, p, lane);
    const int round_span = p.cluster * kSpan, rounds = (a.T + round_span - 1) / round_span;
    const int round0 = s.seg * p.rounds_per, round1 = min(round0 + p.rounds_per, rounds);
    int t0 = round0 * round_span + s.rank * kSpan;  // the CTA's first position of the round
    const T *x = static_cast<const T *>(a.x.p) + s.b * a.x.batch + s.c0 + t0 * a.x.row;
    const T *g = static_cast<const T *>(a.gate.p) + s.b * a.gate.batch + s.c0 + t0 * a.gate.row;
    T *y = static_cast<T *>(a.y.p) + s.b * a.y.batch + s.c + (t0 + warp * kSteps) * a.y.row;
    const auto fetch = [&](int k) {  // the round k rounds ahead
        const int at = t0 + k * round_span;
        if (at < s.n) {
            fetch_tile<T, V, CP>(sh.x[(at / round_span) & 1], x + k * (round_span * a.x.row), a.x.row, s.n - at, a.C - s.c0);
            fetch_tile<T, V, CP>(sh.g[(at / round_span) & 1], g + k * (round_span * a.gate.row), a.gate.row, s.n - at, a.C - s.c0);
        }
        commit_copies();
    };
    fetch(0);
    if (round0 + 1 < round1) fetch(1);
    else commit_copies();

    float bias[V], carry[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        bias[v] = v < s.width ? a.gate_bias[s.c + v] : 0.f;
        carry[v] = MODE == kApply && a.h0 != nullptr && v < s.width ? a.h0[(long long)s.b * a.C + s.c + v] : 0.f;
    }
    if (MODE == kApply && s.seg > 0) fold_segments<V, false>(maps + s.unit * 32 * V, 0, s.seg, sh.maps, warp, lane, carry);
    Span whole[V];
#pragma unroll
    for (int v = 0; v < V; ++v) whole[v] = {1.f, 0.f};
    wait_copies<1>();
    if (p.cluster > 1) cg::this_cluster().sync();  // the others' shared memory is there
    else __syncthreads();
    for (int round = round0; round < round1; ++round) {
        const int t = t0 + warp * kSteps;
        const Tile<T, V> &tx = sh.x[round & 1], &tg = sh.g[round & 1];
        float av[kSteps][V], uv[kSteps][V];
        Span span[V];
#pragma unroll
        for (int v = 0; v < V; ++v) span[v] = {1.f, 0.f};
#pragma unroll
        for (int j = 0; j < kSteps; ++j) {
            const bool live = t + j < s.n;
            float xv[V], gv[V];
            read_few(tx, warp * kSteps + j, lane, xv);
            read_few(tg, warp * kSteps + j, lane, gv);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const Gate q = gate_of(gv[v] + bias[v]);
                av[j][v] = live ? q.a : 1.f;
                uv[j][v] = live ? q.b * xv[v] : 0.f;
                span[v] = span[v].then({av[j][v], uv[j][v]});
            }
        }
        // the barrier inside the exchange ends all reading of this round's tiles and shows the next's
        wait_copies<0>();
        float h[V];
        if constexpr (MODE == kReduce) {
            reduce_round<V, false>(span, sh.maps, round & 1, warp, lane, whole);
        } else {
            exchange<V, false>(span, sh.maps, round & 1, warp, lane, p.cluster, s.rank, carry, h);
        }
        if (round + 2 < round1) fetch(2);
        if constexpr (MODE == kApply) {
            if (a.states_out != nullptr && warp == 0 && t0 < a.T) {
#pragma unroll
                for (int v = 0; v < V; ++v)
                    if (v < s.width) a.states_out[((long long)s.b * a.keep + t0 / WTCONV_SCAN_KEEP) * a.C + s.c + v] = h[v];
            }
#pragma unroll
            for (int j = 0; j < kSteps; ++j) {
                float out[V];
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    h[v] = fmaf(av[j][v], h[v], uv[j][v]);
                    out[v] = t + j < s.n ? h[v] : 0.f;
                }
                if (t + j < a.T) store_few<T, V>(y + j * a.y.row, out, PAIRED && s.width >= V, s.width);
            }
            y += round_span * a.y.row;
        }
        t0 += round_span, x += round_span * a.x.row, g += round_span * a.gate.row;
    }
    if constexpr (MODE == kReduce) {
        if (warp == 0) {
#pragma unroll
            for (int v = 0; v < V; ++v) maps[(s.unit + s.seg) * 32 * V + lane * V + v] = make_float2(whole[v].a, whole[v].u);
        }
    } else if (a.h_last != nullptr && s.seg == p.segments - 1 && s.rank == 0 && warp == 0) {
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (v < s.width) a.h_last[(long long)s.b * a.C + s.c + v] = carry[v];
    }
}

// --------------------------------------------------------------------------------------- backward

template <typename T, int V> struct BackwardShared {
    Tile<T, V> x[2], g[2], dy[2];
    Shared<V> maps;
    float2 forward_maps[kWarps][32 * V];
};

// bias_part: one float per (unit, segment, rank, channel of the strip)
template <typename T, int V, int CP, bool PAIRED, Mode MODE>
__global__ void __launch_bounds__(kThreads, 2) scan_tokens_backward_kernel(const ScanArgs a, const TokenPlan p, float2 *maps,
                                                                           float *bias_part) {
    extern __shared__ __align__(16) unsigned char raw[];
    BackwardShared<T, V> &sh = *reinterpret_cast<BackwardShared<T, V> *>(raw);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const Place s = place_of<V>(a, p, lane);
    const int round_span = p.cluster * kSpan, rounds = (a.T + round_span - 1) / round_span;
    const int round0 = s.seg * p.rounds_per, round1 = min(round0 + p.rounds_per, rounds);
    int t0 = (round1 - 1) * round_span + s.rank * kSpan;
    const T *x = static_cast<const T *>(a.x.p) + s.b * a.x.batch + s.c0 + t0 * a.x.row;
    const T *g = static_cast<const T *>(a.gate.p) + s.b * a.gate.batch + s.c0 + t0 * a.gate.row;
    const T *dy = static_cast<const T *>(a.dy.p) + s.b * a.dy.batch + s.c0 + t0 * a.dy.row;
    T *dx = static_cast<T *>(a.dx.p) + s.b * a.dx.batch + s.c + (t0 + warp * kSteps) * a.dx.row;
    T *dg = static_cast<T *>(a.d_gate.p) + s.b * a.d_gate.batch + s.c + (t0 + warp * kSteps) * a.d_gate.row;
    const auto fetch = [&](int k) {  // the round k rounds on, towards the beginning
        const int at = t0 - k * round_span, buf = (at / round_span) & 1;
        if (at < s.n) {
            fetch_tile<T, V, CP>(sh.g[buf], g - k * (round_span * a.gate.row), a.gate.row, s.n - at, a.C - s.c0);
            fetch_tile<T, V, CP>(sh.dy[buf], dy - k * (round_span * a.dy.row), a.dy.row, s.n - at, a.C - s.c0);
            if (MODE == kApply) fetch_tile<T, V, CP>(sh.x[buf], x - k * (round_span * a.x.row), a.x.row, s.n - at, a.C - s.c0);
        }
        commit_copies();
    };
    fetch(0);
    if (round0 + 1 < round1) fetch(1);
    else commit_copies();

    float bias[V], carry[V], sum[V], nh[V];
    Span whole[V];
    const auto kept_state = [&](int at) {
#pragma unroll
        for (int v = 0; v < V; ++v)
            nh[v] = MODE == kApply && v < s.width && at < a.T
                        ? a.states_in[((long long)s.b * a.keep + at / WTCONV_SCAN_KEEP) * a.C + s.c + v] : 0.f;
    };
    kept_state(t0);
#pragma unroll
    for (int v = 0; v < V; ++v) {
        bias[v] = v < s.width ? a.gate_bias[s.c + v] : 0.f;
        carry[v] = MODE == kApply && a.dh_last != nullptr && v < s.width ? a.dh_last[(long long)s.b * a.C + s.c + v] : 0.f;
        sum[v] = 0.f;
        whole[v] = {1.f, 0.f};
    }
    if (MODE == kApply && s.seg < p.segments - 1)
        fold_segments<V, true>(maps + s.unit * 32 * V, s.seg + 1, p.segments, sh.maps, warp, lane, carry);
    wait_copies<1>();
    if (p.cluster > 1) cg::this_cluster().sync();  // the others' shared memory is there
    else __syncthreads();
    for (int round = round1 - 1; round >= round0; --round) {
        const int t = t0 + warp * kSteps;
        const Tile<T, V> &tx = sh.x[round & 1], &tg = sh.g[round & 1], &tdy = sh.dy[round & 1];
        float av[kSteps][V], bv[kSteps][V], diff[kSteps][V], dyv[kSteps][V], kept[V];
        Span back[V], fwd[V];
#pragma unroll
        for (int v = 0; v < V; ++v) back[v] = {1.f, 0.f}, fwd[v] = {1.f, 0.f}, kept[v] = nh[v];
#pragma unroll
        for (int j = kSteps - 1; j >= 0; --j) {
            const bool live = t + j < s.n;
            float gv[V];
            read_few(tg, warp * kSteps + j, lane, gv);
            read_few(tdy, warp * kSteps + j, lane, dyv[j]);
            if (MODE == kApply) read_few(tx, warp * kSteps + j, lane, diff[j]);  // x, until h is known
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const Gate q = gate_of(gv[v] + bias[v]);
                av[j][v] = live ? q.a : 1.f;
                bv[j][v] = live ? q.b : 0.f;
                if (!live) dyv[j][v] = diff[j][v] = 0.f;
                back[v].u = av[j][v] * (dyv[j][v] + back[v].u);
                back[v].a *= av[j][v];
            }
        }
        wait_copies<0>();
        if constexpr (MODE == kReduce) {
            reduce_round<V, true>(back, sh.maps, round & 1, warp, lane, whole);
            if (round - 2 >= round0) fetch(2);
        } else {
            // h is scanned forward within the CTA's positions from the kept state; dh comes backward
#pragma unroll
            for (int j = 0; j < kSteps; ++j)
#pragma unroll
                for (int v = 0; v < V; ++v) fwd[v] = fwd[v].then({av[j][v], bv[j][v] * diff[j][v]});
#pragma unroll
            for (int v = 0; v < V; ++v) sh.forward_maps[warp][lane * V + v] = make_float2(fwd[v].a, fwd[v].u);
            float flow[V], h[V];
            exchange<V, true>(back, sh.maps, round & 1, warp, lane, p.cluster, s.rank, carry, flow);
            if (round - 2 >= round0) fetch(2);
            if (round > round0) kept_state(t0 - round_span);
#pragma unroll
            for (int v = 0; v < V; ++v) h[v] = kept[v];
            for (int w = 0; w < warp; ++w)
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    const float2 m = sh.forward_maps[w][lane * V + v];
                    h[v] = fmaf(m.x, h[v], m.y);
                }
            __syncthreads();  // forward_maps is written again in the next round
#pragma unroll
            for (int j = 0; j < kSteps; ++j)
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    const float xv = diff[j][v];
                    diff[j][v] = h[v] - xv;
                    h[v] = fmaf(av[j][v], h[v], bv[j][v] * xv);
                }
#pragma unroll
            for (int j = kSteps - 1; j >= 0; --j) {
                float dxv[V], dgv[V];
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    const float dh = dyv[j][v] + flow[v];
                    dxv[v] = bv[j][v] * dh;
                    dgv[v] = dh * diff[j][v] * (av[j][v] * bv[j][v]);
                    sum[v] += dgv[v];
                    flow[v] = av[j][v] * dh;
                }
                if (t + j < a.T) {
                    store_few<T, V>(dx + j * a.dx.row, dxv, PAIRED && s.width >= V, s.width);
                    store_few<T, V>(dg + j * a.d_gate.row, dgv, PAIRED && s.width >= V, s.width);
                }
            }
            dx -= round_span * a.dx.row, dg -= round_span * a.d_gate.row;
        }
        t0 -= round_span, x -= round_span * a.x.row, g -= round_span * a.gate.row, dy -= round_span * a.dy.row;
    }
    if constexpr (MODE == kReduce) {
        if (warp == 0) {
#pragma unroll
            for (int v = 0; v < V; ++v) maps[(s.unit + s.seg) * 32 * V + lane * V + v] = make_float2(whole[v].a, whole[v].u);
        }
    } else {
        if (a.d_h0 != nullptr && s.seg == 0 && s.rank == 0 && warp == 0) {
#pragma unroll
            for (int v = 0; v < V; ++v)
                if (v < s.width) a.d_h0[(long long)s.b * a.C + s.c + v] = carry[v];
        }
        float *sums = reinterpret_cast<float *>(sh.forward_maps);
#pragma unroll
        for (int v = 0; v < V; ++v) sums[warp * 32 * V + lane * V + v] = sum[v];
        __syncthreads();
        if (threadIdx.x < 32 * V) {
            float total = 0.f;
            for (int w = 0; w < kWarps; ++w) total += sums[w * 32 * V + threadIdx.x];
            bias_part[((s.unit + s.seg) * p.cluster + s.rank) * 32 * V + threadIdx.x] = total;
        }
    }
}

// d_gate_bias_c = sum of the parts over sequences, segments and ranks, in a fixed order.
__global__ void __launch_bounds__(256) scan_tokens_bias_kernel(const float *part, float *out, int B, int C, int strips,
                                                               int per_unit, int width) {
    __shared__ float sums[8][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + lane;
    float sum = 0.f;
    if (c < C) {
        const int strip = c / width, count = B * per_unit;
        for (int i = warp; i < count; i += 8) {
            const int b = i / per_unit;
            sum += part[(((long long)b * strips + strip) * per_unit + (i - b * per_unit)) * width + (c - strip * width)];
        }
    }
    sums[warp][lane] = sum;
    __syncthreads();
    if (warp == 0 && c < C) {
        for (int w = 1; w < 8; ++w) sum += sums[w][lane];
        out[c] = sum;
    }
}

// Chains (strips of sequences) that do not give every SM `per_sm` CTAs are shared by clusters; where
// even full clusters give less than one CTA to every second SM, sequences are cut into segments.
TokenPlan plan_of(const ScanArgs &a, int V, int per_sm) {
    TokenPlan p;
    p.strips = (a.C + 32 * V - 1) / (32 * V);
    const long long sms = sm_count(), chains = (long long)a.B * p.strips, want = per_sm * sms;
    const int rounds = (a.T + kSpan - 1) / kSpan;
    p.cluster = p.segments = 1;
    if (chains * kMaxCluster * 2 >= sms) {
        while (p.cluster < kMaxCluster && chains * p.cluster < want && p.cluster < rounds) p.cluster *= 2;
    } else {
        p.segments = (int)((want + chains - 1) / chains);
        if (p.segments > rounds) p.segments = rounds;
    }
    const int cluster_rounds = (rounds + p.cluster - 1) / p.cluster;
    p.rounds_per = (cluster_rounds + p.segments - 1) / p.segments;
    p.segments = (cluster_rounds + p.rounds_per - 1) / p.rounds_per;
    return p;
}
constexpr int kForwardPerSm = 4, kBackwardPerSm = 2;  // CTAs that fit an SM

size_t round256(size_t n) { return (n + 255) / 256 * 256; }
size_t map_bytes(const ScanArgs &a, const TokenPlan &p, int V) {
    return p.segments > 1 ? round256((size_t)a.B * p.strips * p.segments * 32 * V * sizeof(float2)) : 0;
}
size_t part_bytes(const ScanArgs &a, const TokenPlan &p, int V) {
    return round256((size_t)a.B * p.strips * p.segments * p.cluster * 32 * V * sizeof(float));
}

template <typename... P, typename... A>
cudaError_t launch(void (*kernel)(P...), size_t shared, const ScanArgs &a, const TokenPlan &p, cudaStream_t st, A... args) {
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)shared);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t config = {};
    config.gridDim = dim3((unsigned)((long long)a.B * p.strips * p.segments * p.cluster));
    config.blockDim = dim3(kThreads);
    config.dynamicSmemBytes = shared;
    config.stream = st;
    cudaLaunchAttribute attr = {};
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = p.cluster, attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    config.attrs = &attr;
    config.numAttrs = p.cluster > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&config, kernel, a, p, args...);
}

// Whether every row of a tensor starts at a multiple of `bytes`.
bool rows_at(const ScanTensor &s, const ScanArgs &a, int bytes) {
    const int per = bytes / elem_bytes_of(a.dtype);
    return aligned_to(s.p, bytes) && (a.B == 1 || s.batch % per == 0) && (a.T == 1 || s.row % per == 0);
}

template <typename T, int V, int CP, bool PAIRED> cudaError_t forward_typed(const ScanArgs &a, cudaStream_t st) {
    const TokenPlan p = plan_of(a, V, kForwardPerSm);
    const size_t shared = sizeof(ForwardShared<T, V>);
    float2 *maps = static_cast<float2 *>(a.workspace);
    if (p.segments > 1) {
        const cudaError_t e = launch(scan_tokens_forward_kernel<T, V, CP, PAIRED, kReduce>, shared, a, p, st, maps);
        if (e != cudaSuccess) return e;
    }
    return launch(scan_tokens_forward_kernel<T, V, CP, PAIRED, kApply>, shared, a, p, st, maps);
}

template <typename T, int V, int CP, bool PAIRED> cudaError_t backward_typed(const ScanArgs &a, cudaStream_t st) {
    const TokenPlan p = plan_of(a, V, kBackwardPerSm);
    const size_t shared = sizeof(BackwardShared<T, V>);
    float2 *maps = static_cast<float2 *>(a.workspace);
    float *part = reinterpret_cast<float *>(static_cast<char *>(a.workspace) + map_bytes(a, p, V));
    cudaError_t e = cudaSuccess;
    if (p.segments > 1) e = launch(scan_tokens_backward_kernel<T, V, CP, PAIRED, kReduce>, shared, a, p, st, maps, part);
    if (e == cudaSuccess) e = launch(scan_tokens_backward_kernel<T, V, CP, PAIRED, kApply>, shared, a, p, st, maps, part);
    if (e != cudaSuccess) return e;
    scan_tokens_bias_kernel<<<(a.C + 31) / 32, 256, 0, st>>>(part, a.d_gate_bias, a.B, a.C, p.strips,
                                                            p.segments * p.cluster, 32 * V);
    return cudaGetLastError();
}

// Width of the copies that bring the inputs in, and whether 16-bit outputs can be stored in pairs.
struct Access {
    int copy;
    bool paired;
};
Access access_of(const ScanArgs &a, std::initializer_list<const ScanTensor *> in, std::initializer_list<const ScanTensor *> out) {
    Access w = {16, true};
    for (const ScanTensor *s : in)
        while (!rows_at(*s, a, w.copy)) w.copy = w.copy == 16 ? 4 : 2;
    for (const ScanTensor *s : out) w.paired = w.paired && rows_at(*s, a, 4);
    w.paired = w.paired && w.copy >= 4;
    return w;
}

template <typename T> cudaError_t forward_16(const ScanArgs &a, const Access &w, cudaStream_t st) {
    if (w.copy == 16) return w.paired ? forward_typed<T, 2, 16, true>(a, st) : forward_typed<T, 2, 2, false>(a, st);
    return w.paired ? forward_typed<T, 2, 4, true>(a, st) : forward_typed<T, 2, 2, false>(a, st);
}
template <typename T> cudaError_t backward_16(const ScanArgs &a, const Access &w, cudaStream_t st) {
    if (w.copy == 16) return w.paired ? backward_typed<T, 2, 16, true>(a, st) : backward_typed<T, 2, 2, false>(a, st);
    return w.paired ? backward_typed<T, 2, 4, true>(a, st) : backward_typed<T, 2, 2, false>(a, st);
}

// ------------------------------------------------------------------------------------------- step

template <typename T>
__global__ void __launch_bounds__(256) scan_step_kernel(int C, int parts, ScanTensor x, ScanTensor gate, const float *gate_bias,
                                                        float *pool, int n_states, const int *slots, ScanTensor y) {
    const int b = blockIdx.x / parts, c = (blockIdx.x - b * parts) * 256 + threadIdx.x;
    if (c >= C) return;
    const int slot = slots != nullptr ? slots[b] : b;
    float h = 0.f;
    if (slot >= 0 && slot < n_states) {
        float *s = pool + (long long)slot * C + c;
        const Gate q = gate_of(to_f32(static_cast<const T *>(gate.p)[b * gate.row + c]) + gate_bias[c]);
        h = fmaf(q.a, *s, q.b * to_f32(static_cast<const T *>(x.p)[b * x.row + c]));
        *s = h;
    }
    static_cast<T *>(y.p)[b * y.row + c] = from_f32<T>(h);
}

}  // namespace

size_t scan_tokens_workspace(int op, const ScanArgs &a) {
    const int V = a.dtype == WTCONV_F32 ? 1 : 2;
    const bool back = op == WTCONV_SCAN_OP_BACKWARD;
    const TokenPlan p = plan_of(a, V, back ? kBackwardPerSm : kForwardPerSm);
    return map_bytes(a, p, V) + (back ? part_bytes(a, p, V) : 0);
}

cudaError_t launch_scan_tokens_forward(const ScanArgs &a, cudaStream_t st) {
    const Access w = access_of(a, {&a.x, &a.gate}, {&a.y});
    if (a.dtype == WTCONV_F32) return w.copy == 16 ? forward_typed<float, 1, 16, true>(a, st) : forward_typed<float, 1, 4, true>(a, st);
    return a.dtype == WTCONV_BF16 ? forward_16<__nv_bfloat16>(a, w, st) : forward_16<__half>(a, w, st);
}

cudaError_t launch_scan_tokens_backward(const ScanArgs &a, cudaStream_t st) {
    const Access w = access_of(a, {&a.x, &a.gate, &a.dy}, {&a.dx, &a.d_gate});
    if (a.dtype == WTCONV_F32)
        return w.copy == 16 ? backward_typed<float, 1, 16, true>(a, st) : backward_typed<float, 1, 4, true>(a, st);
    return a.dtype == WTCONV_BF16 ? backward_16<__nv_bfloat16>(a, w, st) : backward_16<__half>(a, w, st);
}

cudaError_t launch_scan_step(int B, int C, int dtype, const ScanTensor &x, const ScanTensor &gate, const float *gate_bias,
                             float *pool, int n_states, const int *slots, const ScanTensor &y, cudaStream_t st) {
    const int parts = (C + 255) / 256;
    const unsigned grid = (unsigned)B * parts;
    if (dtype == WTCONV_F32) scan_step_kernel<float><<<grid, 256, 0, st>>>(C, parts, x, gate, gate_bias, pool, n_states, slots, y);
    else if (dtype == WTCONV_BF16)
        scan_step_kernel<__nv_bfloat16><<<grid, 256, 0, st>>>(C, parts, x, gate, gate_bias, pool, n_states, slots, y);
    else scan_step_kernel<__half><<<grid, 256, 0, st>>>(C, parts, x, gate, gate_bias, pool, n_states, slots, y);
    return cudaGetLastError();
}

}  // namespace wtconv
