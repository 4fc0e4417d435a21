// Gated scan of tokens [B][T][C] (channels contiguous): one CTA per strip of channels of a sequence,
// or a cluster of CTAs along its time.
//
// A strip is 128 bytes of every row (32 where there are few channels), a round 64 positions of it,
// brought into shared memory by asynchronous copies two rounds ahead.  A thread owns two neighbouring channels (packed fp32
// arithmetic: one instruction for both) and eight consecutive positions, which it reduces to the map
// h -> a h + u of the state before them; the threads of a position group (a slot: a warp of 16-bit
// strips, half a warp of fp32 ones) cover the strip.  The slots leave their maps in shared memory, one
// of them runs the state through all eight and leaves each slot's start, and every thread runs its
// eight positions again from there, out of registers: x, gate and (backward) dy are read once.  (With
// every slot folding the maps before its own, that fold was half of all instructions.)
//
// A strip of a sequence is a chain along time.  Where there are too few of them to fill the GPU, R
// CTAs of a cluster share one: in a round CTA r takes the r-th 64 positions and pushes its map into the
// shared memory of all, where it counts towards an mbarrier; when that has all of a round's maps, each
// CTA folds those before its own.  (A cluster barrier instead waits for every thread of every CTA, and
// its release for the outputs of the round before: 8x4096x1024 bf16 forward 61 us, 54 so.)  Where even
// that leaves most SMs idle, the sequence is cut into segments whose maps a first kernel reduces
// (reading two inputs twice, the second time mostly from L2).
//
// Bound by the latency of a round's exchange and, after it, by the issue of instructions (25 an element
// forward, 34 backward): the four (backward two) CTAs that fit an SM overlap their rounds only so far.
// Alone, with cold caches: 8x4096x1024 bf16 forward 55 us and backward 88 us (3.7 and 3.8 TB/s, 55 and 57 %
// of a copy), fp32 85 and 136 us (71 and 74 %).  32x2048x768 bf16 forward of ragged sequences that fill 48 %
// of their rows 59 us: 3.4 TB/s of what is read and written, half of a copy.
#include <cooperative_groups.h>

#include <initializer_list>

#include "scan_device.cuh"

namespace wtconv {

namespace {

namespace cg = cooperative_groups;

constexpr int kSlots = 8, kSteps = 8;
constexpr int kSpan = kSlots * kSteps;  // positions of a CTA's round
static_assert(kSpan == WTCONV_SCAN_KEEP, "a round starts at a kept state");
constexpr int kMaxCluster = 8;
// R: bytes of a strip's rows, 128, or 32 where few channels would leave most of such a strip empty.

enum Mode { kReduce, kApply };

// CTAs that an SM is to hold
template <int R> constexpr int kForwardPerSm = 4 * 128 / R;
template <int R> constexpr int kBackwardPerSm = 2 * 128 / R;

template <typename T, int R> constexpr int kWidth = R / (int)sizeof(T);  // channels of a strip
template <typename T, int R> constexpr int kLanes = kWidth<T, R> / 2;    // threads of a slot
template <typename T, int R> constexpr int kThreads = kSlots * kLanes<T, R>;

// Two channels of one position as they lie in memory, and as fp32.
template <typename T> struct Two {
    uint32_t w;
    __device__ __forceinline__ Pair wide() const { return widen<T>(w); }
};
template <> struct Two<float> {
    Pair v;
    __device__ __forceinline__ Pair wide() const { return v; }
};

// kSpan positions of a strip of one tensor.
template <typename T, int CP, int R> struct Tile {
    T v[kSpan][kWidth<T, R>];
    __device__ __forceinline__ Two<T> raw(int r, int lane) const {
        if constexpr (sizeof(T) == 4) {
            const float2 f = *reinterpret_cast<const float2 *>(&v[r][lane * 2]);
            return {Pair(f.x, f.y)};
        } else {
            return {*reinterpret_cast<const uint32_t *>(&v[r][lane * 2])};
        }
    }
};
// The same where rows start at any 16-bit element: whole words are copied, from the one that holds a
// row's first channel on, so that the channels of a row lie one element further where its address is
// not a multiple of 4.  `first` is that offset in row 0, `step` (0 or 1) whether it alternates.
template <typename T, int R> struct Tile<T, 2, R> {
    static constexpr int words = kWidth<T, R> / 2 + 1;
    uint32_t w[kSpan][words];
    int first, step;
    __device__ __forceinline__ Two<T> raw(int r, int lane) const {
        const uint16_t *h = reinterpret_cast<const uint16_t *>(w[r]) + ((first + r * step) & 1) + lane * 2;
        return {(uint32_t)h[0] | (uint32_t)h[1] << 16};
    }
};

// A thread's share of the copies of one tensor's tiles, CP bytes each: column `c` of every
// `rows_at_once`-th row.  What is past the length or the last channel reads as zeros and is not touched.
template <typename T, int CP, int R> struct Loader {
    static constexpr int per_row = R / CP, elems = CP / (int)sizeof(T), rows_at_once = kThreads<T, R> / per_row;
    static_assert(kThreads<T, R> % per_row == 0 && kSpan % rows_at_once == 0, "");
    const T *p, *anchor;  // the thread's element of the next tile; an address that stands in where nothing is read
    long long round, stride;
    // from: the strip's first channel at the CTA's first position; round: elements between its tiles
    __device__ __forceinline__ Loader(const T *base, const T *from, long long row, long long round_)
        : p(from + (threadIdx.x / per_row) * row + (threadIdx.x % per_row) * elems), anchor(base), round(round_),
          stride(rows_at_once * row) {}
    // rows: valid positions of the tile; width: valid channels of the strip
    __device__ __forceinline__ void next(Tile<T, CP, R> &tile, int rows, int width) {
        const int r0 = threadIdx.x / per_row, c = (threadIdx.x % per_row) * elems, left = width - c;
        const int bytes = left <= 0 ? 0 : left >= elems ? CP : left * (int)sizeof(T);
        T *to = &tile.v[r0][c];
        const T *from = p;
#pragma unroll
        for (int k = 0; k < kSpan; k += rows_at_once, from += stride) {
            const bool valid = r0 + k < rows && bytes > 0;
            copy_async<CP>(to + k * kWidth<T, R>, valid ? from : anchor, valid ? bytes : 0);
        }
        p += round;
    }
};
template <typename T, int R> struct Loader<T, 2, R> {
    // A thread copies word k of every eighth row, whose offset is the same in all of them, and the first
    // 64 threads the last word of one row each.
    static constexpr int per_row = kWidth<T, R> / 2, rows_at_once = kThreads<T, R> / per_row;
    static_assert(rows_at_once % 2 == 0 && kSpan <= kThreads<T, R>, "");
    const T *p, *anchor;  // the strip's first channel of the next tile's first row; the tensor's first element
    long long round, row;
    int first, step;
    __device__ __forceinline__ Loader(const T *base, const T *from, long long row_, long long round_)
        : p(from), anchor(base), round(round_), row(row_), first((int)(reinterpret_cast<uintptr_t>(from) >> 1 & 1)),
          step((int)(row_ & 1)) {}
    __device__ __forceinline__ void next(Tile<T, 2, R> &tile, int rows, int width) {
        if (threadIdx.x == 0) tile.first = first, tile.step = step;
        const void *none = reinterpret_cast<const void *>(reinterpret_cast<uintptr_t>(anchor) + 2 & ~(uintptr_t)3);
        const int have = min(width, kWidth<T, R>);
        {
            const int r0 = threadIdx.x / per_row, k = threadIdx.x % per_row;
            const int c = 2 * k - ((first + r0 * step) & 1);  // the word's first channel; -1: the element before the strip
            const int bytes = min(max(have - c, 0), 2) * 2;
            const T *from = p + r0 * row + c;
            uint32_t *to = &tile.w[r0][k];
#pragma unroll
            for (int j = 0; j < kSpan; j += rows_at_once, from += rows_at_once * row) {
                const bool valid = r0 + j < rows && bytes > 0;
                // Before the tensor: its first element alone.  (A row stride of 0 has more rows there, which read the
                // whole word that holds that element: it is aligned, so all of it is memory of the same allocation,
                // and the other half is dropped.  With the test in every row odd rows took 20 to 40 % longer.)
                if (j == 0 && from < anchor) {
                    *to = valid ? (uint32_t)*reinterpret_cast<const uint16_t *>(from + 1) << 16 : 0u;
                } else {
                    copy_async<4>(to + j * Tile<T, 2, R>::words, valid ? from : none, valid ? bytes : 0);
                }
            }
        }
        if (threadIdx.x < kSpan) {
            const int r = threadIdx.x, c = kWidth<T, R> - ((first + r * step) & 1);
            const bool valid = r < rows && c < have;
            copy_async<4>(&tile.w[r][per_row], valid ? p + r * row + c : none, valid ? 2 : 0);
        }
        p += round;
    }
};

// Two channels of one row.  PAIRED: the address allows one store of both.
template <typename T, bool PAIRED> __device__ __forceinline__ void store_two(T *p, Pair v, int width) {
    if constexpr (sizeof(T) == 4) {
        if (PAIRED && width > 1) *reinterpret_cast<float2 *>(p) = make_float2(v.lo(), v.hi());
        else {
            if (width > 0) p[0] = v.lo();
            if (width > 1) p[1] = v.hi();
        }
    } else {
        const uint32_t w = narrow<T>(v);
        if (PAIRED && width > 1) *reinterpret_cast<uint32_t *>(p) = w;
        else {
            if (width > 0) *reinterpret_cast<uint16_t *>(p) = (uint16_t)w;
            if (width > 1) *reinterpret_cast<uint16_t *>(p + 1) = (uint16_t)(w >> 16);
        }
    }
}
template <typename T> __device__ __forceinline__ void store_pair(T *p, Pair v) {
    if constexpr (sizeof(T) == 4) *reinterpret_cast<float2 *>(p) = make_float2(v.lo(), v.hi());
    else *reinterpret_cast<uint32_t *>(p) = narrow<T>(v);
}
__device__ __forceinline__ Pair load_two(const float *p, int width) {
    return {width > 0 ? p[0] : 0.f, width > 1 ? p[1] : 0.f};
}
__device__ __forceinline__ void store_state(float *p, Pair v, int width) {
    if (width > 0) p[0] = v.lo();
    if (width > 1) p[1] = v.hi();
}

struct TokenPlan {
    int strips, cluster, segments, rounds_per;  // rounds_per: rounds of the cluster in a segment
};

// A stretch of two channels as the map h -> a h + u of the state before it; `then` appends the
// stretch that follows.
struct Map {
    Pair a, u;
    __device__ __forceinline__ Map then(const Map &next) const { return {mul(a, next.a), fma(next.a, u, next.u)}; }
    __device__ __forceinline__ Pair of(Pair h) const { return fma(a, h, u); }
};
__device__ __forceinline__ Map identity() { return {Pair(1.f), Pair(0.f)}; }
__device__ __forceinline__ Map load_map(const ulonglong2 *p) {
    Map m;
    const ulonglong2 q = *p;
    m.a.q = q.x, m.u.q = q.y;
    return m;
}
__device__ __forceinline__ void store_map(ulonglong2 *p, const Map &m) { *p = make_ulonglong2(m.a.q, m.u.q); }

template <typename T, int R> struct Maps {
    ulonglong2 slot[kSlots][kLanes<T, R>];          // a round's maps,
    unsigned long long start[kSlots][kLanes<T, R>];  // and the state that reaches each slot
    ulonglong2 cta[2][kMaxCluster][kLanes<T, R>];   // the CTAs' maps of a round and the next,
    unsigned long long arrived[2];               // and the mbarriers that count their bytes
};

// ------------------------------------------------------------- maps of the CTAs of a cluster

// Raised by a wait that gave up (never expected); read by wtconv_scan_status.
__device__ int g_scan_timeout;

constexpr unsigned kMaxTries = 1u << 20, kWaitHintNs = 20000;
constexpr unsigned long long kMaxWaitNs = 500000000ull;

__device__ __forceinline__ unsigned shared_address(const void *p) { return (unsigned)__cvta_generic_to_shared(p); }
__device__ __forceinline__ unsigned remote_address(unsigned local, int rank) {
    unsigned r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(local), "r"(rank));
    return r;
}
__device__ __forceinline__ unsigned long long global_ns() {
    unsigned long long t;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
    return t;
}
// Waits at most half a second for a phase of an mbarrier; false (and the flag) if it did not come.
__device__ __forceinline__ bool wait_phase(unsigned bar, unsigned parity) {
    unsigned long long t0 = 0;
    for (unsigned i = 0; i < kMaxTries; ++i) {
        unsigned done;
        asm volatile("{\n\t.reg .pred p;\n\t"
                     "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2, %3;\n\t"
                     "selp.u32 %0, 1, 0, p;\n\t}"
                     : "=r"(done) : "r"(bar), "r"(parity), "n"(kWaitHintNs) : "memory");
        if (done) return true;
        if ((i & 15) == 0) {
            const unsigned long long now = global_ns();
            if (i == 0) t0 = now;
            else if (now - t0 > kMaxWaitNs) break;
        }
    }
    atomicExch(&g_scan_timeout, 1);
    return false;
}

// What the leading slot's threads carry from round to round.
struct Chain {
    Pair state;           // before the round of the whole cluster
    unsigned phases = 0;  // bit b: phase that arrived[b] completes next
    bool broken = false;  // a wait gave up: the rest comes out as NaN
};

// Runs carry (the state before the round) through the round: start[] of every slot, and carry after
// the whole cluster's round.  By the kLanes threads of one slot, between two barriers; `lane` is the
// thread's place among them.  BACKWARD: the last slot and CTA come first.
template <typename T, int R, bool BACKWARD>
__device__ __forceinline__ void run_chain(Maps<T, R> &sh, int lane, Pair &carry) {
#pragma unroll
    for (int i = 0; i < kSlots; ++i) {
        const int slot = BACKWARD ? kSlots - 1 - i : i;
        sh.start[slot][lane] = carry.q;
        carry = load_map(&sh.slot[slot][lane]).of(carry);
    }
}
// The CTA's map to every CTA of the cluster, then the state through the maps of all.
//
// Two buffers are enough: a CTA pushes the maps of round k + 2 after it has those of round k + 1 from
// all, and each of them pushed those after it had read the maps of round k.  A thread that gave up takes
// no further part (its bytes would count towards a phase that is not over, and an arrival would be one
// too many), so the others give up in the same round or the next: all of a strip's later results are NaN.
template <typename T, int R, bool BACKWARD>
__device__ __forceinline__ void run_cluster(Maps<T, R> &sh, int lane, int parity, int cluster, int rank, Chain &chain) {
    Map all = load_map(&sh.slot[BACKWARD ? kSlots - 1 : 0][lane]);
#pragma unroll
    for (int i = 1; i < kSlots; ++i) all = all.then(load_map(&sh.slot[BACKWARD ? kSlots - 1 - i : i][lane]));
    if (!chain.broken) {
        const unsigned bar = shared_address(&sh.arrived[parity]), place = shared_address(&sh.cta[parity][rank][lane]);
        if (lane == 0)
            asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(cluster * kLanes<T, R> * 16) : "memory");
        for (int r = 0; r < cluster; ++r)
            asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.b32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(
                             remote_address(place, r)),
                         "r"((unsigned)all.a.q), "r"((unsigned)(all.a.q >> 32)), "r"((unsigned)all.u.q),
                         "r"((unsigned)(all.u.q >> 32)), "r"(remote_address(bar, r)) : "memory");
        chain.broken = !wait_phase(bar, chain.phases >> parity & 1);
        chain.phases ^= 1u << parity;
    }
    if (chain.broken) chain.state = Pair(__int_as_float(0x7fc00000));
    Pair mine = chain.state;
    for (int i = 0; i < cluster; ++i) {
        const int r = BACKWARD ? cluster - 1 - i : i;
        if (r == rank) mine = chain.state;
        chain.state = load_map(&sh.cta[parity][r][lane]).of(chain.state);
    }
    run_chain<T, R, BACKWARD>(sh, lane, mine);
}
// Last of all in a kernel with clusters.  Where every wait ended well, every push to this CTA has arrived.
// After one that gave up pushes may still be under way: the thread keeps the CTA, and so its shared
// memory, until all other threads of the cluster have come here too or have exited.
__device__ __forceinline__ void leave_cluster(const Chain &chain) {
    if (chain.broken)
        asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}
// One round's exchange: from the maps in sh.slot to the states in sh.start.  Threads below kLanes hold
// the chain.  `beside`: work of another slot's threads, between the barriers.
template <typename T, int R, bool BACKWARD, typename F>
__device__ __forceinline__ void exchange(Maps<T, R> &sh, int parity, int cluster, int rank, Chain &chain, F beside) {
    __syncthreads();
    if (threadIdx.x < kLanes<T, R>) {
        if (cluster == 1) run_chain<T, R, BACKWARD>(sh, threadIdx.x, chain.state);
        else run_cluster<T, R, BACKWARD>(sh, threadIdx.x, parity, cluster, rank, chain);
    } else {
        beside();
    }
    __syncthreads();
}
// Before the first round: the cluster's mbarriers are ready, and every CTA's shared memory is there.
template <typename T, int R> __device__ __forceinline__ void start_cluster(Maps<T, R> &sh) {
    if (threadIdx.x == 0) {
        for (int b = 0; b < 2; ++b) asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(shared_address(&sh.arrived[b])) : "memory");
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    cg::this_cluster().sync();
}

// A round of a segment's reduction: the leading slot appends the round's maps to whole.
template <typename T, int R, bool BACKWARD> __device__ __forceinline__ void reduce_round(Maps<T, R> &sh, Map &whole) {
    __syncthreads();
    if (threadIdx.x < kLanes<T, R>) {
#pragma unroll
        for (int i = 0; i < kSlots; ++i) whole = whole.then(load_map(&sh.slot[BACKWARD ? kSlots - 1 - i : i][threadIdx.x]));
    }
    __syncthreads();
}

// State that the segments before (after, if BACKWARD) this one leave, from chain (of the leading
// slot): their maps are folded by the slots in parallel, then as in a round.
template <typename T, int R, bool BACKWARD>
__device__ __forceinline__ void fold_segments(const ulonglong2 *maps, int first, int last, Maps<T, R> &sh, int slot, int lane,
                                              Chain &chain) {
    const int count = last - first, per = (count + kSlots - 1) / kSlots;
    Map mine = identity();
    const int place = BACKWARD ? kSlots - 1 - slot : slot;
    for (int i = place * per; i < min((place + 1) * per, count); ++i)
        mine = mine.then(load_map(maps + (long long)(BACKWARD ? last - 1 - i : first + i) * kLanes<T, R> + lane));
    store_map(&sh.slot[slot][lane], mine);
    exchange<T, R, BACKWARD>(sh, 0, 1, 0, chain, [] {});
}

struct Place {
    int b, seg, rank, n, c0, c;  // first channel of the strip and of the thread
    int width;                   // channels that the thread has (2, fewer at the end, or <= 0)
    long long unit;              // (b * strips + strip) * segments
};
template <typename T, int R> __device__ __forceinline__ Place place_of(const ScanArgs &a, const TokenPlan &p, int lane) {
    Place s;
    s.rank = blockIdx.x % p.cluster;
    unsigned i = blockIdx.x / p.cluster;
    s.seg = i % p.segments;
    i /= p.segments;
    s.unit = (long long)i * p.segments;
    const int strip = i % p.strips;
    s.b = i / p.strips;
    s.c0 = strip * kWidth<T, R>;
    s.c = s.c0 + lane * 2;
    s.width = a.C - s.c;
    s.n = scan_length(a.lengths, s.b, a.T);
    return s;
}

// Gates of a thread's positions; those at or past `live` hold the state (a = 1, b = 0).
template <typename T, int CP, int R>
__device__ __forceinline__ void read_gates(const Tile<T, CP, R> &tile, int slot, int lane, Pair bias, int live, Pair (&av)[kSteps],
                                           Pair (&bv)[kSteps]) {
#pragma unroll
    for (int j = 0; j < kSteps; ++j) {
        const Gates q = gates_of(tile.raw(slot * kSteps + j, lane).wide(), bias);
        av[j] = q.a, bv[j] = q.b;
    }
    if (live < kSteps) {
#pragma unroll
        for (int j = 0; j < kSteps; ++j)
            if (j >= live) av[j] = Pair(1.f), bv[j] = Pair(0.f);
    }
}

// ---------------------------------------------------------------------------------------- forward

template <typename T, int CP, int R> struct ForwardShared {
    Tile<T, CP, R> x[2], g[2];
    Maps<T, R> maps;
};

// CP: bytes of a copy; PAIRED: the outputs' rows allow stores of two channels
template <typename T, int CP, int R, bool PAIRED, Mode MODE>
__global__ void __launch_bounds__(kThreads<T, R>, kForwardPerSm<R>) scan_tokens_forward_kernel(const ScanArgs a, const TokenPlan p, ulonglong2 *maps) {
    extern __shared__ __align__(16) unsigned char raw[];
    begin_kernel();
    ForwardShared<T, CP, R> &sh = *reinterpret_cast<ForwardShared<T, CP, R> *>(raw);
    const int lane = threadIdx.x % kLanes<T, R>, slot = threadIdx.x / kLanes<T, R>;
    const Place s = place_of<T, R>(a, p, lane);
    const int round_span = p.cluster * kSpan, rounds = (a.T + round_span - 1) / round_span;
    const int round0 = s.seg * p.rounds_per, round1 = min(round0 + p.rounds_per, rounds);
    int t0 = round0 * round_span + s.rank * kSpan;  // the CTA's first position of the round
    Loader<T, CP, R> x(static_cast<const T *>(a.x.p), static_cast<const T *>(a.x.p) + s.b * a.x.batch + s.c0 + t0 * a.x.row, a.x.row, round_span * a.x.row);
    Loader<T, CP, R> g(static_cast<const T *>(a.gate.p), static_cast<const T *>(a.gate.p) + s.b * a.gate.batch + s.c0 + t0 * a.gate.row, a.gate.row,
                    round_span * a.gate.row);
    T *y = static_cast<T *>(a.y.p) + s.b * a.y.batch + s.c + (t0 + slot * kSteps) * a.y.row;
    const long long y_round = round_span * a.y.row;
    const bool whole_strip = PAIRED && a.C - s.c0 >= kWidth<T, R>;
    int ahead = t0;  // first position of the next tiles to fetch
    const auto fetch = [&](int buf) {
        x.next(sh.x[buf], s.n - ahead, a.C - s.c0);
        g.next(sh.g[buf], s.n - ahead, a.C - s.c0);
        commit_copies();
        ahead += round_span;
    };
    fetch(round0 & 1);
    if (round0 + 1 < round1) fetch((round0 + 1) & 1);
    else commit_copies();

    const Pair bias = load_two(a.gate_bias + s.c, s.width);
    Chain chain;
    chain.state = Pair(0.f);
    Map whole = identity();
    if constexpr (MODE == kApply) {
        if (a.h0 != nullptr) chain.state = load_two(a.h0 + (long long)s.b * a.C + s.c, s.width);
        if (s.seg > 0) fold_segments<T, R, false>(maps + s.unit * kLanes<T, R>, 0, s.seg, sh.maps, slot, lane, chain);
    }
    wait_copies<1>();
    if (p.cluster > 1) start_cluster(sh.maps);
    else __syncthreads();
    // rounds of the whole cluster up to the length; what is left after it is filled below
    const int live1 = min(round1, (s.n + round_span - 1) / round_span);
    for (int round = round0; round < live1; ++round) {
        const int t = t0 + slot * kSteps;
        Pair av[kSteps], uv[kSteps];
        Map mine = identity();
        read_gates(sh.g[round & 1], slot, lane, bias, s.n - t, av, uv);
#pragma unroll
        for (int j = 0; j < kSteps; ++j) {
            uv[j] = mul(uv[j], sh.x[round & 1].raw(slot * kSteps + j, lane).wide());  // (x is 0 beyond the length)
            mine = mine.then({av[j], uv[j]});
        }
        store_map(&sh.maps.slot[slot][lane], mine);
        // the exchange's barriers end all reading of a round's tiles and show the next's
        wait_copies<0>();
        if constexpr (MODE == kReduce) {
            reduce_round<T, R, false>(sh.maps, whole);
            if (round + 2 < live1) fetch(round & 1);
        } else {
            exchange<T, R, false>(sh.maps, round & 1, p.cluster, s.rank, chain, [] {});
            if (round + 2 < live1) fetch(round & 1);
            Pair h;
            h.q = sh.maps.start[slot][lane];
            if (a.states_out != nullptr && slot == 0 && t0 < a.T)
                store_state(a.states_out + ((long long)s.b * a.keep + t0 / WTCONV_SCAN_KEEP) * a.C + s.c, h, s.width);
            T *to = y;
            if (whole_strip && t + kSteps <= s.n) {
#pragma unroll
                for (int j = 0; j < kSteps; ++j, to += a.y.row) {
                    h = fma(av[j], h, uv[j]);
                    store_pair(to, h);
                }
            } else {
#pragma unroll
                for (int j = 0; j < kSteps; ++j, to += a.y.row) {
                    h = fma(av[j], h, uv[j]);
                    if (t + j < a.T) store_two<T, PAIRED>(to, t + j < s.n ? h : Pair(0.f), s.width);
                }
            }
            y += y_round;
        }
        t0 += round_span;
    }
    if constexpr (MODE == kApply) {  // past the length the state stands still, and y is 0
        for (int round = max(live1, round0); round < round1; ++round, t0 += round_span, y += y_round) {
            if (a.states_out != nullptr && slot == 0 && t0 < a.T)
                store_state(a.states_out + ((long long)s.b * a.keep + t0 / WTCONV_SCAN_KEEP) * a.C + s.c, chain.state, s.width);
            T *to = y;
            for (int j = 0; j < kSteps; ++j, to += a.y.row)
                if (t0 + slot * kSteps + j < a.T) store_two<T, PAIRED>(to, Pair(0.f), s.width);
        }
    }
    if constexpr (MODE == kReduce) {
        if (slot == 0) store_map(maps + (s.unit + s.seg) * kLanes<T, R> + lane, whole);
    } else if (a.h_last != nullptr && s.seg == p.segments - 1 && s.rank == 0 && slot == 0) {
        store_state(a.h_last + (long long)s.b * a.C + s.c, chain.state, s.width);
    }
    leave_cluster(chain);
}

// --------------------------------------------------------------------------------------- backward

template <typename T, int CP, int R> struct BackwardShared {
    Tile<T, CP, R> x[2], g[2], dy[2];
    Maps<T, R> maps;
    // h within the CTA's positions, from the kept state: as slot and start of Maps
    ulonglong2 forward[kSlots][kLanes<T, R>];
    unsigned long long forward_start[kSlots][kLanes<T, R>];
};

// bias_part: one float per (unit, segment, rank, channel of the strip)
template <typename T, int CP, int R, bool PAIRED, Mode MODE>
__global__ void __launch_bounds__(kThreads<T, R>, sizeof(T) == 4 ? kBackwardPerSm<R> * 3 / 2 : kBackwardPerSm<R>)
    scan_tokens_backward_kernel(const ScanArgs a, const TokenPlan p, ulonglong2 *maps, float *bias_part) {
    extern __shared__ __align__(16) unsigned char raw[];
    begin_kernel();
    BackwardShared<T, CP, R> &sh = *reinterpret_cast<BackwardShared<T, CP, R> *>(raw);
    const int lane = threadIdx.x % kLanes<T, R>, slot = threadIdx.x / kLanes<T, R>;
    const Place s = place_of<T, R>(a, p, lane);
    const int round_span = p.cluster * kSpan, rounds = (a.T + round_span - 1) / round_span;
    const int round0 = s.seg * p.rounds_per, round1 = min(round0 + p.rounds_per, rounds);
    // the rounds past the length come first: no gradient passes them, dx and d_gate are 0
    const int live1 = max(round0, min(round1, (s.n + round_span - 1) / round_span));
    int t0 = (live1 - 1) * round_span + s.rank * kSpan;
    Loader<T, CP, R> x(static_cast<const T *>(a.x.p), static_cast<const T *>(a.x.p) + s.b * a.x.batch + s.c0 + t0 * a.x.row, a.x.row, -round_span * a.x.row);
    Loader<T, CP, R> g(static_cast<const T *>(a.gate.p), static_cast<const T *>(a.gate.p) + s.b * a.gate.batch + s.c0 + t0 * a.gate.row, a.gate.row,
                    -round_span * a.gate.row);
    Loader<T, CP, R> dy(static_cast<const T *>(a.dy.p), static_cast<const T *>(a.dy.p) + s.b * a.dy.batch + s.c0 + t0 * a.dy.row, a.dy.row, -round_span * a.dy.row);
    T *dx = static_cast<T *>(a.dx.p) + s.b * a.dx.batch + s.c + (t0 + slot * kSteps + kSteps - 1) * a.dx.row;
    T *dg = static_cast<T *>(a.d_gate.p) + s.b * a.d_gate.batch + s.c + (t0 + slot * kSteps + kSteps - 1) * a.d_gate.row;
    const bool whole_strip = PAIRED && a.C - s.c0 >= kWidth<T, R>;
    int ahead = t0;  // first position of the next tiles to fetch, towards the beginning
    const auto fetch = [&](int buf) {
        g.next(sh.g[buf], s.n - ahead, a.C - s.c0);
        dy.next(sh.dy[buf], s.n - ahead, a.C - s.c0);
        if (MODE == kApply) x.next(sh.x[buf], s.n - ahead, a.C - s.c0);
        commit_copies();
        ahead -= round_span;
    };
    if (round0 < live1) fetch((live1 - 1) & 1);
    else commit_copies();
    if (round0 + 1 < live1) fetch(live1 & 1);
    else commit_copies();
    if constexpr (MODE == kApply) {
        for (int t = live1 * round_span + s.rank * kSpan + slot * kSteps, round = live1; round < round1; ++round, t += round_span)
            for (int j = 0; j < kSteps; ++j)
                if (t + j < a.T) {
                    store_two<T, PAIRED>(static_cast<T *>(a.dx.p) + s.b * a.dx.batch + (t + j) * a.dx.row + s.c, Pair(0.f), s.width);
                    store_two<T, PAIRED>(static_cast<T *>(a.d_gate.p) + s.b * a.d_gate.batch + (t + j) * a.d_gate.row + s.c, Pair(0.f),
                                         s.width);
                }
    }

    const Pair bias = load_two(a.gate_bias + s.c, s.width);
    Chain chain;
    chain.state = Pair(0.f);
    Pair sum(0.f), next_kept(0.f);
    Map whole = identity();
    const auto kept_state = [&](int at) {
        if (at < a.T)
            next_kept = load_two(a.states_in + ((long long)s.b * a.keep + at / WTCONV_SCAN_KEEP) * a.C + s.c, s.width);
    };
    // the slot that runs h: in another warp than the leading one, if there is one
    const bool runs_h = slot == (kThreads<T, R> > 32 ? 32 / kLanes<T, R> : 1);
    if constexpr (MODE == kApply) {
        if (round0 < live1 && runs_h) kept_state(t0);
        if (a.dh_last != nullptr) chain.state = load_two(a.dh_last + (long long)s.b * a.C + s.c, s.width);
        if (s.seg < p.segments - 1)
            fold_segments<T, R, true>(maps + s.unit * kLanes<T, R>, s.seg + 1, p.segments, sh.maps, slot, lane, chain);
    }
    wait_copies<1>();
    if (p.cluster > 1) start_cluster(sh.maps);
    else __syncthreads();
    for (int round = live1 - 1; round >= round0; --round) {
        const int t = t0 + slot * kSteps, live = s.n - t, buf = round & 1;
        Pair av[kSteps], bv[kSteps];
        Two<T> dyv[kSteps], xv[kSteps];  // kept as they lie: half the registers in 16 bits
        Map back = identity();
        read_gates(sh.g[buf], slot, lane, bias, live, av, bv);
#pragma unroll
        for (int j = kSteps - 1; j >= 0; --j) {
            dyv[j] = sh.dy[buf].raw(slot * kSteps + j, lane);  // (dy and x are 0 beyond the length)
            back.u = mul(av[j], add(dyv[j].wide(), back.u));
            back.a = mul(back.a, av[j]);
            if (MODE == kApply) xv[j] = sh.x[buf].raw(slot * kSteps + j, lane);
        }
        store_map(&sh.maps.slot[slot][lane], back);
        if constexpr (MODE == kReduce) {
            wait_copies<0>();
            reduce_round<T, R, true>(sh.maps, whole);
            if (round - 2 >= round0) fetch(buf);
        } else {
            // h is scanned forward within the CTA's positions from the kept state; dh comes backward
            Map fwd = {back.a, Pair(0.f)};
#pragma unroll
            for (int j = 0; j < kSteps; ++j) fwd.u = fma(av[j], fwd.u, mul(bv[j], xv[j].wide()));
            store_map(&sh.forward[slot][lane], fwd);
            wait_copies<0>();
            exchange<T, R, true>(sh.maps, buf, p.cluster, s.rank, chain, [&] {
                if (!runs_h) return;
                Pair h = next_kept;
#pragma unroll
                for (int i = 0; i < kSlots; i += 4) {
                    Map m[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) m[k] = load_map(&sh.forward[i + k][lane]);
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        sh.forward_start[i + k][lane] = h.q;
                        h = m[k].of(h);
                    }
                }
                if (round > round0) kept_state(t0 - round_span);
            });
            if (round - 2 >= round0) fetch(buf);
            Pair flow, h;
            flow.q = sh.maps.start[slot][lane];
            h.q = sh.forward_start[slot][lane];
            Pair diff[kSteps];  // h_{t-1} - x_t
#pragma unroll
            for (int j = 0; j < kSteps; ++j) {
                const Pair x_t = xv[j].wide();
                diff[j] = sub(h, x_t);
                h = fma(av[j], h, mul(bv[j], x_t));
            }
            T *to_x = dx, *to_g = dg;
            const auto positions = [&](auto store) {
#pragma unroll
                for (int j = kSteps - 1; j >= 0; --j, to_x -= a.dx.row, to_g -= a.d_gate.row) {
                    const Pair dh = add(dyv[j].wide(), flow);
                    const Pair dgv = mul(mul(dh, diff[j]), mul(av[j], bv[j]));
                    flow = mul(av[j], dh);
                    store(j, mul(bv[j], dh), dgv);
                }
            };
            if (whole_strip && live >= kSteps) {
                positions([&](int, Pair dxv, Pair dgv) {
                    sum = add(sum, dgv);
                    store_pair(to_x, dxv), store_pair(to_g, dgv);
                });
            } else {
                positions([&](int j, Pair dxv, Pair dgv) {
                    // zeros past the length (b is 0 there, but a state or dh that is not finite makes b dh NaN)
                    if (j >= live) dxv = dgv = Pair(0.f);
                    sum = add(sum, dgv);
                    if (t + j < a.T) store_two<T, PAIRED>(to_x, dxv, s.width), store_two<T, PAIRED>(to_g, dgv, s.width);
                });
            }
            dx -= round_span * a.dx.row, dg -= round_span * a.d_gate.row;
        }
        t0 -= round_span;
    }
    if constexpr (MODE == kReduce) {
        if (slot == 0) store_map(maps + (s.unit + s.seg) * kLanes<T, R> + lane, whole);
    } else {
        if (a.d_h0 != nullptr && s.seg == 0 && s.rank == 0 && slot == 0)
            store_state(a.d_h0 + (long long)s.b * a.C + s.c, chain.state, s.width);
        __syncthreads();
        Pair *sums = reinterpret_cast<Pair *>(sh.forward);
        sums[slot * kLanes<T, R> + lane] = sum;
        __syncthreads();
        if (slot == 0) {
            for (int i = 1; i < kSlots; ++i) sum = add(sum, sums[i * kLanes<T, R> + lane]);
            float *to = bias_part + ((s.unit + s.seg) * p.cluster + s.rank) * kWidth<T, R> + lane * 2;
            to[0] = sum.lo(), to[1] = sum.hi();
        }
    }
    leave_cluster(chain);
}

// d_gate_bias_c = sum of the parts over sequences, segments and ranks, in a fixed order.
__global__ void __launch_bounds__(256) scan_tokens_bias_kernel(const float *part, float *out, int B, int C, int strips,
                                                               int per_unit, int width) {
    __shared__ float sums[8][32];
    begin_kernel();
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

// Rows of 32 bytes where that takes at most two thirds of the lanes (104x40909x5 fp16 forward 634 us
// with 128, 271 with 32; 64x8192x24 and wider do as well with either).
int row_bytes(const ScanArgs &a) {
    const long long wide = 128 / elem_bytes_of(a.dtype), slim = wide / 4;
    return (a.C + slim - 1) / slim * slim * 3 <= (a.C + wide - 1) / wide * wide * 2 ? 32 : 128;
}

// Chains (strips of sequences) are shared by clusters as large as the CTAs that fit the GPU allow (one
// more doubling left a second, mostly idle wave: 8x4096x1024 bf16 forward 70 us against 67).  Where even
// full clusters make less than half of those, sequences are cut into segments: 1x10634x1158 fp16 forward,
// 19 chains, took 76 us in clusters and 52 in segments; 2x30730x303, 10 chains, forward + backward 561
// and 194.
TokenPlan plan_of(const ScanArgs &a, bool backward) {
    TokenPlan p;
    const int row = row_bytes(a), width = row / elem_bytes_of(a.dtype), per_sm = (backward ? 2 : 4) * 128 / row;
    p.strips = ceil_div(a.C, width);
    const long long chains = (long long)a.B * p.strips, want = (long long)per_sm * sm_count();
    const int rounds = (a.T + kSpan - 1) / kSpan;
    p.cluster = p.segments = 1;
    if (chains * kMaxCluster * 2 >= want || rounds <= kMaxCluster) {
        while (p.cluster < kMaxCluster && chains * p.cluster * 2 <= want && p.cluster < rounds) p.cluster *= 2;
    } else {
        p.segments = (int)((want + chains - 1) / chains);
        if (p.segments > rounds) p.segments = rounds;
    }
    const int cluster_rounds = (rounds + p.cluster - 1) / p.cluster;
    p.rounds_per = (cluster_rounds + p.segments - 1) / p.segments;
    p.segments = (cluster_rounds + p.rounds_per - 1) / p.rounds_per;
    return p;
}

size_t round256(size_t n) { return (n + 255) / 256 * 256; }
size_t map_bytes(const ScanArgs &a, const TokenPlan &p) {
    const size_t lanes = row_bytes(a) / elem_bytes_of(a.dtype) / 2;
    return p.segments > 1 ? round256((size_t)a.B * p.strips * p.segments * lanes * sizeof(ulonglong2)) : 0;
}
size_t part_bytes(const ScanArgs &a, const TokenPlan &p) {
    return round256((size_t)a.B * p.strips * p.segments * p.cluster * (row_bytes(a) / elem_bytes_of(a.dtype)) * sizeof(float));
}

template <typename... P, typename... A>
cudaError_t launch(void (*kernel)(P...), int threads, size_t shared, const ScanArgs &a, const TokenPlan &p, cudaStream_t st,
                   A... args) {
    const cudaError_t e = allow_shared(kernel, shared);
    if (e != cudaSuccess) return e;
    return launch_kernel(kernel, (unsigned)((long long)a.B * p.strips * p.segments * p.cluster), threads, shared, st, p.cluster, a, p,
                         args...);
}

// Whether every row of a tensor starts at a multiple of `bytes`.
bool rows_at(const ScanTensor &s, const ScanArgs &a, int bytes) {
    const int per = bytes / elem_bytes_of(a.dtype);
    return aligned_to(s.p, bytes) && (a.B == 1 || s.batch % per == 0) && (a.T == 1 || s.row % per == 0);
}

template <typename T, int CP, int R, bool PAIRED> cudaError_t forward_typed(const ScanArgs &a, cudaStream_t st) {
    const TokenPlan p = plan_of(a, false);
    const size_t shared = sizeof(ForwardShared<T, CP, R>);
    ulonglong2 *maps = static_cast<ulonglong2 *>(a.workspace);
    if (p.segments > 1) {
        const cudaError_t e = launch(scan_tokens_forward_kernel<T, CP, R, PAIRED, kReduce>, kThreads<T, R>, shared, a, p, st, maps);
        if (e != cudaSuccess) return e;
    }
    return launch(scan_tokens_forward_kernel<T, CP, R, PAIRED, kApply>, kThreads<T, R>, shared, a, p, st, maps);
}

template <typename T, int CP, int R, bool PAIRED> cudaError_t backward_typed(const ScanArgs &a, cudaStream_t st) {
    const TokenPlan p = plan_of(a, true);
    const size_t shared = sizeof(BackwardShared<T, CP, R>);
    ulonglong2 *maps = static_cast<ulonglong2 *>(a.workspace);
    float *part = reinterpret_cast<float *>(static_cast<char *>(a.workspace) + map_bytes(a, p));
    cudaError_t e = cudaSuccess;
    if (p.segments > 1) e = launch(scan_tokens_backward_kernel<T, CP, R, PAIRED, kReduce>, kThreads<T, R>, shared, a, p, st, maps, part);
    if (e == cudaSuccess) e = launch(scan_tokens_backward_kernel<T, CP, R, PAIRED, kApply>, kThreads<T, R>, shared, a, p, st, maps, part);
    if (e != cudaSuccess) return e;
    return launch_kernel(scan_tokens_bias_kernel, ceil_div(a.C, 32), 256, 0, st, 1, part, a.d_gate_bias, a.B, a.C, p.strips,
                         p.segments * p.cluster, kWidth<T, R>);
}

// How wide rows can be copied in, and whether outputs can be stored two channels at a time.  The
// narrow combinations share one kernel.
template <typename T, typename F16, typename F4, typename FS>
cudaError_t by_access(const ScanArgs &a, std::initializer_list<const ScanTensor *> in,
                      std::initializer_list<const ScanTensor *> out, F16 wide, F4 words, FS single) {
    int copy = 16;
    bool paired = true;
    for (const ScanTensor *s : in)
        while (!rows_at(*s, a, copy)) copy = copy == 16 ? 4 : 2;
    for (const ScanTensor *s : out) paired = paired && rows_at(*s, a, 2 * (int)sizeof(T));
    if (copy == 16 && paired) return wide();
    if (copy >= 4 && paired) return words();
    return single();
}
template <typename T> constexpr int kNarrowest = sizeof(T) == 4 ? 4 : 2;

template <typename T, int R> cudaError_t forward_rows(const ScanArgs &a, cudaStream_t st) {
    return by_access<T>(a, {&a.x, &a.gate}, {&a.y}, [&] { return forward_typed<T, 16, R, true>(a, st); },
                        [&] { return forward_typed<T, 4, R, true>(a, st); },
                        [&] { return forward_typed<T, kNarrowest<T>, R, false>(a, st); });
}
template <typename T, int R> cudaError_t backward_rows(const ScanArgs &a, cudaStream_t st) {
    return by_access<T>(a, {&a.x, &a.gate, &a.dy}, {&a.dx, &a.d_gate}, [&] { return backward_typed<T, 16, R, true>(a, st); },
                        [&] { return backward_typed<T, 4, R, true>(a, st); },
                        [&] { return backward_typed<T, kNarrowest<T>, R, false>(a, st); });
}
template <typename T> cudaError_t forward_any(const ScanArgs &a, cudaStream_t st) {
    return row_bytes(a) == 32 ? forward_rows<T, 32>(a, st) : forward_rows<T, 128>(a, st);
}
template <typename T> cudaError_t backward_any(const ScanArgs &a, cudaStream_t st) {
    return row_bytes(a) == 32 ? backward_rows<T, 32>(a, st) : backward_rows<T, 128>(a, st);
}

// Diagnostic: a wait for an arrival that never comes.
__global__ void __launch_bounds__(32) scan_wait_selftest_kernel() {
    __shared__ unsigned long long bar;
    begin_kernel();
    if (threadIdx.x != 0) return;
    asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(shared_address(&bar)) : "memory");
    wait_phase(shared_address(&bar), 0);
}

// ------------------------------------------------------------------------------------------- step

template <typename T>
__global__ void __launch_bounds__(256) scan_step_kernel(int C, int parts, ScanTensor x, ScanTensor gate, const float *gate_bias,
                                                        float *pool, int n_states, const int *slots, ScanTensor y) {
    begin_kernel();
    const int b = blockIdx.x / parts, c = (blockIdx.x - b * parts) * 256 + threadIdx.x;
    if (c >= C) return;
    const int slot = slots != nullptr ? slots[b] : b;
    float h = 0.f;
    if (slot >= 0 && slot < n_states) {
        float *s = pool + (long long)slot * C + c;
        const Gates q = gates_of(Pair(to_f32(static_cast<const T *>(gate.p)[b * gate.row + c])), Pair(gate_bias[c]));
        h = fmaf(q.a.lo(), *s, q.b.lo() * to_f32(static_cast<const T *>(x.p)[b * x.row + c]));
        *s = h;
    }
    static_cast<T *>(y.p)[b * y.row + c] = from_f32<T>(h);
}

}  // namespace

cudaError_t take_scan_timeout(int *raised) {
    const cudaError_t e = cudaMemcpyFromSymbol(raised, g_scan_timeout, sizeof(int));
    const int zero = 0;
    return e != cudaSuccess || *raised == 0 ? e : cudaMemcpyToSymbol(g_scan_timeout, &zero, sizeof(int));
}

cudaError_t launch_scan_wait_selftest(cudaStream_t st) { return launch_kernel(scan_wait_selftest_kernel, 1, 32, 0, st, 1); }

size_t scan_tokens_workspace(int op, const ScanArgs &a) {
    const bool back = op == WTCONV_SCAN_OP_BACKWARD;
    const TokenPlan p = plan_of(a, back);
    return map_bytes(a, p) + (back ? part_bytes(a, p) : 0);
}

cudaError_t launch_scan_tokens_forward(const ScanArgs &a, cudaStream_t st) {
    if (a.dtype == WTCONV_F32) return forward_any<float>(a, st);
    return a.dtype == WTCONV_BF16 ? forward_any<__nv_bfloat16>(a, st) : forward_any<__half>(a, st);
}

cudaError_t launch_scan_tokens_backward(const ScanArgs &a, cudaStream_t st) {
    if (a.dtype == WTCONV_F32) return backward_any<float>(a, st);
    return a.dtype == WTCONV_BF16 ? backward_any<__nv_bfloat16>(a, st) : backward_any<__half>(a, st);
}

cudaError_t launch_scan_step(int B, int C, int dtype, const ScanTensor &x, const ScanTensor &gate, const float *gate_bias,
                             float *pool, int n_states, const int *slots, const ScanTensor &y, cudaStream_t st) {
    const int parts = ceil_div(C, 256);
    const unsigned grid = (unsigned)B * parts;
    const auto kernel = dtype == WTCONV_F32 ? scan_step_kernel<float>
                        : dtype == WTCONV_BF16 ? scan_step_kernel<__nv_bfloat16> : scan_step_kernel<__half>;
    return launch_kernel(kernel, grid, 256, 0, st, 1, C, parts, x, gate, gate_bias, pool, n_states, slots, y);
}

}  // namespace wtconv
