// Backward of the selective scan.
#pragma once

#include <atomic>
#include <type_traits>

#include "column_sums.cuh"
#include "selective_device.cuh"

namespace wtconv {

// d += A B with A 16 x 8 and B 8 x 8: of A, a lane holds (row, column) (lane / 4, lane % 4) in `low` and (8 + lane / 4,
// 4 + lane % 4) in `high`, the rest is 0; of B (lane % 4, lane / 4) and (4 + lane % 4, lane / 4); of d (lane / 4, 2 (lane %
// 4) + 0 and 1), then the same of row 8 + lane / 4.
// FIRST: d = A B.
template <bool FIRST> __device__ __forceinline__ void mma(float (&d)[4], uint32_t low, uint32_t high, uint32_t b0, uint32_t b1) {
    if constexpr (FIRST) {
        asm("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0, %1, %2, %3}, {%4, %5, %5, %6}, {%7, %8}, {%9, %9, %9, %9};"
            : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
            : "r"(low), "r"(0), "r"(high), "r"(b0), "r"(b1), "f"(0.f));
        return;
    }
    asm("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0, %1, %2, %3}, {%4, %5, %5, %6}, {%7, %8}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(low), "r"(0), "r"(high), "r"(b0), "r"(b1));
}

// A CTA takes 32 channels of a sequence (or of a segment), from the end to the beginning, in blocks of 16
// positions.  LANES lanes with four states each recompute a channel's states of a block from the kept one before it and
// hold them in registers (4 x 16 a lane), then go through the positions backwards; the CTA's other warps, the
// helpers, prepare the next block and finish the one before, as in the forward.
// Sums over a channel's states are put down by its lanes and meet in the helpers.  Those over channels (dB, dC) are the
// larger part: 8 values of every lane and position, over 32 / LANES channels of a warp.  The tensor cores add them up:
// for two positions at a time, the lanes' values of state s of B or C are the columns of a matrix whose rows are
// four channels at one position and the same four at the other, and a product with a matrix of ones in row r of
// the first four columns and row 8 + r of the others leaves the sums in row r (one position) and 8 + r; each of the 8
// values has an r of its own.  The tensor cores read a value's leading 11 bits and leave the rest out; the rest enters as
// a second product, of which they read 11 bits again: a value loses less than 2^-21 of itself, in every type.  (8 x 4096 x
// 1024 with 16 states in bf16: 1087 us, with the leading bits alone 812; but of sums whose channels cancel to a hundredth those are
// 3.0e-2 off, where rounding to bf16 costs 1.7e-3.  The rests of two values at once, as pairs: 1135.)
// Then warps meet in shared memory, and CTAs in selective_sums_kernel.
// With 8 and with 64 states the lanes hold half of a block's states at a time and recompute the first half twice: fewer
// registers are worth it there (8 x 4096 x 1024 in bf16: 720 us instead of 812 with 8 states, 1214 instead of 1087 with 16).
// LOCAL: only the gradient that the segment's beginning passes on if nothing enters at its end, and the sum
// of its steps; the CTAs of earlier segments begin with what these compose to.
template <int LANES, bool PLANES> struct BackwardShared {
    using L = Layout<LANES, PLANES, kSelKeep>;
    using Part = Share<PLANES, kSelTile, kSelKeep, Roles<LANES>::HELPERS, false>;
    static constexpr int ROWS = LANES / LanePlace<LANES>::HALVES;  // warps that have the same states
    alignas(16) float2 coef[L::COEFS];                                 // d, d x
    alignas(16) float r[L::VALUES];                                    // dy silu(z)
    alignas(16) float maps[2][kSelKeep * L::MAP];                      // B, C
    alignas(16) float sums[3][L::PARTS * L::APART];                    // over a channel's states: g B, k A, C h
    float2 stash[2][Part::COUNT][Roles<LANES>::HELPERS];               // of a helper's pairs: slope of d, dy silu'(z)
    float part[ROWS][kSelKeep][2][L::PAD];                             // dB and dC of a row of warps' channels
};

template <typename T, int LANES, bool PLANES, bool WIDE, bool LOCAL>
__global__ void __launch_bounds__(Roles<LANES>::THREADS, LANES <= 4 ? 2 : 1) selective_backward_kernel(const __grid_constant__ SelectiveArgs a) {
    constexpr int BLOCK = kSelKeep, HELD = LANES == 2 || LANES == 16 ? 8 : 16;
    using L = Layout<LANES, PLANES, BLOCK>;
    using R = Roles<LANES>;
    using Shared = BackwardShared<LANES, PLANES>;
    using Place2 = LanePlace<LANES>;
    extern __shared__ float4 shared_memory[];
    Shared *const blocks = reinterpret_cast<Shared *>(shared_memory);  // two
    begin_kernel();
    const Place at_(a, blockIdx.x);
    if (LOCAL && at_.segment == 0) return;  // nobody is before it
    const int b = at_.b, N = a.s.N, stop = min(at_.end, at_.length);
    const int count_blocks = stop > at_.first ? (stop - at_.first + BLOCK - 1) / BLOCK : 0;
    const long long first_sum = ((long long)b * a.segments + at_.segment) * a.s.C + at_.c0;  // of [B][segments][C]
    // the i-th block from the end
    const auto start = [&](int i) { return at_.first + (count_blocks - 1 - i) * BLOCK; };

    if (!R::scans()) {
        if (!LOCAL) R::template give<T>();
        using Part = Share<PLANES, kSelTile, BLOCK, R::HELPERS, WIDE>;
        using Maps = Share<PLANES, L::PAD, BLOCK, R::HELPERS, WIDE>;
        using Two = typename Raw<T>::Two;
        constexpr int COUNT = Part::COUNT, OWN = Part::OWN;
        const int me = R::helper();
        const Part mine(me);
        const Maps maps(me);
        const bool gated = a.in.z.p != nullptr;
        Pair bias[OWN], D[OWN], dD[OWN], d_bias[OWN];
        mine.parameters(a.in.dt_bias == nullptr ? nullptr : a.in.dt_bias + at_.c0, at_.channels, bias);
        mine.parameters(a.in.D == nullptr ? nullptr : a.in.D + at_.c0, at_.channels, D);
#pragma unroll
        for (int i = 0; i < OWN; ++i) dD[i] = d_bias[i] = Pair(0.f);
        struct Fetched {
            Two d[COUNT], x[COUNT], z[COUNT], dy[COUNT], b[Maps::COUNT], c[Maps::COUNT];
        } even, odd;
        Two x[COUNT] = {}, x_old[COUNT] = {};  // of the scanned block, the one finished
        using In = Cursor<const T, PLANES>;
        using Out = Cursor<T, PLANES>;
        const int last = start(0);  // (of no block: nothing is read or written there)
        In d_at(mine, a.in.dt, b, last, at_.c0), x_at(mine, a.in.x, b, last, at_.c0), z_at(mine, a.in.z, b, last, at_.c0);
        In dy_at(mine, a.dy, b, last, at_.c0), b_at(maps, a.in.Bm, b, last, at_.group * N), c_at(maps, a.in.Cm, b, last, at_.group * N);
        const auto fetch = [&](int i, Fetched &f) {
            if (i >= count_blocks) return;
            const int count = stop - start(i);
            mine.load(d_at.p, d_at.row, at_.channels, count, f.d), d_at.step(-BLOCK);
            mine.load(dy_at.p, dy_at.row, at_.channels, count, f.dy), dy_at.step(-BLOCK);
            if (gated) mine.load(z_at.p, z_at.row, at_.channels, count, f.z), z_at.step(-BLOCK);
            maps.load(c_at.p, c_at.row, N, count, f.c), c_at.step(-BLOCK);
            if (LOCAL) return;
            mine.load(x_at.p, x_at.row, at_.channels, count, f.x), x_at.step(-BLOCK);
            maps.load(b_at.p, b_at.row, N, count, f.b), b_at.step(-BLOCK);
        };
        const auto prepare = [&](int i, Fetched &f) {
            if (i >= count_blocks) return;
            Shared &s = blocks[i & 1];
            arrived(f.d), arrived(f.dy), arrived(f.c);
            if (!LOCAL) arrived(f.x), arrived(f.b);
            if (gated) arrived(f.z);
#pragma unroll
            for (int j = 0; j < COUNT; ++j) {
                x[j] = f.x[j];
                if (!mine.busy()) continue;
                const int t = mine.position(j), c = mine.channel(j);
                Pair d = add(pair_of<T>(f.d[j]), bias[PLANES ? j : 0]), r = pair_of<T>(f.dy[j]);
                if (a.s.softplus) {
                    const Pair e = exp_of_minus_abs(d);
                    if (!LOCAL) *reinterpret_cast<unsigned long long *>(&s.stash[0][j][me]) = softplus_slope(d, e).q;
                    d = softplus_of(d, e);
                }
                if (gated) {
                    const Pair z = pair_of<T>(f.z[j]), p = sigmoid_of(z), zp = mul(z, p);
                    // silu'(z) = p + z p (1 - p)
                    if (!LOCAL) *reinterpret_cast<unsigned long long *>(&s.stash[1][j][me]) = mul(r, fma(zp, sub(Pair(1.f), p), p)).q;
                    r = mul(r, zp);
                }
                const Pair dx = LOCAL ? Pair(0.f) : mul(d, pair_of<T>(x[j]));
                *reinterpret_cast<float4 *>(s.coef + L::coef(t, c)) = make_float4(d.lo(), dx.lo(), d.hi(), dx.hi());
                *reinterpret_cast<unsigned long long *>(s.r + L::value(t, c)) = r.q;
            }
            if (!LOCAL) L::template put_map<T>(maps, f.b, s.maps[0]);
            L::template put_map<T>(maps, f.c, s.maps[1]);
        };
        Out dx_at(mine, a.g.dx, b, last, at_.c0), dd_at(mine, a.g.d_dt, b, last, at_.c0), dz_at(mine, a.g.dz, b, last, at_.c0);
        float *part_at = a.part_bc + (((long long)at_.tile * a.s.B + b) * a.s.T + last) * 2 * L::PAD;
        const auto finish = [&](int i) {
            Shared &s = blocks[i & 1];
            const int count = min(BLOCK, stop - start(i));
            Pair dx[COUNT], dd[COUNT], dz[COUNT];
            const auto stashed = [&](int which, int j) { return Pair(*reinterpret_cast<const unsigned long long *>(&s.stash[which][j][me])); };
#pragma unroll
            for (int j = 0; j < COUNT; ++j) {
                if (!mine.busy()) continue;
                const int t = mine.position(j), c = mine.channel(j), place = L::value(t, c);
                // (an element past the end or beside the tile has whatever an earlier block left: it is neither stored nor summed)
                const float4 q = *reinterpret_cast<const float4 *>(s.coef + L::coef(t, c));
                const Pair into = L::get_sums(s.sums[0], place), xj = pair_of<T>(x_old[j]), Dj = D[PLANES ? j : 0];
                const Pair r(*reinterpret_cast<const unsigned long long *>(s.r + place));
                dd[j] = fma(xj, into, mul(L::get_sums(s.sums[1], place), Pair(kSelLn2)));
                if (a.s.softplus) dd[j] = mul(dd[j], stashed(0, j));
                dx[j] = fma(Dj, r, mul(Pair(q.x, q.z), into));
                if (gated) dz[j] = mul(stashed(1, j), fma(Dj, xj, L::get_sums(s.sums[2], place)));
                Pair rx = mul(r, xj), di = dd[j];
                if (count < BLOCK || at_.channels < kSelTile) {
                    const bool first = mine.in(j, 0, at_.channels, count), second = mine.in(j, 1, at_.channels, count);
                    rx = {first ? rx.lo() : 0.f, second ? rx.hi() : 0.f}, di = {first ? di.lo() : 0.f, second ? di.hi() : 0.f};
                }
                dD[PLANES ? j : 0] = add(dD[PLANES ? j : 0], rx), d_bias[PLANES ? j : 0] = add(d_bias[PLANES ? j : 0], di);
            }
            mine.store(dx_at.p, dx_at.row, at_.channels, count, [&](int j) { return dx[j]; }), dx_at.step(-BLOCK);
            mine.store(dd_at.p, dd_at.row, at_.channels, count, [&](int j) { return dd[j]; }), dd_at.step(-BLOCK);
            if (gated) mine.store(dz_at.p, dz_at.row, at_.channels, count, [&](int j) { return dz[j]; }), dz_at.step(-BLOCK);
            const auto part_sum = [&](int e) {
                const float *const from = &s.part[0][0][0][0] + e;
                Pair v(*reinterpret_cast<const unsigned long long *>(from));
#pragma unroll
                for (int w = 1; w < Shared::ROWS; ++w)
                    v = add(v, Pair(*reinterpret_cast<const unsigned long long *>(from + w * BLOCK * 2 * L::PAD)));
                *reinterpret_cast<unsigned long long *>(part_at + e) = v.q;
            };
            if (count == BLOCK) {
#pragma unroll
                for (int e = 0; e < BLOCK * 2 * L::PAD; e += 2 * R::HELPERS)
                    if (BLOCK * 2 * L::PAD % (2 * R::HELPERS) == 0 || e + 2 * me < BLOCK * 2 * L::PAD) part_sum(e + 2 * me);
            } else {
                for (int e = 2 * me; e < count * 2 * L::PAD; e += 2 * R::HELPERS) part_sum(e);
            }
            part_at -= BLOCK * 2 * L::PAD;
        };
        const auto during = [&](int i, Fetched &next, Fetched &after) {  // block i is scanned
            fetch(i + 2, after);
            if (!LOCAL && i > 0) finish(i - 1);
#pragma unroll
            for (int j = 0; j < COUNT; ++j) x_old[j] = x[j];
            prepare(i + 1, next);
            R::meet();
        };
        fetch(0, even), fetch(1, odd), prepare(0, even);
        R::meet();
        for (int i = 0; i < count_blocks; i += 2) {
            during(i, odd, even);
            if (i + 1 < count_blocks) during(i + 1, even, odd);
        }
        if (LOCAL) return;
        if (count_blocks > 0) finish(count_blocks - 1);
        // dD and d_dt_bias: the helpers that share a channel
        const long long half = (long long)a.s.B * a.segments * a.s.C;
        if (PLANES) {  // neighbouring lanes
#pragma unroll
            for (int j = 0; j < OWN; ++j) {
                float v = dD[j].lo() + dD[j].hi(), w = d_bias[j].lo() + d_bias[j].hi();
#pragma unroll
                for (int m = Part::INNER / 2; m >= 1; m /= 2) v += __shfl_xor_sync(0xffffffffu, v, m), w += __shfl_xor_sync(0xffffffffu, w, m);
                const int c = mine.channel(j);
                if (mine.busy() && mine.inner == 0 && c < at_.channels) a.part_c[first_sum + c] = v, a.part_c[half + first_sum + c] = w;
            }
        } else {
            R::helpers_meet();
            float2 *const meet = reinterpret_cast<float2 *>(blocks[0].sums);  // [2][HELPERS]
            *reinterpret_cast<unsigned long long *>(meet + me) = dD[0].q, *reinterpret_cast<unsigned long long *>(meet + R::HELPERS + me) = d_bias[0].q;
            R::helpers_meet();
            if (me < at_.channels) {
                float v = 0.f, w = 0.f;
                for (int j = 0; j < R::HELPERS / Part::INNER; ++j) {
                    const float *const p = reinterpret_cast<const float *>(meet + j * Part::INNER) + me;
                    v += p[0], w += p[2 * R::HELPERS];
                }
                a.part_c[first_sum + me] = v, a.part_c[half + first_sum + me] = w;
            }
        }
        // positions past the sequence's end
        for (int t0 = max(at_.first, at_.length); t0 < at_.end; t0 += BLOCK) {
            mine.clear(mine.mine(at<T, PLANES>(a.g.dx, b, t0, at_.c0), a.g.dx.row), a.g.dx.row, at_.channels, at_.end - t0);
            mine.clear(mine.mine(at<T, PLANES>(a.g.d_dt, b, t0, at_.c0), a.g.d_dt.row), a.g.d_dt.row, at_.channels, at_.end - t0);
            if (gated) mine.clear(mine.mine(at<T, PLANES>(a.g.dz, b, t0, at_.c0), a.g.dz.row), a.g.dz.row, at_.channels, at_.end - t0);
        }
        return;
    }

    if (!LOCAL) R::template take<T>();
    const Place2 lane;
    const int c = lane.c, quad = lane.quad, n0 = lane.n0;
    const bool live = c < at_.channels;
    const long long row = (long long)b * a.s.C + at_.c0 + c;  // of [B][C]
    Quad decay = {Pair(0.f), Pair(0.f)}, carry = decay, dA = decay;
    if (live) {
        decay = load_rates(a.in.A + (long long)(at_.c0 + c) * N, n0, N);
        decay.a = mul(decay.a, Pair(kSelLog2E)), decay.b = mul(decay.b, Pair(kSelLog2E));
    }
    if (!LOCAL && live) {
        if (a.dh_last != nullptr) carry = load_quad(a.dh_last + row * N, n0, N);
        if (count_blocks > 0)
#pragma unroll 4
            for (int k = (at_.length - 1) / a.segment; k > at_.segment; --k) {
                const long long i = ((long long)b * a.segments + k) * a.s.C + at_.c0 + c;
                const Pair d(0.25f * a.steps[i]);
                const Quad u = quad_of(*reinterpret_cast<const float4 *>(a.ends + i * L::PAD + n0));
                carry.a = through_part(mul(d, decay.a), carry.a, u.a), carry.b = through_part(mul(d, decay.b), carry.b, u.b);
            }
    }
    float step_sum = 0.f;
    const auto kept = [&](int i) {
        if (!live || i >= count_blocks) return make_float4(0.f, 0.f, 0.f, 0.f);
        return *reinterpret_cast<const float4 *>(a.states_in + (((long long)b * a.keep + start(i) / kSelKeep) * a.s.C + at_.c0 + c) * L::PAD + n0);
    };
    float4 kept_next = LOCAL ? make_float4(0.f, 0.f, 0.f, 0.f) : kept(0);
    uint32_t one[8];  // the 1 of a row r of the matrix of ones
#pragma unroll
    for (int r = 0; r < 8; ++r) one[r] = lane.lane / 4 == r ? 0x3f800000u : 0u;
    R::meet();
    for (int i = 0; i < count_blocks; ++i) {
        Shared &s = blocks[i & 1];
        const int count = min(BLOCK, stop - start(i));
        const auto map = [&](int which, int t) { return *reinterpret_cast<const float4 *>(s.maps[which] + t * L::MAP + n0); };
        if (LOCAL) {
            const auto pass = [&](int t) {
                const float2 q = s.coef[L::coef(t, c)];
                const Quad o = quad_of(map(1, t));
                const Pair d(q.x), r(s.r[L::value(t, c)]);
                carry.a = mul(decays_of(d, decay.a), fma(o.a, r, carry.a));
                carry.b = mul(decays_of(d, decay.b), fma(o.b, r, carry.b));
                step_sum += q.x;
            };
            if (count == BLOCK) {
#pragma unroll
                for (int t = BLOCK - 1; t >= 0; --t) pass(t);
            } else {
                for (int t = count - 1; t >= 0; --t) pass(t);
            }
            R::meet();
            continue;
        }

        asm volatile("" : "+f"(kept_next.x), "+f"(kept_next.y), "+f"(kept_next.z), "+f"(kept_next.w));  // (see arrived)
        const Quad before = quad_of(kept_next);
        kept_next = kept(i + 1);
        const auto scan = [&](auto full) {
            constexpr bool FULL = decltype(full)::value;
            constexpr int TOGETHER = L::TOGETHER;
            Quad dA_block = {Pair(0.f), Pair(0.f)};
            const auto advance = [&](const Quad &h, int t) {
                const float2 q = s.coef[L::coef(t, c)];
                const Quad u = quad_of(map(0, t));
                const Pair d(q.x), dx(q.y);
                return Quad{fma(decays_of(d, decay.a), h.a, mul(dx, u.a)), fma(decays_of(d, decay.b), h.b, mul(dx, u.b))};
            };
            // (what a position needs is loaded before the one after it is stored, as in the forward)
            struct Operands {
                float2 q;
                float4 u, o;
                float r;
            };
            const auto operands = [&](int t) { return Operands{s.coef[L::coef(t, c)], map(0, t), map(1, t), s.r[L::value(t, c)]}; };
            Operands next = operands(FULL ? BLOCK - 1 : count - 1);
            float s1[TOGETHER] = {}, s2[TOGETHER] = {}, s3[TOGETHER] = {};
            float sums[4];  // of the last two positions
            const auto put_part = [&](int t) {
                // row lane / 4: value (state, B or C); columns: the group of four channels, then the quad of states
                const int r = lane.lane / 4, j = lane.lane % 4, which = r / 4, state = r % 4;
                constexpr int FOURS = Place2::CHANNELS / 4;  // columns of a quad: 4, 2 or 1
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    float *const to = s.part[lane.row][t + k][which] + lane.warp % Place2::HALVES * 4 * Place2::WITHIN + state;
                    const float v0 = sums[2 * k], v1 = sums[2 * k + 1];
                    if constexpr (FOURS == 1) {
                        to[8 * j] = v0, to[8 * j + 4] = v1;
                    } else {
                        float v = v0 + v1;
                        if (FOURS == 4) v += __shfl_xor_sync(0xffffffffu, v, 1);
                        if (FOURS == 2) to[4 * j] = v;
                        else if (j % 2 == 0) to[2 * j] = v;
                    }
                }
            };
            bool first = true;
            // parts of the block, from the last: a part's states are held in registers
#pragma unroll 1
            for (int from = BLOCK - HELD; from >= 0; from -= HELD) {
                if (!FULL && from >= count) continue;
                Quad before_part = before;
                for (int t = 0; t < from; ++t) before_part = advance(before_part, t);
                Quad h[HELD];
#pragma unroll
                for (int t = 0; t < HELD; ++t) {
                    if (!FULL && from + t >= count) break;
                    h[t] = advance(t == 0 ? before_part : h[t == 0 ? 0 : t - 1], from + t);
                }
                // Position from + t; v: its products of the lane's states, B's and C's.
                const auto pass = [&](int t, float (&v)[8]) {
                    const Operands now = next;
                    if (HELD < BLOCK || t > 0) next = operands(max(from + t - 1, 0));
                    const Quad u = quad_of(now.u), o = quad_of(now.o), last = t == 0 ? before_part : h[t == 0 ? 0 : t - 1];
                    const Pair d(now.q.x), dx(now.q.y), r(now.r);
                    const Quad g = {fma(o.a, r, carry.a), fma(o.b, r, carry.b)};
                    carry.a = mul(decays_again(d, decay.a), g.a), carry.b = mul(decays_again(d, decay.b), g.b);
                    const Quad kk = {mul(carry.a, last.a), mul(carry.b, last.b)};
                    dA_block.a = fma(kk.a, d, dA_block.a), dA_block.b = fma(kk.b, d, dA_block.b);
                    const Pair p1 = fma(g.a, u.a, mul(g.b, u.b)), p2 = fma(kk.a, decay.a, mul(kk.b, decay.b));
                    const Pair p3 = fma(o.a, h[t].a, mul(o.b, h[t].b));
                    s1[t % TOGETHER] = p1.lo() + p1.hi(), s2[t % TOGETHER] = p2.lo() + p2.hi(), s3[t % TOGETHER] = p3.lo() + p3.hi();
                    const Pair b0 = mul(g.a, dx), b1 = mul(g.b, dx), c0 = mul(h[t].a, r), c1 = mul(h[t].b, r);
                    v[0] = b0.lo(), v[1] = b0.hi(), v[2] = b1.lo(), v[3] = b1.hi();
                    v[4] = c0.lo(), v[5] = c0.hi(), v[6] = c1.lo(), v[7] = c1.hi();
                };
                const auto put_sums = [&](int t) {  // once its TOGETHER positions are through
                    if (t % TOGETHER != 0) return;
                    const int at_t = from + t;
                    L::put_sums(s.sums[0], at_t, c, quad, s1), L::put_sums(s.sums[1], at_t, c, quad, s2), L::put_sums(s.sums[2], at_t, c, quad, s3);
                };
#pragma unroll
                for (int t = HELD - 2; t >= 0; t -= 2) {
                    if (!FULL && from + t >= count) continue;
                    float v0[8], v1[8] = {};
                    if (FULL || from + t + 1 < count) pass(t + 1, v1), put_sums(t + 1);
                    else if (TOGETHER > 1) s1[(t + 1) % TOGETHER] = s2[(t + 1) % TOGETHER] = s3[(t + 1) % TOGETHER] = 0.f;
                    pass(t, v0), put_sums(t);
                    // (the sums of the two positions after these: the products have had the time of two more)
                    if (HELD == BLOCK && FULL ? t < HELD - 2 : !first) put_part(from + t + 2);
                    first = false;
#pragma unroll
                    for (int r = 0; r < 8; ++r) {
                        const uint32_t h0 = __float_as_uint(v0[r]), h1 = __float_as_uint(v1[r]);
                        if (r == 0) mma<true>(sums, one[r], one[r], h0, h1);
                        else mma<false>(sums, one[r], one[r], h0, h1);
                        // what the product with the upper 11 bits left
                        const float l0 = v0[r] - __uint_as_float(h0 & 0xffffe000u), l1 = v1[r] - __uint_as_float(h1 & 0xffffe000u);
                        mma<false>(sums, one[r], one[r], __float_as_uint(l0), __float_as_uint(l1));
                    }
                }
            }
            put_part(0);
            dA.a = add(dA.a, dA_block.a), dA.b = add(dA.b, dA_block.b);
        };
        if (count == BLOCK) scan(std::true_type{});
        else scan(std::false_type{});
        R::meet();
    }

    if (LOCAL) {
        if (live && count_blocks > 0) {
            *reinterpret_cast<float4 *>(a.ends + (first_sum + c) * L::PAD + n0) = float4_of(carry);
            if (quad == 0) a.steps[first_sum + c] = step_sum;
        }
        return;
    }
    if (at_.segment == 0 && live && a.g.d_h0 != nullptr) store_quad(a.g.d_h0 + row * N, n0, N, carry);
    if (live) store_quad(a.part_a + (first_sum + c) * N, n0, N, dA);
}

// dB and dC: the sums over a group's tiles, in their order, of 32 positions; 0 past a sequence's end.
constexpr int kSelSumsThreads = 256;
template <typename T, int LANES, bool PLANES> __global__ void __launch_bounds__(kSelSumsThreads) selective_sums_kernel(const __grid_constant__ SelectiveArgs a) {
    constexpr int PAD = 4 * LANES, WIDTH = 2 * PAD, TURN = 32;
    __shared__ float sums[WIDTH][TURN + 1];
    begin_kernel();
    const int turns = (a.s.T + TURN - 1) / TURN, N = a.s.N;
    const int t0 = blockIdx.x % turns * TURN, g = blockIdx.x / turns % a.s.G, b = blockIdx.x / turns / a.s.G;
    const int length = a.in.lengths == nullptr ? a.s.T : min(max(a.in.lengths[b], 0), a.s.T);
    const int live = max(min(TURN, length - t0), 0), count = min(TURN, a.s.T - t0);
    const long long per = (long long)a.s.B * a.s.T * WIDTH;  // of a tile
    const float *const from = a.part_bc + (long long)g * a.tiles * per + ((long long)b * a.s.T + t0) * WIDTH;
    for (int e = 4 * threadIdx.x; e < TURN * WIDTH; e += 4 * kSelSumsThreads) {  // (67 MB: 14 us; one value at a time 42)
        Quad v = {Pair(0.f), Pair(0.f)};
        if (e / WIDTH < live) {
#pragma unroll 8
            for (int i = 0; i < a.tiles; ++i) {
                const Quad q = quad_of(*reinterpret_cast<const float4 *>(from + i * per + e));
                v.a = add(v.a, q.a), v.b = add(v.b, q.b);
            }
        }
        const int j = e % WIDTH, t = e / WIDTH;
        sums[j][t] = v.a.lo(), sums[j + 1][t] = v.a.hi(), sums[j + 2][t] = v.b.lo(), sums[j + 3][t] = v.b.hi();
    }
    __syncthreads();
    for (int e = threadIdx.x; e < TURN * WIDTH; e += kSelSumsThreads) {
        const int t = PLANES ? e % TURN : e / WIDTH, j = PLANES ? e / TURN : e % WIDTH, n = j % PAD;
        if (t < count && n < N) *at<T, PLANES>(j / PAD ? a.g.dC : a.g.dB, b, t0 + t, g * N + n) = from_f32<T>(sums[j][t]);
    }
}

template <typename T, int LANES, bool PLANES, bool WIDE> cudaError_t launch_selective_backward_as(const SelectiveArgs &a, cudaStream_t st) {
    const unsigned threads = Roles<LANES>::THREADS, grid = (unsigned)a.ctas() * a.segments;
    const size_t shared = 2 * sizeof(BackwardShared<LANES, PLANES>);
    // (the scanners would wait for registers that the CTA does not have)
    if (Roles<LANES>::TRADE) {
        static std::atomic<int> registers{0};
        if (registers == 0) {
            cudaFuncAttributes attributes;
            const cudaError_t e = cudaFuncGetAttributes(&attributes, selective_backward_kernel<T, LANES, PLANES, WIDE, false>);
            if (e != cudaSuccess) return e;
            registers = attributes.numRegs;
        }
        if (registers != Roles<LANES>::LAUNCHED) return cudaErrorLaunchOutOfResources;
    }
    const auto local = selective_backward_kernel<T, LANES, PLANES, WIDE, true>, whole = selective_backward_kernel<T, LANES, PLANES, WIDE, false>;
    cudaError_t e = cudaSuccess;
    if (a.segments > 1) {
        if ((e = allow_shared(local, shared)) != cudaSuccess) return e;
        if ((e = launch_kernel(local, grid, threads, shared, st, 1, a)) != cudaSuccess) return e;
    }
    if ((e = allow_shared(whole, shared)) != cudaSuccess) return e;
    if ((e = launch_kernel(whole, grid, threads, shared, st, 1, a)) != cudaSuccess) return e;
    const unsigned turns = (unsigned)a.s.B * a.s.G * ceil_div(a.s.T, 32);
    if ((e = launch_kernel(selective_sums_kernel<T, LANES, PLANES>, turns, kSelSumsThreads, 0, st, 1, a)) != cudaSuccess) return e;
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
