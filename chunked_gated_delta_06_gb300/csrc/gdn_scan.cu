// gdn_scan.cu -- the selective scan's forward (packed, and over pool slots), its state pass over the
// segments of a split scan, and the step of one token for each row.
#include <type_traits>

#include "gdn_scan.cuh"

namespace gdn {
namespace {

// What a walk is for: the outputs; a segment's end, for the segments behind it; or, for a gradient, the
// states ahead of the tiles and, of a split sequence, both the segment's end and its start's gradient.
enum WalkFor { kOutputs, kEnds, kMarks };

// Half of a block's warps ("formers") form d, d x and the outputs, the others ("walkers") walk the
// states, up to 16 of a channel a thread (8 where each has its decay since the start and its gradient
// too).  While one tile is walked the next one is formed, the outputs of the one before are written and
// the inputs of the one after next are on their way.
//
// What bounds it: a state takes an exponential and four products or multiply-adds a token (a gradient's walk
// six), far more than its share of the bytes.  4 x 4096 tokens of 4096 channels of 16 states, bf16: 334 us, where
// the bytes are 80; 128 blocks of the 152 SMs work.  The walk's exponentials, products and multiply-adds by
// themselves take 178 of it.  Left out one at a time, the walk's reads of d and d x are 47 us, the formers'
// arithmetic 37, the exponentials 30, the sums over lanes 22, the outputs' product 18, the inputs' product 12, the
// reads of B and C 11: the other half is what passes through shared memory and between lanes, and the formers.
// (All in one kind of thread, states in registers and no tiles ahead: 835 us.  A tile's tokens unrolled: 349
// before.)  65536 tokens of 2048 channels in one sequence, split: 917 us, unsplit 5200.  A tile is walked in full: 256
// sequences of one token of 2048 channels take 97 us.
template <int NS, WalkFor kFor>
struct WalkShape {
    static constexpr int kMost = kFor == kMarks ? 8 : 16;           // states of a walker
    // its channels, and states of each: two channels read a token's B and C once (4 x 4096 tokens of 4096
    // channels of 8 states 279 us, one channel 289), but of 32 states for outputs would make four sum up
    // (2048 channels 351 us, one channel 338)
    static constexpr int P = NS == 32 && kFor == kOutputs ? 1 : 2, S = (NS < kMost ? NS : kMost) / P;
    static constexpr int L = NS / S;                                // walkers of a channel
    static constexpr int kHalf = 128;                         // threads of either kind
    static constexpr int CB = P * kHalf / L;                  // channels of a block
    static constexpr int TT = 16;                             // tokens of a tile
    static constexpr int kRing = 4;                           // tiles of inputs: finished, walked, formed, on their way
};

template <typename T, int NS, WalkFor kFor>
struct ScanTiles {
    using Shape = WalkShape<NS, kFor>;
    static constexpr int CB = Shape::CB, TT = Shape::TT, kRing = Shape::kRing;
    static constexpr int kMore = kFor == kEnds ? 1 : kRing, kDy = kFor == kMarks ? kRing : 1;
    float d[2][TT][CB], dx[2][TT][CB];   // d and d x, channels at channel_at
    float B[2][TT][NS], C[2][kFor == kEnds ? 1 : TT][NS];
    float y[2][kFor == kEnds ? 1 : TT][CB];   // the walkers' sums; for marks o, of the formers, at channel_at
    float bias[CB], skip[CB];
    alignas(16) T x[kRing][TT * CB], dt[kRing][TT * CB], z[kMore][TT * CB], dy[kDy][TT * CB];
    alignas(16) T rB[kRing][TT * NS], rC[kMore][TT * NS];
};

// Runs of four channels change places, so that formers that write eight each meet no bank twice.
__device__ __forceinline__ int channel_at(int c) { return c ^ (c >> 3 & 4); }

// A segment's end is had without its start (from nothing): the join adds what the start leaves.  So is the
// gradient at the start from nothing behind, walking forward too, as each token's part decays by what the
// walk has gone through: with P_t the product of the decays up to t it is the sum of P_t C_t o_t.
// In 32 bits, P loses 2^-22 a token, as the walked state does.
template <typename T, int NS, bool kWide, WalkFor kFor>
__global__ void __launch_bounds__(2 * WalkShape<NS, kFor>::kHalf, 2)
    k_scan_fwd(const __grid_constant__ ScanArgs a) {
    using Shape = WalkShape<NS, kFor>;
    constexpr int CB = Shape::CB, L = Shape::L, P = Shape::P, S = Shape::S, TT = Shape::TT, R = Shape::kRing, EV = 8;
    constexpr int kHalf = Shape::kHalf;
    using Tile = TileOf<T, CB, TT, EV, kHalf, kWide>;
    using Rows = RowsOf<T, NS, TT, kHalf>;
    using Tiles = ScanTiles<T, NS, kFor>;
    extern __shared__ float4 smem[];
    Tiles &m = *reinterpret_cast<Tiles *>(smem);

    ScanPlace w;
    if (!scan_place<CB>(a, blockIdx.x, &w)) {
        if (kFor == kOutputs && a.pack.status && w.item == a.pack.N + a.pack.T / a.seg) check_offsets(a.pack);
        return;
    }
    if (kFor == kEnds && w.seg == w.segs - 1) return;
    for (int i = threadIdx.x; i < CB; i += 2 * kHalf) {
        const bool there = w.c0 + i < w.cend && in_range(w.c0 + i, 1, a.C, a.pack.status);
        m.bias[i] = there && a.dt_bias ? a.dt_bias[w.c0 + i] : 0.f;
        m.skip[i] = there && a.D ? a.D[w.c0 + i] : 0.f;
    }
    __syncthreads();
    const int tiles = (w.f - w.b + TT - 1) / TT;

    if (threadIdx.x < kHalf) {
        using V = typename Tile::V;
        using U = typename Rows::V;
        using Feed = FeedOf<Tile, T, kHalf, kWide>;
        using RowFeed = RowFeedOf<Rows, T, NS, kHalf, kWide>;
        const bool gated = a.z != nullptr, more = kFor == kOutputs || (kFor == kMarks && w.seg > 0);   // C, and the gate
        Feed x(static_cast<const T *>(a.x), a.xs, a, w, TT), dt(static_cast<const T *>(a.dt), a.dts, a, w, TT);
        Feed z(static_cast<const T *>(a.z), a.zs, a, w, TT), dy(static_cast<const T *>(a.dy), a.C, a, w, TT);
        RowFeed B(static_cast<const T *>(a.B), a.bs, a, w, TT), C(static_cast<const T *>(a.Cm), a.cs, a, w, TT);
        const int col = Tile::col();
        auto place = [&](T (*ring)[TT * CB], int i) { return reinterpret_cast<V *>(ring[i % R]); };
        auto fetch = [&](int i) {
            if (i < tiles) {
                x.next(place(m.x, i), a, w, TT);
                dt.next(place(m.dt, i), a, w, TT);
                B.next(reinterpret_cast<U *>(m.rB[i % R]), a, TT);
                if (more) {
                    if (gated) z.next(place(m.z, i), a, w, TT);
                    if (kFor == kMarks) dy.next(place(m.dy, i), a, w, TT);
                    C.next(reinterpret_cast<U *>(m.rC[i % R]), a, TT);
                }
            }
            copies_commit();
        };
        // d and d x of tile i; a token past the segment has d = 0, which leaves the state alone
        auto form = [&](int i) {
#pragma unroll
            for (int k = 0; k < Tile::NV; ++k) {
                const int row = Tile::row(k);
                if (row >= TT) break;
                float xv[EV], dv[EV], d4[EV], dx4[EV];
                unpack(place(m.x, i)[Tile::thread() + k * kHalf], xv);
                unpack(place(m.dt, i)[Tile::thread() + k * kHalf], dv);
                const bool there = w.b + i * TT + row < w.f;
#pragma unroll
                for (int j = 0; j < EV; j += 2) {
                    float2 d = softplus_of(add2(make_float2(dv[j], dv[j + 1]),
                                                *reinterpret_cast<const float2 *>(&m.bias[col + j])));
                    if (!there) d = both(0.f);
                    const float2 dx = mul2(d, make_float2(xv[j], xv[j + 1]));
                    d4[j] = d.x;
                    d4[j + 1] = d.y;
                    dx4[j] = dx.x;
                    dx4[j + 1] = dx.y;
                }
#pragma unroll
                for (int j = 0; j < EV; j += 4) {
                    *reinterpret_cast<float4 *>(&m.d[i & 1][row][channel_at(col + j)]) = make_float4(d4[j], d4[j + 1], d4[j + 2], d4[j + 3]);
                    *reinterpret_cast<float4 *>(&m.dx[i & 1][row][channel_at(col + j)]) = make_float4(dx4[j], dx4[j + 1], dx4[j + 2], dx4[j + 3]);
                }
                if (kFor != kMarks || !more) continue;
                float o[EV], zv[EV];
                unpack(place(m.dy, i)[Tile::thread() + k * kHalf], o);
                if (gated) {
                    unpack(place(m.z, i)[Tile::thread() + k * kHalf], zv);
#pragma unroll
                    for (int j = 0; j < EV; j += 2) {
                        const float2 g = mul2(make_float2(o[j], o[j + 1]), silu_of(make_float2(zv[j], zv[j + 1])));
                        o[j] = g.x;
                        o[j + 1] = g.y;
                    }
                }
#pragma unroll
                for (int j = 0; j < EV; j += 4)
                    *reinterpret_cast<float4 *>(&m.y[i & 1][row][channel_at(col + j)]) = make_float4(o[j], o[j + 1], o[j + 2], o[j + 3]);
            }
            Rows::keep_copied(reinterpret_cast<const U *>(m.rB[i % R]), m.B[i & 1]);
            if (more) Rows::keep_copied(reinterpret_cast<const U *>(m.rC[i % R]), m.C[i & 1]);
        };
        auto finish = [&](int i) {
#pragma unroll
            for (int k = 0; k < Tile::NV; ++k) {
                const int row = Tile::row(k);
                if (row >= TT) break;
                float xv[EV], zv[EV], out[EV];
                unpack(place(m.x, i)[Tile::thread() + k * kHalf], xv);
                if (gated) unpack(place(m.z, i)[Tile::thread() + k * kHalf], zv);
                const float *sums = m.y[i & 1][row] + col;
#pragma unroll
                for (int j = 0; j < EV; j += 2) {
                    float2 y = fma2(*reinterpret_cast<const float2 *>(&m.skip[col + j]),
                                    make_float2(xv[j], xv[j + 1]), *reinterpret_cast<const float2 *>(&sums[j]));
                    if (gated) y = mul2(y, silu_of(make_float2(zv[j], zv[j + 1])));
                    out[j] = y.x;
                    out[j + 1] = y.y;
                }
                Tile::store(static_cast<T *>(a.y), a, w, w.b + i * TT, w.f, k, pack<T>(out));
            }
        };
        fetch(0);
        fetch(1);
        copies_wait<1>();
        if (tiles > 0) form(0);
        __syncthreads();
        for (int i = 0; i <= tiles; ++i) {
            fetch(i + 2);
            copies_wait<1>();
            if (i + 1 < tiles) form(i + 1);
            if (kFor == kOutputs && i > 0) finish(i - 1);
            __syncthreads();
        }
        return;
    }

    using Lane = ScanLane<NS, P, S, kHalf>;
    constexpr int H = S / 2, BT = L < 4 ? L : 4;
    const Lane lane(a, w);
    const long long items = a.pack.N + (long long)(a.pack.T / a.seg);
    const int last = w.item - w.seg + w.segs - 1;   // the item of the sequence's last segment
    // The state ahead of the segment.  The record of the last segment, which has no end to keep, first
    // holds the state ahead of the sequence: a slot is read once, before any block writes it.
    typename Lane::States h;
    if (kFor != kOutputs || w.segs == 1) {
        const int from = w.seg == 0 ? scan_start_row(a, w.n) : -1;
        lane.load(a.s0, from, a.slots.idx ? a.slots.num_slots : a.pack.N, a, w, h);
        if (kFor != kOutputs && w.segs > 1 && w.seg == 0) lane.store(a.rec_h, last, items, a, w, h);
    } else {
        lane.load(a.rec_h, w.item, items, a, w, h);
    }
    float2 total = both(0.f);   // sums of d, of each channel
    const int place = channel_at(P * lane.at);
    const long long marks = a.pack.N + (long long)(a.pack.T / kMarkTile), mark = first_mark(a, w);
    auto keep_total = [&](float *to, long long row, long long rows, float2 sum) {   // [rows, C]
        const long long at = row * a.C + lane.c;
        if (lane.q) return;
        if (lane.c < w.cend && in_range(at, 1, rows * a.C, a.pack.status)) to[at] = sum.x;
        if (P == 2 && lane.c + 1 < w.cend && in_range(at + 1, 1, rows * a.C, a.pack.status)) to[at + 1] = sum.y;
    };
    __syncthreads();
    // kBoth: with the gradient at the segment's start, from nothing behind it
    auto walk = [&](auto both_) {
        constexpr bool kBoth = decltype(both_)::value, kC = kFor == kOutputs || kBoth;
        typename Lane::States gone, g;   // the product of the decays, and the gradient
        if constexpr (kBoth) {
#pragma unroll
            for (int p = 0; p < P; ++p)
#pragma unroll
                for (int k = 0; k < H; ++k) {
                    gone[p][k] = both(1.f);
                    g[p][k] = both(0.f);
                }
        }
        for (int i = 0; i <= tiles; ++i) {
            if (i < tiles) {
                auto row = [&](const float *rows, int t) {   // of the walker's channels
                    const float *at = rows + t * CB + place;
                    return P == 2 ? *reinterpret_cast<const float2 *>(at) : make_float2(*at, 0.f);
                };
                const float *ds = m.d[i & 1][0], *dxs = m.dx[i & 1][0], *os = m.y[i & 1][0];
                const float4 *B = reinterpret_cast<const float4 *>(m.B[i & 1][0] + S * lane.q);
                const float4 *C = reinterpret_cast<const float4 *>(m.C[i & 1][0] + S * lane.q);
                // All of the tile's tokens: those past the segment change nothing.  The decays, B and C are
                // formed and read one token ahead of the states that take them.
                float2 d = row(ds, 0), dx = row(dxs, 0), o = both(0.f), dec[P][H], b[H], c[H];
                if (kBoth) o = row(os, 0);
                auto ahead = [&](int t) {
#pragma unroll
                    for (int k = 0; k < H; k += 2) {
                        const float4 v = B[(t * NS + 2 * k) / 4];
                        b[k] = make_float2(v.x, v.y);
                        b[k + 1] = make_float2(v.z, v.w);
                        if (kC) {
                            const float4 u = C[(t * NS + 2 * k) / 4];
                            c[k] = make_float2(u.x, u.y);
                            c[k + 1] = make_float2(u.z, u.w);
                        }
                    }
                };
                auto decays = [&] {
#pragma unroll
                    for (int p = 0; p < P; ++p)
#pragma unroll
                        for (int k = 0; k < H; ++k) dec[p][k] = lane.decay(p, k, both(p ? d.y : d.x));
                };
                decays();
                ahead(0);
                float2 next_d = row(ds, 1), next_dx = row(dxs, 1), sum = both(0.f);
#pragma unroll
                for (int t0 = 0; t0 < TT; t0 += BT) {
                    if (kFor == kMarks && t0 % kMarkTile == 0 && w.b + i * TT + t0 < w.f) {
                        const long long to = mark + (i * TT + t0) / kMarkTile;
                        lane.store(a.marks, to, marks, a, w, h);
                        if (kBoth) keep_total(a.mark_d, to, marks, add2(total, sum));
                    }
                    float part[BT][P];
#pragma unroll
                    for (int j = 0; j < BT; ++j) {
                        const int t = t0 + j;
#pragma unroll
                        for (int p = 0; p < P; ++p) {
                            float2 y = both(0.f);
                            const float2 input = both(p ? dx.y : dx.x);
#pragma unroll
                            for (int k = 0; k < H; ++k) {
                                h[p][k] = fma2(dec[p][k], h[p][k], mul2(input, b[k]));
                                if (kFor == kOutputs) y = k ? fma2(c[k], h[p][k], y) : mul2(c[k], h[p][k]);
                                if constexpr (kBoth) {
                                    gone[p][k] = mul2(gone[p][k], dec[p][k]);
                                    g[p][k] = fma2(gone[p][k], mul2(both(p ? o.y : o.x), c[k]), g[p][k]);
                                }
                            }
                            part[j][p] = y.x + y.y;
                        }
                        if (kFor != kOutputs) sum = add2(sum, d);
                        const int u = min(t + 1, TT - 1), v = min(t + 2, TT - 1);
                        d = next_d;
                        dx = next_dx;
                        if (kBoth) o = row(os, u);
                        next_d = row(ds, v);
                        next_dx = row(dxs, v);
                        ahead(u);
                        decays();
                    }
                    if (kFor == kOutputs) {
                        lane_sums<L, BT, P>(part, lane.q);
                        if (lane.q < BT) {
                            float *y = &m.y[i & 1][t0 + lane.q][P * lane.at];
                            if constexpr (P == 2) *reinterpret_cast<float2 *>(y) = make_float2(part[0][0], part[0][1]);
                            else *y = part[0][0];
                        }
                    }
                }
                total = add2(total, sum);
            }
            __syncthreads();
        }
        if constexpr (kBoth) {
            if (w.seg == w.segs - 1 && a.ds1) {
                typename Lane::States end;
                lane.load(a.ds1, w.n, a.pack.N, a, w, end);
#pragma unroll
                for (int p = 0; p < P; ++p)
#pragma unroll
                    for (int k = 0; k < H; ++k) g[p][k] = fma2(gone[p][k], end[p][k], g[p][k]);
            }
            lane.store(a.rec_g, w.item, items, a, w, g);
        }
    };
    if constexpr (kFor == kMarks) {
        if (w.seg > 0) walk(std::true_type{});
        else walk(std::false_type{});
    } else {
        walk(std::false_type{});
    }
    if (kFor != kOutputs) {
        if (w.seg == w.segs - 1) return;
        lane.store(a.rec_h, w.item, items, a, w, h);
        keep_total(a.rec_d, w.item, items, total);
        return;
    }
    if (w.seg != w.segs - 1) return;
    if (a.slots.idx && a.slots.status && threadIdx.x == kHalf && a.slots.idx[w.n] >= a.slots.num_slots) *a.slots.status = 1;
    const int to = a.slots.idx ? slot_of(a.slots, w.n) : w.n;
    lane.store(a.s1, to, a.slots.idx ? a.slots.num_slots : a.pack.N, a, w, h);
}

// One thread for four states of a channel, from segment to segment; eight records on their way at once.
template <bool kBackward>
__global__ void __launch_bounds__(128) k_scan_join(const __grid_constant__ ScanArgs a, int across) {
    const int n = blockIdx.x / across;
    const long long i = ((long long)(blockIdx.x % across) * 128 + threadIdx.x) * 4, per = (long long)a.C * a.Ns;
    const int b = offset_of(a.pack, n), e = max(b, offset_of(a.pack, n + 1));
    const int segs = max(1, (int)(((long long)e - b + a.seg - 1) / a.seg)), first = first_item(a, n);
    if (i >= per || segs < 2) return;
    const long long items = a.pack.N + (long long)(a.pack.T / a.seg);
    const int c = (int)(i / a.Ns);
    float rate[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
        rate[j] = in_range(i + j, 1, per, a.pack.status) ? rate_of(a.A_log[i + j]) : 0.f;
    float *rec = kBackward ? a.rec_g : a.rec_h;
    auto read = [&](int seg) { return load_vec<4>(rec, (first + seg) * per + i, items * per, a.pack.status); };
    auto write = [&](int seg, const Vec<float, 4> &v) { store_vec<4>(rec, (first + seg) * per + i, items * per, a.pack.status, v); };
    // the j-th segment of the walk, and the last one that it reads
    auto segment = [&](int j) { return kBackward ? segs - 1 - j : j; };
    const Vec<float, 4> start = read(segs - 1);
    Vec<float, 4> run = read(segment(0));
    constexpr int U = 8;
    for (int j0 = 1; j0 < segs; j0 += U) {
        Vec<float, 4> end[U];
        float d[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int seg = segment(j0 + u);
            // (the last one has no decay: nothing is behind it that reads it)
            if (j0 + u >= segs - 1) continue;
            end[u] = read(seg);
            d[u] = load_vec<1>(a.rec_d, (first + seg) * (long long)a.C + c, items * a.C, a.pack.status).x[0];
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (j0 + u >= segs) break;
            write(segment(j0 + u), run);
            if (j0 + u >= segs - 1) break;
#pragma unroll
            for (int k = 0; k < 4; ++k) run.x[k] = fmaf(exp2_of(rate[k] * d[u]), run.x[k], end[u].x[k]);
        }
    }
    if (!kBackward) write(0, start);
}

// One token for each of `rows` rows, one after another (the rates are formed once, the next row is read while
// this one is computed).  A thread has four states of K channels in turn, so that of its L lanes the first K
// form d, the gate and the output of one channel each.  Bound by HBM, the states read and written once.
template <int NS>
struct StepShape {
    static constexpr int L = NS / 4, K = L < 4 ? L : 4, kStart = 256 / L, CB = kStart * K;
    static constexpr int kBlocks = NS == 8 ? 3 : 2;   // of an SM
};

template <typename T, int NS, bool kWide>
__global__ void __launch_bounds__(256, StepShape<NS>::kBlocks) k_scan_step(const __grid_constant__ ScanArgs a, int across, int rows) {
    using Shape = StepShape<NS>;
    constexpr int L = Shape::L, K = Shape::K, kStart = Shape::kStart;
    const int q = threadIdx.x % L, lane = threadIdx.x % 32;
    const int c0 = ((int)(blockIdx.x % across) * kStart + (int)threadIdx.x / L) * K, c = c0 + q;   // c: the lane's own
    const int b0 = (int)(blockIdx.x / across) * rows, b1 = min(b0 + rows, a.pack.T);
    const int per_group = a.C / a.G;
    const bool mine = q < K && c < a.C;
    const long long extent = (long long)a.pack.T * a.C, states = (long long)a.slots.num_slots * a.C * NS;
    float rate[K][4];
#pragma unroll
    for (int i = 0; i < K; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const long long at = (long long)(c0 + i) * NS + 4 * q + j;
            rate[i][j] = c0 + i < a.C && in_range(at, 1, (long long)a.C * NS, a.pack.status)
                             ? rate_of(a.A_log[at])
                             : 0.f;
        }
    const float bias = mine && a.dt_bias ? a.dt_bias[c] : 0.f, skip = mine && a.D ? a.D[c] : 0.f;
    T *y = static_cast<T *>(a.y);
    auto own = [&](const void *p, long long stride, int b) {
        return mine && p ? as_float(load_vec<1>(static_cast<const T *>(p), b * stride + c, (a.pack.T - 1) * stride + a.C, a.pack.status).x[0]) : 0.f;
    };
    auto shared = [&](const void *p, long long stride, int b, int i, float (&out)[4]) {
        const int g = min(c0 + i, a.C - 1) / per_group;
        const long long at = b * stride + g * NS + 4 * q, n = (a.pack.T - 1) * stride + (long long)a.G * NS;
        if (kWide) {
            const Vec<T, 4> v = load_vec<4>(static_cast<const T *>(p), at, n, a.pack.status);
#pragma unroll
            for (int j = 0; j < 4; ++j) out[j] = as_float(v.x[j]);
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) out[j] = as_float(load_vec<1>(static_cast<const T *>(p), at + j, n, a.pack.status).x[0]);
        }
    };
    const bool one_group = c0 / per_group == min(c0 + K - 1, a.C - 1) / per_group;
    struct Row {
        int slot;
        Vec<float, 4> h[K];
        float x, dt, z, B[4], C[4];
    };
    auto read = [&](int b, Row &r) {
        r.slot = slot_of(a.slots, b);
        if (r.slot < 0) return;
#pragma unroll
        for (int i = 0; i < K; ++i)
            if (c0 + i < a.C) r.h[i] = load_vec<4>(a.s1, ((long long)r.slot * a.C + c0 + i) * NS + 4 * q, states, a.pack.status);
        r.x = own(a.x, a.xs, b);
        r.dt = own(a.dt, a.dts, b);
        r.z = own(a.z, a.zs, b);
        shared(a.B, a.bs, b, 0, r.B);
        shared(a.Cm, a.cs, b, 0, r.C);
    };
    Row r, next;
    read(b0, r);
    for (int b = b0; b < b1; ++b) {
        // (no two active rows have one slot: what the next row reads this one does not write)
        if (b + 1 < b1) read(b + 1, next);
        if (r.slot < 0) {   // (the same for all threads of the block)
            if (threadIdx.x == 0 && a.slots.status && a.slots.idx[b] >= a.slots.num_slots) *a.slots.status = 1;
            if (mine) store_vec<1>(y, (long long)b * a.C + c, extent, a.pack.status, Vec<T, 1>{{as_type<T>(0.f)}});
            r = next;
            continue;
        }
        const float d = softplus_of(r.dt + bias), dx = d * r.x;
        float sums[K][1];
#pragma unroll
        for (int i = 0; i < K; ++i) {
            const float di = __shfl_sync(0xffffffffu, d, lane - q + i), dxi = __shfl_sync(0xffffffffu, dx, lane - q + i);
            if (i > 0 && !one_group) {
                shared(a.B, a.bs, b, i, r.B);
                shared(a.Cm, a.cs, b, i, r.C);
            }
            sums[i][0] = 0.f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                r.h[i].x[j] = fmaf(exp2_of(fmaf(di, rate[i][j], kLift)), r.h[i].x[j], dxi * r.B[j]);
                sums[i][0] = fmaf(r.C[j], r.h[i].x[j], sums[i][0]);
            }
            if (c0 + i < a.C) store_vec<4>(a.s1, ((long long)r.slot * a.C + c0 + i) * NS + 4 * q, states, a.pack.status, r.h[i]);
        }
        lane_sums<L, K, 1>(sums, q);
        float out = fmaf(skip, r.x, sums[0][0]);
        if (a.z) out *= r.z * sigmoid_of(r.z);
        if (mine) store_vec<1>(y, (long long)b * a.C + c, extent, a.pack.status, Vec<T, 1>{{as_type<T>(out)}});
        r = next;
    }
}

template <typename T, int NS, bool kWide, WalkFor kFor>
cudaError_t scan_kernel(const ScanArgs &a, cudaStream_t s) {
    using Shape = WalkShape<NS, kFor>;
    const long long blocks = scan_items(a.pack.N, a.pack.T, a.seg) * scan_across<Shape::CB>(a);
    const unsigned grid = (unsigned)(blocks + (kFor == kOutputs && a.pack.status ? 1 : 0));
    constexpr int bytes = (int)sizeof(ScanTiles<T, NS, kFor>), threads = 2 * Shape::kHalf;
    const cudaError_t e = cudaFuncSetAttribute(k_scan_fwd<T, NS, kWide, kFor>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    k_scan_fwd<T, NS, kWide, kFor><<<grid, threads, bytes, s>>>(a);
    return cudaGetLastError();
}

template <typename T, int NS, WalkFor kFor>
cudaError_t scan(const ScanArgs &a, cudaStream_t s) {
    return scan_wide(a, 8) ? scan_kernel<T, NS, true, kFor>(a, s) : scan_kernel<T, NS, false, kFor>(a, s);
}

template <typename T, int NS>
cudaError_t step(const ScanArgs &a, int batch, cudaStream_t s) {
    using Shape = StepShape<NS>;
    const int across = (a.C + Shape::CB - 1) / Shape::CB;
    // (256 rows x 4096 x 16, cold: 14 rows a block, one wave, 33 us; 8 rows, 1.7 waves, 36; one row after another, not
    // read ahead, 42)
    const int rows = step_rows(batch, across, 152 * Shape::kBlocks);
    const unsigned grid = (unsigned)((batch + rows - 1) / rows * (long long)across);
    auto fits = [](const void *p, long long stride) {
        return reinterpret_cast<uintptr_t>(p) % (4 * sizeof(T)) == 0 && stride % 4 == 0;
    };
    if (fits(a.B, a.bs) && fits(a.Cm, a.cs)) k_scan_step<T, NS, true><<<grid, 256, 0, s>>>(a, across, rows);
    else k_scan_step<T, NS, false><<<grid, 256, 0, s>>>(a, across, rows);
    return cudaGetLastError();
}

template <WalkFor kFor>
cudaError_t scan_of(const ScanArgs &a, cudaStream_t s) {
    if (a.f32) return a.Ns == 8 ? scan<float, 8, kFor>(a, s) : a.Ns == 16 ? scan<float, 16, kFor>(a, s) : scan<float, 32, kFor>(a, s);
    return a.Ns == 8 ? scan<bf16, 8, kFor>(a, s) : a.Ns == 16 ? scan<bf16, 16, kFor>(a, s) : scan<bf16, 32, kFor>(a, s);
}

}  // namespace

cudaError_t launch_scan_marks(const ScanArgs &a, cudaStream_t s) { return scan_of<kMarks>(a, s); }

cudaError_t launch_scan_join(const ScanArgs &a, bool backward, cudaStream_t s) {
    const int across = (int)(((long long)a.C * a.Ns / 4 + 127) / 128);
    const unsigned grid = (unsigned)((long long)a.pack.N * across);
    if (backward) k_scan_join<true><<<grid, 128, 0, s>>>(a, across);
    else k_scan_join<false><<<grid, 128, 0, s>>>(a, across);
    return cudaGetLastError();
}

cudaError_t launch_scan_fwd(const ScanArgs &a, cudaStream_t s) {
    if (a.seg <= a.pack.T) {
        cudaError_t e = scan_of<kEnds>(a, s);
        if (e == cudaSuccess) e = launch_scan_join(a, false, s);
        if (e != cudaSuccess) return e;
    }
    return scan_of<kOutputs>(a, s);
}

cudaError_t launch_scan_step(const ScanArgs &a, int batch, cudaStream_t s) {
    if (a.f32) return a.Ns == 8 ? step<float, 8>(a, batch, s) : a.Ns == 16 ? step<float, 16>(a, batch, s) : step<float, 32>(a, batch, s);
    return a.Ns == 8 ? step<bf16, 8>(a, batch, s) : a.Ns == 16 ? step<bf16, 16>(a, batch, s) : step<bf16, 32>(a, batch, s);
}

}  // namespace gdn
